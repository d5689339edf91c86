"""The linear-attention layer's operators in 64 bits (numpy), token by token.
TEST INFRASTRUCTURE ONLY, like the rest of this package.

Sequences of new tokens start[b] .. start[b + 1] - 1; state[slots[b]] is read
(zeros where slots[b] < 0 or past[b] == 0) and the new state goes to dst[b]
(nowhere where negative).  Every function returns its outputs beside the sums of
magnitudes that their error bounds are made of.
"""
from __future__ import annotations

import numpy as np


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-np.asarray(x, dtype=np.float64)))


def softplus(x):
    x = np.asarray(x, dtype=np.float64)
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def rms_norm(x, weight, residual=None, scale=1.0, gate=None, act="silu", eps=1e-6, offset=0.0, after=False):
    """(out, h): rows over the last axis."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(weight, dtype=np.float64) + offset
    h = x if after or residual is None else residual + scale * x
    y = h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps) * w
    if gate is not None:
        y = y * sigmoid(gate) * (gate if act == "silu" else 1.0)
    if after:
        y = scale * y + (0.0 if residual is None else residual)
    return y, h


def _initial(state, slots, past, b):
    if slots[b] < 0 or (past is not None and past[b] == 0):
        return np.zeros(state.shape[1:])
    return np.array(state[slots[b]])


def short_conv(x, weight, state, slots, start, bias=None, silu=True, past=None, dst=None):
    """(out [T, C] with NaN in rows of no sequence, new state, sums of magnitudes [T, C])."""
    x, weight = np.asarray(x, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    new, dst = np.array(state, dtype=np.float64), slots if dst is None else dst
    out, size = np.full(x.shape, np.nan), np.zeros(x.shape)
    W = weight.shape[1]
    for b in range(len(slots)):
        line = np.concatenate([_initial(np.asarray(state, dtype=np.float64), slots, past, b), x[start[b]:start[b + 1]]])
        for i in range(start[b + 1] - start[b]):
            y = (weight.T * line[i:i + W]).sum(0)
            size[start[b] + i] = np.abs(weight.T * line[i:i + W]).sum(0)
            if bias is not None:
                y = y + bias
                size[start[b] + i] += np.abs(bias)
            out[start[b] + i] = y * sigmoid(y) if silu else y
        if dst[b] >= 0:
            new[dst[b]] = line[len(line) - (W - 1):]
    return out, new, size


def gated_delta(q, k, v, g, beta, state, slots, start, scale, norm=False, a_log=None, dt_bias=None, past=None, dst=None):
    """(out [T, Hv, Dv] with NaN in rows of no sequence, new state, reach, memory): `reach` [Hv] the
    largest length of a row of S plus the largest |v|, `memory` [Hv] the largest sum over the tokens so
    far of what their decays leave of each."""
    q, k, v, g, beta = (np.array(x, dtype=np.float64) for x in (q, k, v, g, beta))
    if a_log is not None:
        g, beta = -np.exp(a_log) * softplus(g + dt_bias), sigmoid(beta)
    if norm:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6) for x in (q, k))
    Hv, group = v.shape[1], v.shape[1] // q.shape[1]
    q, k = np.repeat(q, group, axis=1), np.repeat(k, group, axis=1)
    new, dst = np.array(state, dtype=np.float64), slots if dst is None else dst
    out = np.full(v.shape, np.nan)
    reach, memory = np.zeros(Hv), np.ones(Hv)
    for b in range(len(slots)):
        S = _initial(np.asarray(state, dtype=np.float64), slots, past, b)
        left, top = np.ones(Hv), np.abs(v[start[b]:start[b + 1]]).max((0, 2), initial=0.0)
        reach = np.maximum(reach, np.sqrt((S * S).sum(-1)).max(-1) + top)
        for t in range(start[b], start[b + 1]):
            S = S * np.exp(g[t])[:, None, None]
            u = beta[t][:, None] * (v[t] - np.einsum("hvk,hk->hv", S, k[t]))
            S = S + u[:, :, None] * k[t][:, None, :]
            out[t] = scale * np.einsum("hvk,hk->hv", S, q[t])
            left = left * np.exp(g[t]) + 1.0
            memory, reach = np.maximum(memory, left), np.maximum(reach, np.sqrt((S * S).sum(-1)).max(-1) + top)
        if dst[b] >= 0:
            new[dst[b]] = S
    return out, new, reach, memory
