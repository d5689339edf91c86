"""The paged-cache operators' definitions in 64 bits (numpy), one query row and
one key at a time where that is what the definition says.  TEST INFRASTRUCTURE
ONLY, like the rest of this package.

Arrays are float64 unless said otherwise; the cache is [pages, kv_heads,
page_size, D], key j of sequence b in slot j % page_size of page
table[b][j // page_size].  Query i of a sequence's n sits at position
len - n + i and sees key j when 0 <= j <= position and, with window > 0,
j > position - window.
"""
from __future__ import annotations

import numpy as np


def rope(x, positions, inv_freq, factor, interleaved):
    """x [T, heads, D] turned by positions[t] * inv_freq[i]; len(inv_freq) pairs."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = (factor * np.cos(ang))[:, None], (factor * np.sin(ang))[:, None]
    ia = 2 * np.arange(half) if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = b * c + a * s
    return x


def rope_frequencies(rot_dim, base, scaling="none", factor=1.0, original_len=0, turns_fast=32.0, turns_slow=1.0):
    i = np.arange(rot_dim // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-2 * i / rot_dim)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        def index_of(turns):   # base^(-2 i / r) * original_len = 2 pi turns
            return rot_dim / 2 * np.log(original_len / (2 * np.pi * turns)) / np.log(base)
        lo = max(np.floor(index_of(turns_fast)), 0.0)
        hi = min(np.ceil(index_of(turns_slow)), rot_dim - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * np.log(factor) + 1.0
    return f, 1.0


def sequence(cache, table_row, length):
    """Keys 0 .. length - 1 of one sequence: [kv_heads, length, ...]."""
    page = cache.shape[2]
    j = np.arange(length)
    return np.moveaxis(cache[np.asarray(table_row)[j // page], :, j % page], 1, 0)


def _scores(q, keys, scale, window, n, length):
    """[n, heads, keys] scores, -inf where unseen, and the sums of |q k| scale."""
    T, Hq, D = q.shape
    g = Hq // keys.shape[0]
    k = np.repeat(keys, g, axis=0)                                   # [Hq, L, D]
    s = scale * np.einsum("nhd,hld->nhl", q, k)
    a = abs(scale) * np.einsum("nhd,hld->nhl", np.abs(q), np.abs(k))
    pos = (length - n + np.arange(n))[:, None]
    j = np.arange(length)[None]
    seen = j <= pos
    if window:
        seen &= j > pos - window
    return np.where(seen[:, None], s, -np.inf), a, seen


def attention(q, k_cache, v_cache, table, lens, q_start, scale, window=0):
    """(out, lse, sum p |v|, largest sum |q k| scale) per row."""
    T, Hq, D = q.shape
    out, A = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, S = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b in range(len(lens)):
        q0, n, L = q_start[b], q_start[b + 1] - q_start[b], int(lens[b])
        if n == 0 or L == 0:
            continue
        keys, vals = sequence(k_cache, table[b], L), sequence(v_cache, table[b], L)
        g = Hq // keys.shape[0]
        s, a, seen = _scores(q[q0:q0 + n], keys, scale, window, n, L)
        m = s.max(axis=-1)
        with np.errstate(invalid="ignore", divide="ignore"):
            p = np.where(np.isfinite(s), np.exp(s - m[..., None]), 0.0)
            l = p.sum(-1)
            lse[q0:q0 + n] = np.where(l > 0, m + np.log(l), -np.inf)
            p /= np.where(l > 0, l, 1.0)[..., None]
        v = np.repeat(vals, g, axis=0)
        out[q0:q0 + n] = np.einsum("nhl,hld->nhd", p, v)
        A[q0:q0 + n] = np.einsum("nhl,hld->nhd", p, np.abs(v))
        S[q0:q0 + n] = np.where(seen[:, None], a, 0).max(-1)
    return out, lse, A, S


def mass(q, k_cache, table, lens, q_start, scale, window, lse, decay, mass_in, mass_out):
    """mass_out (float64, changed in place) and the added sums, same shape."""
    added = np.zeros_like(mass_out)
    page = k_cache.shape[2]
    for b in range(len(lens)):
        q0, n, L = q_start[b], q_start[b + 1] - q_start[b], int(lens[b])
        if L == 0:
            continue
        keys = sequence(k_cache, table[b], L)
        Hkv = keys.shape[0]
        tot = np.zeros((Hkv, L))
        if n:
            s, _, _ = _scores(q[q0:q0 + n], keys, scale, window, n, L)
            z = lse[q0:q0 + n, :, None]
            with np.errstate(invalid="ignore"):
                w = np.where(np.isfinite(s) & np.isfinite(z), np.exp(s - z), 0.0)
            tot = w.reshape(n, Hkv, -1, L).sum(axis=(0, 2))
        for j in range(L):
            pg, sl = table[b][j // page], j % page
            added[pg, :, sl] = tot[:, j]
            mass_out[pg, :, sl] = decay * mass_in[pg, :, sl] + tot[:, j]
    return mass_out, added


def evict(mass, table, lens, budget, recent):
    """keep [B][kv_heads] as lists of kept key indices, ascending."""
    keep = []
    for b, L in enumerate(lens):
        L = int(L)
        n = min(L, budget)
        r = min(recent, n)
        m = sequence(mass, table[b], L)
        rows = []
        for h in range(m.shape[0]):
            v = [(-np.inf if np.isnan(x) else x) for x in m[h, :L - r].tolist()]
            nan = [np.isnan(x) for x in m[h, :L - r].tolist()]
            best = sorted(range(L - r), key=lambda j: (nan[j], -v[j], j))[:n - r]
            rows.append(sorted(best) + list(range(L - r, L)))
        keep.append(rows)
    return keep
