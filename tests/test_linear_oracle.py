"""Pins of the 64-bit definitions of the linear-attention layer's operators."""
import numpy as np
import pytest

from oracle import linear as ref


def test_norm_pins():
    x = np.array([[3.0, -4.0, 0.0, 0.0]])
    w = np.array([1.0, 2.0, 3.0, 4.0])
    assert np.allclose(ref.rms_norm(x, w, eps=0.0)[0], [[1.2, -3.2, 0, 0]])           # rms = 2.5
    assert np.allclose(ref.rms_norm(x, w - 1.0, eps=0.0, offset=1.0)[0], [[1.2, -3.2, 0, 0]])
    assert np.allclose(ref.rms_norm(x - 1.0, w, residual=np.ones((1, 4)), eps=0.0)[0], [[1.2, -3.2, 0, 0]])
    assert np.allclose(ref.rms_norm(x, w, gate=np.zeros((1, 4)), act="sigmoid", eps=0.0)[0], [[0.6, -1.6, 0, 0]])
    assert np.allclose(ref.rms_norm(x, w, gate=np.full((1, 4), 40.0), eps=0.0)[0], [[48.0, -128.0, 0, 0]])
    assert np.allclose(ref.rms_norm(x, w, residual=np.ones((1, 4)), scale=-2.0, eps=0.0, after=True)[0],
                       [[-1.4, 7.4, 1, 1]])


def test_conv_is_numpy_convolve():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((9, 3)), rng.standard_normal((3, 4))
    state = rng.standard_normal((2, 3, 3))
    out, new, _ = ref.short_conv(x, w, state, [1], [0, 9], silu=False)
    for c in range(3):
        line = np.concatenate([state[1, :, c], x[:, c]])
        assert np.allclose(out[:, c], np.convolve(line, w[c][::-1], "valid"))
        assert np.array_equal(new[1, :, c], line[-3:])
    assert np.array_equal(new[0], state[0])
    # a part at a time gives the same
    a, mid, _ = ref.short_conv(x[:2], w, state, [1], [0, 2], silu=False)
    b, end, _ = ref.short_conv(x[2:], w, mid, [1], [0, 7], silu=False)
    assert np.allclose(np.concatenate([a, b]), out) and np.array_equal(end, new)


def test_delta_with_unit_steps_is_a_dictionary():
    """No decay, beta 1 and orthonormal keys: the state stores values by key, a key written again is overwritten."""
    k = np.eye(4)[[0, 2, 0]][:, None]
    v = np.arange(9.0).reshape(3, 1, 3)
    one, zero = np.ones((3, 1)), np.zeros((3, 1))
    out, new, _, _ = ref.gated_delta(k, k, v, zero, one, np.zeros((1, 1, 3, 4)), [0], [0, 3], 1.0)
    assert np.array_equal(out, v)
    assert np.array_equal(new[0, 0], np.stack([v[2, 0], np.zeros(3), v[1, 0], np.zeros(3)], axis=1))


@pytest.mark.parametrize("beta", [0.0, 0.3])
def test_delta_without_correction_is_decayed_linear_attention(beta):
    """Keys orthogonal to all before them: o_t = sum_j exp(G_t - G_j) beta (q_t . k_j) v_j."""
    rng = np.random.default_rng(2)
    n = 6
    k = np.linalg.qr(rng.standard_normal((8, 8)))[0][:n, None]
    q, v, g = rng.standard_normal((n, 1, 8)), rng.standard_normal((n, 2, 3)), -rng.random((n, 2))
    out, _, _, _ = ref.gated_delta(q, k, v, g, np.full((n, 2), beta), np.zeros((1, 2, 3, 8)), [0], [0, n], 0.5)
    G = np.cumsum(g, axis=0)
    for h in range(2):
        P = np.tril(np.exp(G[:, None, h] - G[None, :, h])) * (q[:, 0] @ k[:, 0].T)
        assert np.allclose(out[:, h], 0.5 * beta * P @ v[:, h])


def test_delta_chunk_form():
    """The whole sequence as one chunk: U = (I + A)^-1 beta (V - e^G K S), as the definition has it token by token."""
    rng = np.random.default_rng(3)
    n, D, E = 12, 16, 5
    q, k = rng.standard_normal((2, n, 1, D))
    v, g, b, S = rng.standard_normal((n, 1, E)), -rng.random((n, 1)), rng.random((n, 1)), rng.standard_normal((1, 1, E, D))
    out, new, _, _ = ref.gated_delta(q, k, v, g, b, S, [0], [0, n], D ** -0.5, norm=True)
    q, k = (x[:, 0] / np.sqrt((x[:, 0] ** 2).sum(-1, keepdims=True) + 1e-6) for x in (q, k))
    G = np.cumsum(g[:, 0])
    decay = np.exp(G[:, None] - G[None])
    A = np.tril(b * decay * (k @ k.T), -1)
    U = np.linalg.solve(np.eye(n) + A, b * (v[:, 0] - np.exp(G)[:, None] * (k @ S[0, 0].T)))
    assert np.allclose(out[:, 0], D ** -0.5 * (np.exp(G)[:, None] * (q @ S[0, 0].T) + np.tril(decay * (q @ k.T)) @ U))
    assert np.allclose(new[0, 0], np.exp(G[-1]) * S[0, 0] + (np.exp(G[-1] - G)[:, None] * U).T @ k)


def test_raw_gates_and_beginnings():
    rng = np.random.default_rng(4)
    n = 3
    q, k = rng.standard_normal((2, n, 1, 4))
    v, a, b, S = rng.standard_normal((n, 2, 3)), rng.standard_normal((n, 2)), rng.standard_normal((n, 2)), \
        rng.standard_normal((4, 2, 3, 4))
    al, dt = np.array([0.0, 1.0]), np.array([-1.0, 2.0])
    raw = ref.gated_delta(q, k, v, a, b, S, [2], [0, n], 1.0, a_log=al, dt_bias=dt)
    plain = ref.gated_delta(q, k, v, -np.exp(al) * np.log(1 + np.exp(a + dt)), 1 / (1 + np.exp(-b)), S, [2], [0, n], 1.0)
    assert np.allclose(raw[0], plain[0]) and np.allclose(raw[1], plain[1])
    zero = ref.gated_delta(q, k, v, -np.abs(a), b, 0 * S, [2], [0, n], 1.0)
    for kw in (dict(slots=[-1], dst=[2]), dict(slots=[2], past=[0])):
        got = ref.gated_delta(q, k, v, -np.abs(a), b, S, kw["slots"], [0, n], 1.0, past=kw.get("past"), dst=kw.get("dst"))
        assert np.array_equal(got[0], zero[0]) and np.array_equal(got[1][2], zero[1][2])
        assert np.array_equal(got[1][3], S[3])
    got = ref.gated_delta(q, k, v, -np.abs(a), b, S, [1], [0, 0], 1.0, dst=[3])
    assert np.isnan(got[0]).all() and np.array_equal(got[1][3], S[1])
