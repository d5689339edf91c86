"""The linear-attention layer's operators on the GPU against their definitions in 64 bits.

Bounds.  A rounding to bf16 is off by at most 2^-8 of the value (half a step), one
to fp32 by 2^-24.  Norm: the sum of squares of D terms, its root and the three
products add at most (D / 8 + 40) 2^-24 in relative terms (8 partial sums at
least a row), a residual's sum 2^-24 of its parts, and a gate's exponential
2^-16.  Convolution: 8 products and sums, 2^-20 of the sum of magnitudes; what it
does to y passes through an activation whose slope is at most 1.1, and whose own
relative error is 2^-16 from the exponential.  The delta rule: with R the
largest row of S plus the largest |v|, a token adds errors of at most 2^-17 R to
a row (two dot products of Dk <= 128 terms, an update; in the chunk form the
same products, and those from piece to piece, with operands in parts that carry 2^-17
of each factor), decays shrink them and the
correction does not grow them (|k| <= 1, beta <= 1), so a row of the final state is
off by at most `memory` 2^-17 R, `memory` the largest sum of what the decays
leave.  out reads that with |q| <= 1, and in the chunk form adds products of
bf16 roundings within a chunk: at most 2^-7 of scale memory R beside its own
rounding.
"""
import numpy as np
import pytest
import torch

from oracle import linear as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def tern():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_gemv_gemm_gb300 import build
    build.build()
    import bit_gemv_gemm_gb300 as t
    return t


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(shape, g, kind=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(kind)


def within(got, want, bound, what):
    err = np.abs(f64(got) - want)
    bad = ~(err <= bound)
    if bad.any():
        i = np.argwhere(bad)[:4].tolist()
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first {i}: got {f64(got)[bad][:4]}, "
                             f"want {want[bad][:4]}, bound {np.broadcast_to(bound, want.shape)[bad][:4]}")


# ---------------------------------------------------------------------------
# rms_norm
# ---------------------------------------------------------------------------

KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}


def check_norm(tern, x, w, out, residual=None, scale=1.0, gate=None, act="silu", offset=0.0, after=False, res_out=None,
               residual_was=None):
    D = x.shape[-1]
    r = f64(residual) if residual_was is None else residual_was
    want, h = ref.rms_norm(f64(x), f64(w), r, scale, f64(gate), act, EPS, offset, after)
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -23
    rel = (D / 8 + 40) * 2.0 ** -24 + (2.0 ** -15 if gate is not None else 0.0)
    parts = np.abs(scale * f64(x)) + (0 if r is None else np.abs(r))
    own = want if not after else want - (0 if r is None else r)
    bound = half * np.abs(want) + 2 * rel * np.abs(own) + 1e-30
    if not after:   # h's own rounding, through the same factors
        inv = 1 / np.sqrt(np.mean(h * h, -1, keepdims=True) + EPS)
        z = 1.0 if gate is None else np.abs(f64(gate)) + 1.0
        bound = bound + 2.0 ** -23 * parts * inv * (np.abs(f64(w)) + abs(offset)) * z * 2
    within(out, want, bound, "norm")
    if res_out is not None:
        half = 2.0 ** -8 if res_out.dtype == torch.bfloat16 else 2.0 ** -24
        within(res_out, h, half * np.abs(h) + 2.0 ** -23 * parts, "residual")


@pytest.mark.parametrize("T,heads,D", [(1, 1, 8), (3, 1, 64), (7, 5, 72), (33, 3, 128), (5, 7, 176), (9, 1, 256),
                                       (4, 2, 264), (6, 1, 512), (3, 1, 520), (2, 1, 1000), (700, 1, 1032), (5, 1, 5120),
                                       (3, 1, 8192), (2, 2, 8200), (2, 1, 17408), (1, 1, 32768), (1000, 9, 128)])
@pytest.mark.parametrize("kinds", ["f32", "bf16"])
def test_norm_sizes(tern, T, heads, D, kinds):
    g, kind = gen(T + D), KINDS[kinds]
    x, r, z = rand((T, heads, D), g, kind), 3 * rand((T, heads, D), g, kind), rand((T, heads, D), g, kind)
    r = r.to(kind)
    w = 1 + 0.3 * rand(D, g)
    out = tern.rms_norm(x, w)
    check_norm(tern, x, w, out)
    new = torch.empty_like(r)
    out = tern.rms_norm(x, w, residual=r, scale=0.5, gate=z, residual_out=new)
    check_norm(tern, x, w, out, r, 0.5, z, res_out=new)
    out = tern.rms_norm(x, w, residual=r, scale=-0.5, gate=z, gate_act="sigmoid", weight_offset=1.0, after=True)
    assert out.dtype == kind
    check_norm(tern, x, w, out, r, -0.5, z, "sigmoid", 1.0, True)


@pytest.mark.parametrize("T,heads,D", [(41, 3, 128), (23, 2, 48), (11, 1, 400), (330, 1, 1288), (310, 1, 2568), (307, 1, 8200)])
@pytest.mark.parametrize("residual", [None, "f32", "bf16"])
@pytest.mark.parametrize("gate", [None, "f32", "bf16"])
def test_norm_types(tern, T, heads, D, residual, gate):
    """Every mix of types, before and after a block, the new residual over the old."""
    g = gen(T + D)
    w, z = 1 + 0.3 * rand(D, g), None if gate is None else rand((T, heads, D), g, KINDS[gate])
    for xk in KINDS.values():
        for ok in KINDS.values():
            x, r = rand((T, heads, D), g, xk), None if residual is None else 3 * rand((T, heads, D), g, KINDS[residual])
            was = None if r is None else f64(r)
            out = tern.rms_norm(x, w, residual=r, scale=0.5, gate=z, after=True, out_dtype=ok)
            assert out.dtype == ok
            check_norm(tern, x, w, out, r, 0.5, z, after=True)
            out = tern.rms_norm(x, w, residual=r, scale=1.0 if r is None else 0.5, gate=z, residual_out=r, out_dtype=ok)
            check_norm(tern, x, w, out, None, 1.0 if r is None else 0.5, z, res_out=r, residual_was=was)
    assert tern.device_error() == 0


def test_norm_in_place_strided_and_mixed(tern):
    g = gen(2)
    T, H, D = 37, 4, 128
    wide = rand((T, 64 + H * D + 8), g)
    x = wide[:, 64:64 + H * D].unflatten(1, (H, D))
    z = rand((H, T, D), g, torch.bfloat16).transpose(0, 1)
    r, w = rand((T, H, D), g, torch.bfloat16), rand(D, g)
    was = f64(r)
    out = tern.rms_norm(x, w, residual=r, gate=z, residual_out=r, out_dtype=torch.float32)
    assert out.dtype == torch.float32
    check_norm(tern, x, w, out, r, 1.0, z, res_out=r, residual_was=was)
    # one row of a residual read by all, and the output over the input
    row = rand((1, 5120), g).expand(9, 5120)
    y = rand((9, 5120), g, torch.bfloat16)
    x = y.clone()
    tern.rms_norm(y, torch.ones(5120, device="cuda"), residual=row, out=y)
    check_norm(tern, x, torch.ones(5120), y, row)
    # after a block, over the residual
    r = rand((6, 1024), g)
    was, x = f64(r), rand((6, 1024), g, torch.bfloat16)
    tern.rms_norm(x, torch.ones(1024, device="cuda"), residual=r, scale=0.25, after=True, out=r)
    check_norm(tern, x, torch.ones(1024), r, None, 0.25, after=True, residual_was=was)


def test_norm_rows_alone(tern):
    """A row of zeros, of huge and tiny values, of NaN: none touches another."""
    x = torch.ones((6, 256), device="cuda")
    x[0], x[1], x[2], x[3, 5], x[4] = 0.0, 1e18, 1e-18, float("nan"), -2.0
    w = torch.arange(256, device="cuda").float()
    for D in (256, 2048):
        xx, ww = x.repeat(1, D // 256), w.repeat(D // 256)
        out = f64(tern.rms_norm(xx, ww, out_dtype=torch.float32))
        assert (out[0] == 0).all() and np.isnan(out[3]).all() and np.isfinite(out[[1, 2, 4, 5]]).all()
        assert np.allclose(out[1], f64(ww), rtol=1e-6) and np.allclose(out[4], -f64(ww), rtol=1e-6)
        assert np.abs(out[2] - 1e-15 * f64(ww)).max() < 1e-18


def test_norm_of_no_tokens(tern):
    assert tern.rms_norm(torch.zeros((0, 64), device="cuda"), torch.ones(64, device="cuda")).shape == (0, 64)


# ---------------------------------------------------------------------------
# short_conv
# ---------------------------------------------------------------------------

def sequences(lens, behind=0):
    start = np.cumsum([0] + list(lens))
    return start.tolist(), int(start[-1]) + behind


def check_conv(x, w, bias, silu, before, after, out, sl, start, past=None, dst=None, out_was=None):
    want, new, size = ref.short_conv(f64(x), f64(w), before, sl, start, None if bias is None else f64(bias), silu, past,
                                     dst)
    rows = ~np.isnan(want).all(-1)
    bound = 2.0 ** -8 * np.abs(want) + (1.2 * 2.0 ** -20) * size + (2.0 ** -15 * np.abs(want) if silu else 0) + 1e-30
    within(out[torch.from_numpy(rows).cuda()], want[rows], bound[rows], "conv")
    if out_was is not None:
        assert np.array_equal(f64(out)[~rows], out_was[~rows])
    assert np.array_equal(f64(after), new)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,C", [([1], 8), ([1] * 5, 520), ([0, 2, 3, 1, 0], 64), ([31, 32, 33, 0, 65], 1032),
                                    ([300], 512), ([7, 100, 1], 2048)])
def test_conv(tern, W, kind, lens, C):
    g, B = gen(W + C), len(lens)
    start, T = sequences(lens, behind=3)
    x = rand((T, C + 16), g, kind)[:, 8:8 + C]
    w, bias, pool = rand((C, W), g), rand(C, g), rand((2 * B + 2, W - 1, C), g)
    order = torch.randperm(2 * B + 2, generator=gen(1), device="cuda").tolist()
    sl, dst = order[:B], order[B:2 * B]
    past = [int(b % 3 != 1) for b in range(B)]
    for kw in (dict(), dict(dst=dst), dict(dst=dst, past=past, bias=bias, silu=False)):
        state, before = pool.clone(), f64(pool)
        out = torch.full((T, C), 7.0, dtype=torch.bfloat16, device="cuda")
        tern.short_conv(x, w, state, i32(sl), q_start=i32(start), max_new=max(max(lens), 1), bias=kw.get("bias"),
                        silu=kw.get("silu", True), past=i32(kw.get("past")), dst_slots=i32(kw.get("dst")), out=out)
        check_conv(x, w, kw.get("bias"), kw.get("silu", True), before, state, out, sl, start, kw.get("past"),
                   kw.get("dst"), np.full((T, C), 7.0))
    assert tern.device_error() == 0


def test_conv_equal_lengths_negative_slots_and_a_split(tern):
    g = gen(5)
    x, w, pool = rand((12, 64), g), rand((64, 4), g), rand((3, 3, 64), g)
    state = pool.clone()
    out = tern.short_conv(x, w, state, i32([2, -1, 0]), dst_slots=i32([-1, 1, 0]))
    check_conv(x, w, None, True, f64(pool), state, out, [2, -1, 0], [0, 4, 8, 12], dst=[-1, 1, 0])
    # in one piece and in three
    x, state, whole = rand((70, 64), g, torch.bfloat16), pool.clone(), pool.clone()
    once = tern.short_conv(x, w, whole, i32([1]))
    parts = [tern.short_conv(x[a:b], w, state, i32([1])) for a, b in ((0, 1), (1, 3), (3, 70))]
    assert torch.equal(torch.cat(parts), once) and torch.equal(state, whole)
    assert tern.short_conv(x[:0], w, state, i32([1])).shape == (0, 64) and torch.equal(state, whole)
    assert tern.device_error() == 0


def test_conv_reports_bad_values(tern):
    g = gen(6)
    x, w, pool = rand((4, 64), g), rand((64, 4), g), rand((3, 3, 64), g)
    for sl, dst, start, code in (([0, 3], [1, 2], [0, 2, 4], tern.DEVERR_STATE_SLOT),
                                 ([0, 1], [2, 1 << 30], [0, 2, 4], tern.DEVERR_STATE_SLOT),
                                 ([0, 1], [1, 2], [0, 2, 5], tern.DEVERR_CACHE_SEQUENCE),
                                 ([0, 1], [1, 2], [0, 3, 4], tern.DEVERR_CACHE_SEQUENCE),
                                 ([0, 1], [1, 2], [0, 2, -7], tern.DEVERR_CACHE_SEQUENCE)):
        state = pool.clone()
        tern.short_conv(x, w, state, i32(sl), q_start=i32(start), max_new=2, dst_slots=i32(dst))
        assert tern.device_error() == code
        if code == tern.DEVERR_STATE_SLOT:   # nothing is written in the place of a bad slot
            bad = [s for s in range(3) if s not in dst]
            assert torch.equal(state[bad], pool[bad])
    assert tern.device_error() == 0


# ---------------------------------------------------------------------------
# gated_delta
# ---------------------------------------------------------------------------

HEADS = [(2, 4, 64, 16), (1, 3, 128, 48), (2, 2, 128, 128), (1, 2, 64, 256), (1, 1, 128, 176)]


def delta_inputs(T, Hk, Hv, Dk, Dv, g, raw=False, norm=True):
    x = rand((T, 2 * Hk * Dk + Hv * Dv + 8), g)
    x = x * torch.sigmoid(x)
    if not norm:
        qk = x[:, :2 * Hk * Dk].view(T, 2 * Hk, Dk)
        qk *= 0.99 / (qk.norm(dim=-1, keepdim=True) + 1e-3)
    x = x.bfloat16()
    q, k = x[:, :Hk * Dk].view(T, Hk, Dk), x[:, Hk * Dk:2 * Hk * Dk].view(T, Hk, Dk)
    v = x[:, 2 * Hk * Dk:2 * Hk * Dk + Hv * Dv].view(T, Hv, Dv)
    gates = rand((T, 2 * Hv + 3), g)
    a, b = gates[:, :Hv], gates[:, Hv + 2:2 * Hv + 2]
    if raw:
        return q, k, v, a, b, torch.log(1 + 3 * torch.rand(Hv, generator=g, device="cuda")), rand(Hv, g) - 2
    a.copy_(-0.3 * torch.exp(a))
    b.copy_(torch.sigmoid(b))
    return q, k, v, a, b, None, None


def check_delta(inputs, scale, norm, before, after, out, sl, start, past=None, dst=None, out_was=None):
    q, k, v, g, b, al, dt = (f64(t) for t in inputs)
    want, new, reach, memory = ref.gated_delta(q, k, v, g, b, before, sl, start, scale, norm, al, dt, past, dst)
    rows = ~np.isnan(want).all((1, 2)) if len(want) else np.zeros(0, bool)
    step = 2.0 ** -17 * memory * reach
    longest = max(b - a for a, b in zip(start, start[1:]))
    inside = 2.0 ** -7 * memory * reach if longest > 1 else 0 * reach
    length = 1.0 if norm else max(1.0, np.sqrt((q * q).sum(-1)).max())
    bound = 2.0 ** -8 * np.abs(want) + (abs(scale) * length * (step + 2.0 ** -17 * reach + inside))[None, :, None]
    within(out[torch.from_numpy(rows).cuda()], want[rows], bound[rows], "delta")
    if out_was is not None:
        assert np.array_equal(f64(out)[~rows], out_was[~rows])
    moved = (new != before).any((1, 2, 3))
    assert np.array_equal(f64(after)[~moved], before[~moved])
    within(after[torch.from_numpy(moved).cuda()], new[moved], step[None, :, None, None] + 2.0 ** -23 * np.abs(new[moved]),
           "state")
    # as a whole far nearer than the worst case: roundings to 32 bits alone (2e-7 each, a few of them)
    err = f64(after) - new
    assert np.linalg.norm(err[moved]) <= 4e-6 * np.linalg.norm(new[moved]) + 1e-30
    if rows.any() and longest > 1:
        assert np.linalg.norm((f64(out) - want)[rows]) <= 2.0 ** -8 * np.linalg.norm(want[rows])


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", [[1], [1, 1, 1], [0, 3, 1], [5, 8, 0, 9], [16, 2], [17], [24, 1], [25], [33, 64, 1, 0, 31],
                                  [128, 65, 63], [200, 47], [500], [64, 1100, 0, 513, 300], [1800]])
@pytest.mark.parametrize("raw", [False, True])
def test_delta(tern, heads, lens, raw):
    Hk, Hv, Dk, Dv = heads
    g, B = gen(sum(lens) + Dv), len(lens)
    start, T = sequences(lens, behind=2)
    inputs = delta_inputs(T, *heads, g, raw, norm=raw)
    pool = rand((2 * B + 2, Hv, Dv, Dk), g)
    order = torch.randperm(2 * B + 2, generator=gen(7), device="cuda").tolist()
    sl, dst = order[:B], order[B:2 * B]
    past = [int(b % 3 != 2) for b in range(B)]
    scale = Dk ** -0.5
    for kw in (dict(), dict(dst=dst, past=past)):
        state, before = pool.clone(), f64(pool)
        out = torch.full((T, Hv, Dv), 7.0, dtype=torch.bfloat16, device="cuda")
        tern.gated_delta(*inputs[:5], state, i32(sl), q_start=i32(start), max_new=max(max(lens), 1), qk_norm=raw,
                         a_log=inputs[5], dt_bias=inputs[6], past=i32(kw.get("past")), dst_slots=i32(kw.get("dst")),
                         out=out)
        assert tern.device_error() == 0
        check_delta(inputs, scale, raw, before, state, out, sl, start, kw.get("past"), kw.get("dst"),
                    np.full(out.shape, 7.0))


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", [[25], [64], [33, 64, 1, 0, 31], [200, 47], [700, 65]])
def test_delta_outputs_are_rounded_once(tern, heads, lens):
    """A chunk's products leave less of an output than its own rounding does: it is the rounded value, but
    where that lies next to a border.

    Every factor of Q S^T and P U is two bf16 values (2^-17 of it) and their smallest product is left out
    (2^-18); with what U and S are off by, a few times 2^-17 of what goes into an output, e <= 2^-13 of it here
    (it is the norm of a sum of at least as many parts).  A rounding changes to the neighbour, a step of at
    most 2^-7 of the value away, for a share e / step of the values: the mean square of what changes is at
    most e 2^-7, its root 2^-10.  One bf16 for P (e = 2^-9.5) would change half of them, 2^-8.3."""
    Hk, Hv, Dk, Dv = heads
    g, B = gen(sum(lens) + Dk), len(lens)
    start, T = sequences(lens)
    q, k, v, a, b, _, _ = delta_inputs(T, *heads, g)
    pool = 0.1 * rand((B, Hv, Dv, Dk), g)
    state, sl = pool.clone(), list(range(B))
    out = tern.gated_delta(q, k, v, a, b, state, i32(sl), q_start=i32(start), max_new=max(lens), qk_norm=True)
    assert tern.device_error() == 0
    want = ref.gated_delta(f64(q), f64(k), f64(v), f64(a), f64(b), f64(pool), sl, start, Dk ** -0.5, True)[0]
    rounded = f64(torch.from_numpy(want).to(torch.bfloat16))
    assert np.linalg.norm(f64(out) - rounded) <= 2.0 ** -10 * np.linalg.norm(want)


def delta_call(tern, inputs, scale, state, sl, start, max_new, ws_bytes):
    """The C entry point with a workspace of `ws_bytes` bytes (0: none); its status and output."""
    q, k, v, g, b, al, dt = inputs
    B, T, (pool, Hv, Dv, Dk), at, first = len(sl), q.shape[0], state.shape, i32(sl), i32(start)
    out = torch.full((T, Hv, Dv), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((max(ws_bytes, 1),), 0xFF, dtype=torch.uint8, device="cuda")     # (not a number, wherever it is read)
    status = tern.lib().tern_gated_delta(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q.stride(0), k.stride(0), v.stride(0), g.data_ptr(), g.stride(0),
        b.data_ptr(), b.stride(0), None if al is None else al.data_ptr(), None if dt is None else dt.data_ptr(), scale, 1,
        state.data_ptr(), pool, at.data_ptr(), None, None, first.data_ptr(), B, T, max_new, q.shape[1], Hv, Dk, Dv,
        out.data_ptr(), ws.data_ptr() if ws_bytes else None, ws_bytes, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return status, out


# the most pieces of each: 11, 2 (the root), 2 and 3 (the SMs), as many rows of S as two tiles have, one head alone
@pytest.mark.parametrize("heads,lens", [((1, 1, 64, 16), [8192]), ((1, 2, 128, 128), [512, 3, 0, 511]),
                                        ((5, 15, 64, 96), [700, 65, 640]), ((4, 24, 128, 128), [64 * 17 + 1]),
                                        ((1, 7, 128, 256), [1300, 64]), ((2, 6, 128, 176), [1024, 1025]),
                                        ((1, 40, 64, 64), [577])])
def test_delta_in_pieces_and_whole(tern, heads, lens):
    Hk, Hv, Dk, Dv = heads
    g = gen(21)
    T, B = sum(lens), len(lens)
    start, sl = sequences(lens)[0], list(range(B, 0, -1))
    inputs = delta_inputs(T, Hk, Hv, Dk, Dv, g)
    pool = rand((B + 1, Hv, Dv, Dk), g)
    need = tern.lib().tern_gated_delta_workspace_bytes(B, T, max(lens), Hv, Dk, Dv)
    assert need > 0 and need % 256 == 0
    assert tern.lib().tern_gated_delta_workspace_bytes(B, T, 448, Hv, Dk, Dv) == 0      # too short
    for ws in (need, 0):
        state = pool.clone()
        status, out = delta_call(tern, inputs, Dk ** -0.5, state, sl, start, max(lens), ws)
        assert status == 0 and tern.lib().tern_last_launch_count() in ((2, 3) if ws else (1,))
        assert tern.device_error() == 0
        check_delta(inputs, Dk ** -0.5, True, f64(pool), state, out, sl, start)
    assert delta_call(tern, inputs, Dk ** -0.5, pool.clone(), sl, start, max(lens), need - 256)[0] == 4


@pytest.mark.parametrize("heads", [(1, 2, 64, 48), (2, 2, 128, 128)])
@pytest.mark.parametrize("n", [64, 130, 640])
@pytest.mark.parametrize("kind", ["one key", "two signs", "nearly one", "some zero", "one key, a little decay"])
def test_delta_of_like_keys(tern, heads, n, kind):
    """Keys that depend on one another as far as keys can, full steps and (but in one) no decay: every entry of A
    is 1, -1 or 0 and all of T counts; whole and, of 640 tokens, in pieces.

    Bounds.  A token adds roundings of at most 2^-17 R to a row of S (R its length plus the largest |v|): those
    of its u, of what is taken of the u before it, of its key's share.  The products with I - k k^T do not make
    them grow.  Their sum over n tokens is at most n 2^-17 R; as roundings of no one sign its length is at most
    sqrt(3 n) 2^-17 times that of R.  out reads it with |q| <= 1 and is rounded: 2^-8 at most, in length
    2^-7 / sqrt(12)."""
    Hk, Hv, Dk, Dv = heads
    g = gen(n + Dk)
    q, k, v, a, b, _, _ = delta_inputs(n, *heads, g)
    k = k.clone()
    one = rand((1, Hk, Dk), g)
    if kind in ("one key", "one key, a little decay"):
        k.copy_(one.expand_as(k))
    elif kind == "two signs":
        k.copy_(one * (1 - 2 * (torch.arange(n, device="cuda") % 2)).view(-1, 1, 1))
    elif kind == "nearly one":
        k.copy_(one + 1e-2 * rand(k.shape, g))
    else:
        k[torch.rand(n, generator=g, device="cuda") < 0.4] = 0.0
    a.fill_(-1e-3 if "decay" in kind else 0.0)
    b.fill_(1.0)
    inputs, pool = (q, k, v, a, b, None, None), rand((1, Hv, Dv, Dk), g)
    want, new, reach, _ = ref.gated_delta(f64(q), f64(k), f64(v), f64(a), f64(b), f64(pool), [0], [0, n], Dk ** -0.5, True)
    need = tern.lib().tern_gated_delta_workspace_bytes(1, n, n, Hv, Dk, Dv)
    assert (need > 0) == (n == 640)
    for ws in {0, need}:
        state = pool.clone()
        status, out = delta_call(tern, inputs, Dk ** -0.5, state, [0], [0, n], n, ws)
        assert status == 0 and tern.device_error() == 0
        worst, length = n * 2.0 ** -17 * reach, (3 * n) ** 0.5 * 2.0 ** -17 * np.linalg.norm(reach) * Dv ** 0.5
        within(state, new, worst[None, :, None, None], "state")
        assert np.linalg.norm(f64(state) - new) <= length
        within(out, want, 2.0 ** -8 * np.abs(want) + Dk ** -0.5 * worst[None, :, None], "delta")
        assert np.linalg.norm(f64(out) - want) <= 2.0 ** -7 / 12 ** 0.5 * np.linalg.norm(want) + Dk ** -0.5 * length * n ** 0.5


@pytest.mark.parametrize("n", [1, 6, 70, 640])
def test_delta_extreme_gates(tern, n):
    """Decays of 0 (-inf, far below fp32's least), of 1, steps of 0 and 1, in one sequence."""
    Hk, Hv, Dk, Dv = 1, 2, 128, 32
    g = gen(n)
    inputs = list(delta_inputs(2 * n, Hk, Hv, Dk, Dv, g))
    inputs[3][:, 0] = torch.tensor([0.0, -float("inf"), -1e30, -150.0, -1e-7, 0.0, 0.0])[torch.arange(2 * n) % 7].cuda()
    inputs[3][:, 1] = torch.where(torch.arange(2 * n) % 5 == 3, -90.0, -1e-3).cuda()
    inputs[4][:, 0] = torch.tensor([0.0, 1.0, 1.0, 0.5])[torch.arange(2 * n) % 4].cuda()
    pool = rand((2, Hv, Dv, Dk), g)
    state = pool.clone()
    out = tern.gated_delta(*inputs[:5], state, i32([1, 0]), qk_norm=True)
    assert tern.device_error() == 0
    check_delta(inputs, Dk ** -0.5, True, f64(pool), state, out, [1, 0], [0, n, 2 * n])


def test_delta_negative_slots_shared_reads_and_no_tokens(tern):
    Hk, Hv, Dk, Dv = 1, 2, 64, 32
    g = gen(11)
    for n in (1, 20, 40, 600):
        inputs = delta_inputs(3 * n, Hk, Hv, Dk, Dv, g)
        pool = rand((5, Hv, Dv, Dk), g)
        state = pool.clone()
        out = tern.gated_delta(*inputs[:5], state, i32([1, 1, -1]), dst_slots=i32([2, -1, 4]), qk_norm=True, scale=-2.0)
        check_delta(inputs, -2.0, True, f64(pool), state, out, [1, 1, -1], [0, n, 2 * n, 3 * n], dst=[2, -1, 4])
    # no tokens at all: states move
    state = pool.clone()
    e = [t[:0] for t in inputs[:5]]
    assert tern.gated_delta(*e, state, i32([1, 0]), dst_slots=i32([3, 2]), past=i32([1, 0])).shape == (0, Hv, Dv)
    assert torch.equal(state[3], pool[1]) and not state[2].any() and torch.equal(state[[0, 1, 4]], pool[[0, 1, 4]])
    assert tern.device_error() == 0


def test_delta_in_one_piece_and_in_several(tern):
    """A prompt at once, in unlike parts, and token by token: the same states, within their bounds."""
    heads = (2, 4, 128, 64)
    g = gen(12)
    inputs = delta_inputs(150, *heads, g)
    pool = rand((1, 4, 64, 128), g)
    for cuts in ([0, 150], [0, 64, 65, 100, 150], list(range(0, 151, 3))):
        state, outs = pool.clone(), []
        for a, b in zip(cuts, cuts[1:]):
            outs.append(tern.gated_delta(*[t[a:b] for t in inputs[:5]], state, i32([0]), qk_norm=True))
        check_delta(inputs, 128 ** -0.5, True, f64(pool), state, torch.cat(outs), [0], [0, 150])


@pytest.mark.parametrize("n", [1, 40, 600])
def test_delta_reports_bad_values(tern, n):
    Hk, Hv, Dk, Dv = 1, 2, 64, 32
    g = gen(13)
    inputs = delta_inputs(2 * n, Hk, Hv, Dk, Dv, g)
    pool = rand((3, Hv, Dv, Dk), g)
    for sl, dst, start, code in (([0, 3], [1, 2], [0, n, 2 * n], tern.DEVERR_STATE_SLOT),
                                 ([0, 1], [2, 1 << 30], [0, n, 2 * n], tern.DEVERR_STATE_SLOT),
                                 ([0, 1], [1, 2], [0, n, 2 * n + 1], tern.DEVERR_CACHE_SEQUENCE),
                                 ([0, 1], [1, 2], [-1, n, 2 * n], tern.DEVERR_CACHE_SEQUENCE),
                                 ([0, 1], [1, 2], [0, n, -9], tern.DEVERR_CACHE_SEQUENCE)):
        state = pool.clone()
        tern.gated_delta(*inputs[:5], state, i32(sl), q_start=i32(start), max_new=n, dst_slots=i32(dst), qk_norm=True)
        assert tern.device_error() == code
        if code == tern.DEVERR_STATE_SLOT:
            bad = [s for s in range(3) if s not in dst]
            assert torch.equal(state[bad], pool[bad])
    assert tern.device_error() == 0


def test_states_past_2_to_the_31(tern):
    """Slots whose offsets do not fit 32 bits."""
    Hk, Hv, Dk, Dv = 2, 32, 128, 128
    slots = [4200, 4150]
    state = torch.empty((4201, Hv, Dv, Dk), device="cuda")
    g = gen(14)
    for n in (1, 70, 600):
        inputs = delta_inputs(n, Hk, Hv, Dk, Dv, g)
        state[slots] = 0.1 * rand((2, Hv, Dv, Dk), g)
        before = f64(state[slots])
        out = tern.gated_delta(*inputs[:5], state, i32(slots[:1]), dst_slots=i32(slots[1:]), qk_norm=True)
        check_delta(inputs, Dk ** -0.5, True, before, state[slots], out, [0], [0, n], dst=[1])
    assert tern.device_error() == 0


def test_one_head_alone(tern):
    """NaN in one sequence's values, state and gates: the other sequences and heads stay as they were."""
    heads = (1, 2, 64, 32)
    for n in (1, 45, 600):
        g = gen(15)
        inputs = [t if t is None else t.clone() for t in delta_inputs(3 * n, *heads, g)]
        pool = rand((3, 2, 32, 64), g)
        clean, state = pool.clone(), pool.clone()
        want = tern.gated_delta(*inputs[:5], clean, i32([0, 1, 2]), qk_norm=True)
        inputs[2][n:2 * n, 1, 5] = float("nan")
        inputs[4][n, 1] = float("inf")
        state[1, 1, 3] = float("nan")
        got = tern.gated_delta(*inputs[:5], state, i32([0, 1, 2]), qk_norm=True)
        keep = [i for i in range(3 * n) if not n <= i < 2 * n]
        assert torch.equal(got[keep], want[keep]) and torch.equal(got[:, 0], want[:, 0])
        assert torch.equal(state[[0, 2]], clean[[0, 2]]) and torch.equal(state[:, 0], clean[:, 0])
        assert torch.isnan(got[2 * n - 1, 1]).any()


@pytest.mark.parametrize("heads", [(1, 2, 64, 48), (2, 2, 128, 144)])
@pytest.mark.parametrize("n", [20, 64, 100, 640])
@pytest.mark.parametrize("what", ["q", "k", "v", "g", "beta", "v inf", "k inf", "beta inf"])
def test_not_finite_goes_forward_only(tern, heads, n, what):
    """One value that is not finite: the rows and heads that it does not concern are bit for bit as with a finite
    one, and so is what comes before it but for roundings (its rows of S go token by token then: two results of
    half a step, 2^-8, and of at most 2^-15 of scale memory R each); the rest is not finite where it is not in the
    definition."""
    Hk, Hv, Dk, Dv = heads
    g = gen(n + Dv)
    clean = [t.clone() for t in delta_inputs(n, *heads, g)[:5]]
    pool = rand((1, Hv, Dv, Dk), g)
    need = tern.lib().tern_gated_delta_workspace_bytes(1, n, n, Hv, Dk, Dv)
    assert (need > 0) == (n == 640)
    bad = float("inf" if "inf" in what else "nan")
    _, _, reach, memory = ref.gated_delta(*(f64(t) for t in clean), f64(pool), [0], [0, n], Dk ** -0.5, True)
    for ws in {0, need}:
        state = pool.clone()
        assert delta_call(tern, (*clean, None, None), Dk ** -0.5, state, [0], [0, n], n, ws)[0] == 0
        state, fine = pool.clone(), state
        want = delta_call(tern, (*clean, None, None), Dk ** -0.5, state, [0], [0, n], n, ws)[1]
        assert torch.equal(state, fine)
        for at in sorted({0, 3, 14, 17 % n, 35 % n, 47 % n, 63 % n, n // 2 + 7, n - 1}):
            inputs = [t.clone() for t in clean]
            i = {"q": 0, "k": 1, "v": 2, "g": 3, "beta": 4}[what.split()[0]]
            inputs[i][(at, 0, 5)[:inputs[i].dim()]] = bad
            state = pool.clone()
            status, out = delta_call(tern, (*inputs, None, None), Dk ** -0.5, state, [0], [0, n], n, ws)
            assert status == 0 and tern.device_error() == 0
            hit = torch.zeros((n, Hv, Dv), dtype=torch.bool, device="cuda")       # what it concerns
            if what.startswith("v"):
                hit[at:, 0, 5] = True
            elif what == "q":
                hit[at, :Hv // Hk] = True
            else:
                hit[at:, :Hv // Hk if what.startswith("k") else 1] = True
            assert torch.equal(torch.isfinite(out), ~hit), (at, torch.nonzero(torch.isfinite(out) == hit)[:4])
            before = hit.any(0, keepdim=True).expand_as(hit) & ~hit if what != "q" else torch.zeros_like(hit)
            assert torch.equal(out[~hit & ~before], want[~hit & ~before]), at
            near = 2.0 ** -7 * np.abs(f64(want)) + (Dk ** -0.5 * 2.0 ** -14 * memory * reach)[None, :, None]
            within(out[before], f64(want)[f64(before) > 0], near[f64(before) > 0], f"before {at}")
            rows = hit[-1] if what != "q" else torch.zeros_like(hit[0])
            assert torch.equal(state[0][~rows], fine[0][~rows]), at
            assert not torch.isfinite(state[0][rows]).any(), at


@pytest.mark.parametrize("lens", [[0, 40, 70], [0, 40, 900, 3], [0, 40, 130] + [70] * 40])
def test_states_that_are_not_finite(tern, lens):
    """A value of a state that is not finite takes its row with it, in its own sequence; a state that only moves
    keeps it where it is; a value among the tokens of a sequence that is not stored, of one among many."""
    Hk, Hv, Dk, Dv = 2, 8, 64, 48
    B, g = len(lens), gen(31)
    start, T = sequences(lens)
    inputs = delta_inputs(T, Hk, Hv, Dk, Dv, g)
    pool = rand((2 * B, Hv, Dv, Dk), g)
    sl, dst = list(range(B)), [B + b if b != 2 else -1 for b in range(B)]

    def run(inputs, pool):
        state = pool.clone()
        out = tern.gated_delta(*inputs[:5], state, i32(sl), q_start=i32(start), max_new=max(lens), qk_norm=True, dst_slots=i32(dst))
        assert tern.device_error() == 0
        return out, state

    want, fine = run(inputs, pool)
    pool[0, 1, 7, 3] = float("inf")
    pool[1, 2, 9, 5] = float("nan")
    v = inputs[2].clone()
    v[start[2] + 33, 0, 4] = float("nan")
    out, state = run((inputs[0], inputs[1], v, *inputs[3:]), pool)
    same = lambda a, b: torch.equal(a.view(torch.int32), b.view(torch.int32))    # noqa: E731
    assert same(state[:B], pool[:B]) and same(state[dst[0]], pool[0])
    hit = torch.zeros((T, Hv, Dv), dtype=torch.bool, device="cuda")
    hit[start[1]:start[2], 2, 9] = True
    hit[start[2] + 33:start[3], 0, 4] = True
    assert torch.equal(torch.isfinite(out), ~hit)
    before = torch.zeros_like(hit)
    before[start[2]:start[2] + 33, 0, 4] = True
    assert torch.equal(out[~hit & ~before], want[~hit & ~before])
    # (two results of half a step each, and of 2^-13 of what goes into them)
    a, b = f64(out[before]), f64(want[before])
    assert np.abs(a - b).max() <= 2.0 ** -7 * np.abs(b).max() + 2.0 ** -12 * np.abs(f64(want)).max()
    row = torch.zeros((Hv, Dv), dtype=torch.bool, device="cuda")
    row[2, 9] = True
    assert not torch.isfinite(state[dst[1]][row]).any() and torch.equal(state[dst[1]][~row], fine[dst[1]][~row])
    assert torch.equal(state[B + 3:], fine[B + 3:])


def test_another_stream_and_replays(tern):
    """The three calls captured once and replayed on new inputs, on a stream of their own."""
    g = gen(16)
    B, Hk, Hv, D = 3, 1, 2, 64
    C = (2 * Hk + Hv) * D
    side = torch.cuda.Stream()
    for n in (1, 21, 75, 600):
        T = B * n
        x, w = rand((T, C), g, torch.bfloat16), rand((C, 4), g)
        gates, nw = rand((T, 2, Hv), g), 1 + 0.1 * rand(D, g)
        conv, delta, slots = rand((B, 3, C), g), rand((B, Hv, D, D), g), i32([2, 0, 1])
        al, dt = torch.zeros(Hv, device="cuda"), torch.zeros(Hv, device="cuda") - 2

        def layer(stream=None):
            y = tern.short_conv(x, w, conv, slots, stream=stream)
            q, k, v = y[:, :D].view(T, 1, D), y[:, D:2 * D].view(T, 1, D), y[:, 2 * D:].view(T, Hv, D)
            o = tern.gated_delta(q, k, v, gates[:, 0], gates[:, 1], delta, slots, qk_norm=True, a_log=al, dt_bias=dt,
                                 stream=stream)
            return tern.rms_norm(o, nw, gate=x.view(T, -1, D)[:, :Hv], stream=stream)

        keep = [t.clone() for t in (conv, delta)]
        first = layer().clone()
        second_x = rand((T, C), g, torch.bfloat16)
        then = [t.clone() for t in (conv, delta)]
        old_x = x.clone()
        x.copy_(second_x)
        second = layer().clone()
        last = [t.clone() for t in (conv, delta)]

        def reset(a, b):
            for t, s in zip((conv, delta), a):
                t.copy_(s)
            x.copy_(b)

        reset(keep, old_x)
        torch.cuda.synchronize()
        got = layer(side)
        side.synchronize()
        assert torch.equal(got, first)
        reset(keep, old_x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer()
        graph.replay()
        assert torch.equal(out, first) and torch.equal(conv, then[0]) and torch.equal(delta, then[1])
        x.copy_(second_x)
        graph.replay()
        assert torch.equal(out, second) and torch.equal(conv, last[0]) and torch.equal(delta, last[1])
    assert tern.device_error() == 0


def test_streams_at_once(tern):
    """Sequences in pieces on two streams and products on a third, all at once: each as if alone."""
    g = gen(23)
    heads, n = (2, 8, 64, 64), 640
    C = 2 * 2 * 64 + 8 * 64
    inputs = [delta_inputs(n, *heads, g) for _ in range(2)]
    pools = [rand((1, 8, 64, 64), g) for _ in range(2)]
    t = torch.randint(-1, 2, (1024, C - C % 128), dtype=torch.int8, device="cuda", generator=g)
    codes, scales = tern.pack(t), torch.full((1024, t.shape[1] // 128), 0.01, dtype=torch.half, device="cuda")
    x = rand((512, t.shape[1]), g, torch.bfloat16)

    def run(i, state, stream=None):
        return tern.gated_delta(*inputs[i][:5], state, i32([0]), qk_norm=True, stream=stream)

    alone = [pools[i].clone() for i in range(2)]
    want = [[run(i, alone[i]) for _ in range(4)] for i in range(2)]
    product = tern.gemm(x, codes, scales)
    streams = [torch.cuda.Stream() for _ in range(3)]
    state = [p.clone() for p in pools]
    torch.cuda.synchronize()
    got, products = [[], []], []
    for _ in range(4):
        for i in range(2):
            got[i].append(run(i, state[i], streams[i]))
        products.append(tern.gemm(x, codes, scales, stream=streams[2]))
    torch.cuda.synchronize()
    assert tern.device_error() == 0
    for i in range(2):
        assert torch.equal(state[i], alone[i]) and all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    assert all(torch.allclose(p, product, rtol=1e-4, atol=1e-4) for p in products)


@pytest.mark.parametrize("heads,lens", [((5, 15, 64, 96), [700, 65, 640]), ((1, 40, 64, 64), [577]), ((4, 24, 128, 128), [1089])])
@pytest.mark.parametrize("whole", [False, True])
def test_delta_repeats_bit_for_bit(tern, heads, lens, whole):
    """Every run of a call gives the same bits (what products read may not be written before they have: when X took
    S's place beside Q S^T, one run in forty of the first case differed)."""
    Hk, Hv, Dk, Dv = heads
    g = gen(21)
    start, T = sequences(lens)
    inputs, sl = delta_inputs(T, Hk, Hv, Dk, Dv, g), list(range(len(lens)))
    pool = rand((len(lens), Hv, Dv, Dk), g)
    ws = 0 if whole else tern.lib().tern_gated_delta_workspace_bytes(len(lens), T, max(lens), Hv, Dk, Dv)
    first = None
    for _ in range(150):
        state = pool.clone()
        status, out = delta_call(tern, inputs, Dk ** -0.5, state, sl, start, max(lens), ws)
        assert status == 0
        first = first or (out, state)
        assert torch.equal(out, first[0]) and torch.equal(state, first[1])


@pytest.mark.parametrize("lens", [[70] * 33 + [1, 0, 200] + [65] * 30, [64, 320, 0, 130, 64, 500, 30]])
def test_more_sequences_than_sms(tern, lens):
    """Sequences by length, past 32 of them, equal and unequal, with a bad range among them."""
    Hk, Hv, Dk, Dv = 2, 24, 64, 16
    g = gen(25)
    start, T = sequences(lens, behind=3)
    inputs = delta_inputs(T, Hk, Hv, Dk, Dv, g)
    B = len(lens)
    state = rand((B, Hv, Dv, Dk), g)
    before, sl = f64(state), list(range(B))[::-1]
    out = torch.full((T, Hv, Dv), 7.0, dtype=torch.bfloat16, device="cuda")
    tern.gated_delta(*inputs[:5], state, i32(sl), q_start=i32(start), max_new=max(lens), qk_norm=True, out=out)
    assert tern.device_error() == 0
    check_delta(inputs, Dk ** -0.5, True, before, state, out, sl, start, out_was=np.full(out.shape, 7.0))
    good, kept = out.clone(), state.clone()
    state.copy_(torch.from_numpy(before))
    start[2] = -5                              # its own range and the one before it
    tern.gated_delta(*inputs[:5], state, i32(sl), q_start=i32(start), max_new=max(lens), qk_norm=True, out=out)
    assert tern.device_error() == tern.DEVERR_CACHE_SEQUENCE
    last = start[4]
    assert torch.equal(out[last:], good[last:]) and torch.equal(state[:B - 4], kept[:B - 4])


def test_short_sequences_of_a_long_call(tern):
    """max_new as large as all tokens together: sequences too short for pieces stay whole, beside one that is not."""
    Hk, Hv, Dk, Dv = 1, 2, 64, 64
    g = gen(24)
    lens = [300, 1, 448, 449, 0, 700, 65]
    start, T = sequences(lens)
    inputs = delta_inputs(T, Hk, Hv, Dk, Dv, g)
    state = rand((8, Hv, Dv, Dk), g)
    before, sl = f64(state), [6, 5, 4, 3, 2, 1, 0]
    out = tern.gated_delta(*inputs[:5], state, i32(sl), q_start=i32(start), qk_norm=True)
    assert tern.device_error() == 0
    check_delta(inputs, Dk ** -0.5, True, before, state, out, sl, start)
    with pytest.raises(tern.TernError):
        tern.gated_delta(*inputs[:5], state, i32([]), qk_norm=True)


def run_out(tern, which, code):
    """Milliseconds of a self-test with a limit of 2 ms, whose code is read once."""
    assert tern.device_error() == 0
    tern.wait_selftest(which, 1000)
    assert tern.device_error() == code
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    tern.wait_selftest(which, 2000)
    end.record()
    assert tern.device_error() == code and tern.device_error() == 0
    return begin.elapsed_time(end)


def test_waits_that_run_out(tern):
    """A wait that nothing ends: every role goes on to the kernel's end, the error is read, calls after it work."""
    # four times the limit (a try may end a little before or after its 2 us), far from a second
    assert 1.0 < run_out(tern, tern.SELFTEST_DELTA, tern.DEVERR_DELTA_WAIT) < 100.0
    inputs = delta_inputs(70, 1, 2, 64, 32, gen(1))
    state = torch.zeros((1, 2, 32, 64), device="cuda")
    out = tern.gated_delta(*inputs[:5], state, i32([0]), qk_norm=True)
    assert tern.device_error() == 0
    check_delta(inputs, 64 ** -0.5, True, np.zeros((1, 2, 32, 64)), state, out, [0], [0, 70])


def test_a_row_that_never_comes(tern):
    """The ring's wait runs out, then the one for what is on its way: twice the limit; rows after it are right."""
    assert 1.0 < run_out(tern, tern.SELFTEST_NORM, tern.DEVERR_NORM_WAIT) < 100.0
    x, w = rand((700, 1032), gen(2)), torch.ones(1032, device="cuda")
    check_norm(tern, x, w, tern.rms_norm(x, w))
    assert tern.device_error() == 0
