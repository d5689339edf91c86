"""The linear-attention layer's entry points without a GPU: argument errors come
before any device use, and the binding checks shapes before pointers.  Fake
pointers: every call of the library here is one that is refused."""
import pytest
import torch

P = 4096
NULL, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def tern():
    from bit_gemv_gemm_gb300 import build
    build.build()
    import bit_gemv_gemm_gb300 as t
    return t


def norm(tern, **k):
    a = dict(x=P, x_f32=0, xt=256, xh=0, r=P, r_f32=0, rt=256, rh=0, g=P, g_f32=0, gt=256, gh=0, act=0, w=P, off=0.0,
             scale=1.0, eps=1e-6, after=0, T=3, heads=1, dim=256, out=P, out_f32=0, ro=P, stream=None)
    assert set(k) <= set(a)
    return tern.lib().tern_rms_norm(*{**a, **k}.values())


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), SHAPE), (dict(heads=0), SHAPE), (dict(heads=65536), SHAPE), (dict(T=1 << 20, heads=1 << 11), SHAPE),
    (dict(dim=0), SHAPE), (dict(dim=100), SHAPE), (dict(dim=32776), SHAPE), (dict(xt=-8), SHAPE), (dict(xt=260), SHAPE),
    (dict(gh=4), SHAPE), (dict(rt=1 << 37), SHAPE), (dict(act=2), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(after=1), SHAPE), (dict(r=None), SHAPE), (dict(w=None), NULL),
    (dict(x=None), NULL), (dict(out=None), NULL), (dict(x=P + 8), ALIGN), (dict(r=P + 2), ALIGN), (dict(g=P + 4), ALIGN),
    (dict(w=P + 4), ALIGN), (dict(out=P + 8), ALIGN), (dict(ro=P + 8), ALIGN)])
def test_norm_refuses(tern, bad, code):
    assert norm(tern, **bad) == code


def conv(tern, **k):
    a = dict(x=P, f32=0, xt=64, w=P, width=4, bias=P, silu=1, state=P, pool=5, slots=P, dst=P, past=P, start=P, B=2, T=4,
             max_new=3, channels=64, out=P, stream=None)
    assert set(k) <= set(a)
    return tern.lib().tern_short_conv(*{**a, **k}.values())


@pytest.mark.parametrize("bad,code", [
    (dict(width=1), SHAPE), (dict(width=5), SHAPE), (dict(channels=60), SHAPE), (dict(channels=0), SHAPE),
    (dict(channels=(1 << 20) + 8, xt=1 << 21), SHAPE), (dict(xt=56), SHAPE), (dict(xt=68), SHAPE), (dict(xt=-64), SHAPE),
    (dict(B=0), SHAPE), (dict(B=65536), SHAPE), (dict(T=-1), SHAPE), (dict(max_new=-1), SHAPE), (dict(pool=0), SHAPE),
    (dict(start=None, T=5), SHAPE), (dict(T=1 << 21, max_new=1 << 21), SHAPE), (dict(slots=None), NULL),
    (dict(w=None), NULL), (dict(state=None), NULL), (dict(x=None), NULL), (dict(out=None), NULL), (dict(x=P + 8), ALIGN),
    (dict(w=P + 4), ALIGN), (dict(bias=P + 2), ALIGN), (dict(state=P + 4), ALIGN), (dict(out=P + 2), ALIGN),
    (dict(slots=P + 1), ALIGN), (dict(dst=P + 2), ALIGN), (dict(past=P + 2), ALIGN), (dict(start=P + 2), ALIGN)])
def test_conv_refuses(tern, bad, code):
    assert conv(tern, **bad) == code


def delta(tern, **k):
    a = dict(q=P, k=P, v=P, qt=256, kt=256, vt=512, g=P, gt=4, beta=P, bt=4, al=P, dt=P, scale=0.1, norm=1, state=P,
             pool=5, slots=P, dst=P, past=P, start=P, B=2, T=4, max_new=3, hk=2, hv=4, dk=128, dv=128, out=P, ws=None, ws_bytes=0,
             stream=None)
    assert set(k) <= set(a)
    return tern.lib().tern_gated_delta(*{**a, **k}.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dk=32), SHAPE), (dict(dk=96), SHAPE), (dict(dk=256), SHAPE), (dict(dv=8), SHAPE), (dict(dv=120), SHAPE),
    (dict(dv=272, vt=1 << 12), SHAPE), (dict(hk=0), SHAPE), (dict(hv=3), SHAPE), (dict(hv=0), SHAPE),
    (dict(hv=65536, hk=1), SHAPE), (dict(qt=248), SHAPE), (dict(kt=260), SHAPE), (dict(vt=504), SHAPE),
    (dict(gt=3), SHAPE), (dict(bt=3), SHAPE), (dict(gt=-4), SHAPE), (dict(vt=1 << 37), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(B=0), SHAPE), (dict(T=-1), SHAPE),
    (dict(pool=0), SHAPE), (dict(start=None, T=5), SHAPE), (dict(al=None), NULL), (dict(dt=None), NULL),
    (dict(state=None), NULL), (dict(q=None), NULL), (dict(v=None), NULL), (dict(g=None), NULL), (dict(out=None), NULL),
    (dict(slots=None), NULL), (dict(q=P + 8), ALIGN), (dict(k=P + 2), ALIGN), (dict(v=P + 8), ALIGN),
    (dict(state=P + 8), ALIGN), (dict(out=P + 2), ALIGN), (dict(g=P + 2), ALIGN), (dict(al=P + 1), ALIGN),
    (dict(start=P + 1), ALIGN), (dict(ws=P + 128, ws_bytes=1 << 20), ALIGN)])
def test_delta_refuses(tern, bad, code):
    assert delta(tern, **bad) == code


@pytest.mark.parametrize("bad", [(0, 4096, 4096, 8, 128, 128), (1, -1, 4096, 8, 128, 128), (1, 4096, -1, 8, 128, 128),
                                 (1, 4096, 4096, 0, 128, 128), (1, 4096, 4096, 8, 96, 128), (1, 4096, 4096, 8, 128, 272),
                                 (1, 4096, 4096, 8, 128, 24), (1, 4096, 24, 8, 128, 128), (1, 64, 4096, 8, 128, 128)])
def test_delta_workspace_of_nothing(tern, bad):
    assert tern.lib().tern_gated_delta_workspace_bytes(*bad) == 0


# --- the binding (CPU tensors: shapes first, then the device) ---

def test_norm_binding(tern):
    x, w = torch.zeros(3, 4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="gate_act"):
        tern.rms_norm(x, w, gate_act="relu")
    with pytest.raises(ValueError, match="x must be"):
        tern.rms_norm(x.transpose(1, 2), w)
    with pytest.raises(TypeError, match="x must be"):
        tern.rms_norm(x, w)
    with pytest.raises(ValueError, match="residual must have x's shape"):
        tern._row_strides("residual", (3, 64), (64, 1), (3, 4, 64))
    assert tern._row_strides("x", (3, 4, 64), (512, 64, 1)) == (512, 64)
    assert tern._row_strides("x", (1, 64), (7, 1)) == (64, 0)


def test_conv_binding(tern):
    x, slots = torch.zeros(3, 64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="x must be"):
        tern.short_conv(x.t(), torch.zeros(3, 4), torch.zeros(2, 3, 3), slots)
    with pytest.raises(ValueError, match="weight"):
        tern.short_conv(x, torch.zeros(32, 4), torch.zeros(2, 3, 64), slots)
    with pytest.raises(ValueError, match="state"):
        tern.short_conv(x, torch.zeros(64, 4), torch.zeros(2, 4, 64), slots)
    with pytest.raises(TypeError, match="x must be"):
        tern.short_conv(x, torch.zeros(64, 4), torch.zeros(2, 3, 64), slots)


def test_delta_binding(tern):
    bf = torch.bfloat16
    q, k, v = torch.zeros(3, 2, 64, dtype=bf), torch.zeros(3, 2, 64, dtype=bf), torch.zeros(3, 4, 32, dtype=bf)
    g, slots = torch.zeros(3, 4), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="state"):
        tern.gated_delta(q, k, v, g, g, torch.zeros(2, 4, 32), slots)
    with pytest.raises(ValueError, match="q must hold"):
        tern.gated_delta(q, k, v, g, g, torch.zeros(2, 4, 32, 128), slots)
    with pytest.raises(TypeError, match="q must be"):
        tern.gated_delta(q, k, v, g, g, torch.zeros(2, 4, 32, 64), slots)
    with pytest.raises(ValueError, match="g must be"):
        tern._gate_stride("g", (3, 5), (5, 1), 3, 4)
    with pytest.raises(ValueError, match="beta must be"):
        tern._gate_stride("beta", (3, 4), (1, 3), 3, 4)
    assert tern._gate_stride("g", (3, 4), (16, 1), 3, 4) == 16 and tern._gate_stride("g", (1, 4), (0, 1), 1, 4) == 4


def test_binding_takes_no_other_shapes(tern):
    """A tensor of another shape with elements enough would give numbers, not an error."""
    bf, i32 = torch.bfloat16, torch.int32
    x, w = torch.zeros(3, 4, 64), torch.ones(64)
    for name, kw in (("weight", dict(weight=torch.ones(4, 64))), ("weight", dict(weight=torch.ones(65))),
                     ("weight", dict(weight=torch.ones(63))), ("out", dict(out=torch.zeros(4, 4, 64))),
                     ("out", dict(out=torch.zeros(3, 64, 4))), ("out", dict(out=torch.zeros(12, 64))),
                     ("residual_out", dict(residual=x, residual_out=torch.zeros(64, 4, 3))),
                     ("residual_out", dict(residual=x, residual_out=torch.zeros(4, 4, 64)))):
        with pytest.raises(ValueError, match=f"^{name} must be"):
            tern.rms_norm(**{**dict(x=x, weight=w), **kw})
    for kw in (dict(out=torch.zeros(3, 4, 64)), dict(out=torch.zeros(3, 256)),
               dict(residual=x, residual_out=torch.zeros(3, 256))):   # (these get as far as the device)
        with pytest.raises(TypeError, match="x must be"):
            tern.rms_norm(x, w, **kw)
    x, slots = torch.zeros(3, 64), torch.zeros(1, dtype=i32)
    for name, kw in (("bias", dict(bias=torch.zeros(65))), ("bias", dict(bias=torch.zeros(64, 1))),
                     ("out", dict(out=torch.zeros(4, 64))), ("out", dict(out=torch.zeros(64, 3)))):
        with pytest.raises(ValueError, match=f"^{name} must be"):
            tern.short_conv(x, torch.zeros(64, 4), torch.zeros(2, 3, 64), slots, **kw)
    q, v, g = torch.zeros(3, 2, 64, dtype=bf), torch.zeros(3, 4, 32, dtype=bf), torch.zeros(3, 4)
    h = torch.zeros(4)
    for name, kw in (("a_log", dict(a_log=torch.zeros(5), dt_bias=h)), ("dt_bias", dict(a_log=h, dt_bias=torch.zeros(1, 4))),
                     ("out", dict(out=torch.zeros(4, 4, 32))), ("out", dict(out=torch.zeros(3, 32, 4)))):
        with pytest.raises(ValueError, match=f"^{name} must be"):
            tern.gated_delta(q, q, v, g, g, torch.zeros(2, 4, 32, 64), slots, **kw)
    two = torch.zeros(2, dtype=i32)
    for name, (sl, dst, past, start) in (("slots", (torch.zeros(2, 1, dtype=i32), None, None, None)), ("dst_slots", (slots, two, None, None)),
                                         ("past", (slots, None, two, None)), ("q_start", (slots, None, None, slots)),
                                         ("q_start", (two, None, None, torch.zeros(4, dtype=i32)))):
        with pytest.raises(ValueError, match=f"^{name} must be"):
            tern._states(4, sl, dst, past, start, None, -2)


def test_wait_selftest_refuses(tern):
    for which, limit in ((2, 1000), (5, 1000), (tern.SELFTEST_DELTA, 0), (tern.SELFTEST_DELTA, 1000001),
                         (tern.SELFTEST_NORM, 0), (tern.SELFTEST_NORM, 1000001)):
        assert tern.lib().tern_wait_selftest(which, limit, None) == SHAPE
