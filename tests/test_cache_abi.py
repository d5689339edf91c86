"""The paged-cache entry points without a GPU: argument errors come before any
device use, sizes and frequencies are host arithmetic, and the binding checks
shapes before pointers."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache as ref

P = 4096   # a fake aligned address; nothing dereferences it
NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def tern():
    from bit_gemv_gemm_gb300 import build
    build.build()
    import bit_gemv_gemm_gb300 as t
    return t


def layout(tern, **k):
    v = dict(pages=10, page_size=16, kv_heads=2, head_dim=128, page_stride=2 * 16 * 128, head_stride=16 * 128,
             slot_stride=128)
    v.update(k)
    return tern.CacheLayout(*[v[n] for n, _ in tern.CacheLayout._fields_])


def attention(tern, lay=None, **k):
    a = dict(q=P, q_stride=8 * 128, k=P, v=P, table=P, width=4, lens=P, q_start=P, B=2, T=2, max_new=1, q_heads=8,
             scale=0.1, window=0, out=P, lse=P, ws=P, n=1 << 27)
    a.update(k)
    lay = layout(tern) if lay is None else lay
    return tern.lib().tern_paged_attention(a["q"], a["q_stride"], a["k"], a["v"], ctypes.addressof(lay), a["table"],
                                           a["width"], a["lens"], a["q_start"], a["B"], a["T"], a["max_new"],
                                           a["q_heads"], a["scale"], a["window"], a["out"], a["lse"], a["ws"], a["n"],
                                           None)


@pytest.mark.parametrize("bad", [dict(pages=0), dict(page_size=8), dict(page_size=20), dict(kv_heads=0),
                                 dict(head_dim=100), dict(slot_stride=64), dict(slot_stride=132),
                                 dict(head_stride=1 << 40), dict(page_stride=-2048), dict(head_dim=96)])
def test_attention_refuses_layouts(tern, bad):
    assert attention(tern, layout(tern, **bad)) == SHAPE


@pytest.mark.parametrize("bad,code", [(dict(B=0), SHAPE), (dict(width=0), SHAPE), (dict(T=-1), SHAPE),
                                      (dict(width=1 << 27), SHAPE), (dict(q_stride=1 << 37), SHAPE),
                                      (dict(q_heads=7), SHAPE), (dict(q_heads=2 * 65, q_stride=1 << 20), SHAPE),
                                      (dict(q_stride=1000), SHAPE), (dict(q_stride=1028), SHAPE),
                                      (dict(window=-1), SHAPE), (dict(scale=float("nan")), SHAPE),
                                      (dict(q_start=None, T=3), SHAPE), (dict(q=None), NULL), (dict(k=None), NULL),
                                      (dict(v=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL),
                                      (dict(lens=None), NULL), (dict(q=P + 8), ALIGN), (dict(k=P + 2), ALIGN),
                                      (dict(out=P + 4), ALIGN), (dict(lens=P + 2), ALIGN), (dict(lse=P + 1), ALIGN),
                                      (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE), (dict(ws=P + 16), ALIGN)])
def test_attention_refuses_arguments(tern, bad, code):
    assert attention(tern, **bad) == code


def test_attention_workspace_never_passes_its_limit(tern):
    for B, T, n, hq, hk, d in [(1, 1, 1, 32, 8, 128), (1, 1 << 16, 1 << 16, 32, 8, 128), (4096, 4096, 1, 64, 1, 256),
                               (65535, 65535, 1, 64, 64, 64), (2, 10, 5, 4, 4, 256)]:
        assert 256 <= tern.paged_attention_workspace_bytes(B, T, n, hq, hk, d) <= 1 << 27
    for bad in [(0, 1, 1, 4, 4, 64), (1, 1, 1, 5, 4, 64), (1, 1, 1, 4, 4, 96), (1, -1, 1, 4, 4, 64)]:
        assert tern.paged_attention_workspace_bytes(*bad) == 0


def mass(tern, **k):
    a = dict(q=P, q_stride=8 * 128, k=P, table=P, width=4, lens=P, q_start=P, B=2, T=2, max_new=1, q_heads=8, scale=0.1,
             window=0, lse=P, decay=1.0, mass=P, out=P)
    a.update(k)
    lay = layout(tern)
    return tern.lib().tern_attention_mass(a["q"], a["q_stride"], a["k"], ctypes.addressof(lay), a["table"], a["width"],
                                          a["lens"], a["q_start"], a["B"], a["T"], a["max_new"], a["q_heads"],
                                          a["scale"], a["window"], a["lse"], a["decay"], a["mass"], a["out"], None)


@pytest.mark.parametrize("bad,code", [(dict(q_heads=9), SHAPE), (dict(decay=float("inf")), SHAPE),
                                      (dict(window=-2), SHAPE), (dict(lse=None), NULL), (dict(mass=None), NULL),
                                      (dict(out=None), NULL), (dict(mass=P + 2), ALIGN), (dict(q=P + 2), ALIGN)])
def test_mass_refuses_arguments(tern, bad, code):
    assert mass(tern, **bad) == code


def evict(tern, lay=None, dlay=None, **k):
    a = dict(k=P, v=P, mass=P, table=P, width=100, lens=P, B=2, budget=100, recent=10, dk=P, dv=P, dm=P, dt=P, dw=7,
             keep=P, dl=P)
    a.update(k)
    lay, dlay = lay or layout(tern), dlay or layout(tern)
    return tern.lib().tern_cache_evict(a["k"], a["v"], ctypes.addressof(lay), a["mass"], a["table"], a["width"],
                                       a["lens"], a["B"], a["budget"], a["recent"], a["dk"], a["dv"],
                                       ctypes.addressof(dlay), a["dm"], a["dt"], a["dw"], a["keep"], a["dl"], None)


@pytest.mark.parametrize("bad,code", [(dict(budget=0), SHAPE), (dict(recent=101), SHAPE), (dict(recent=-1), SHAPE),
                                      (dict(dw=6), SHAPE), (dict(B=0), SHAPE), (dict(width=1 << 28), SHAPE),
                                      (dict(keep=None), NULL), (dict(dm=None), NULL), (dict(dk=P + 8), ALIGN)])
def test_evict_refuses_arguments(tern, bad, code):
    assert evict(tern, **bad) == code


def test_evict_refuses_unlike_caches(tern):
    assert evict(tern, dlay=layout(tern, kv_heads=1)) == SHAPE
    assert evict(tern, dlay=layout(tern, head_dim=64)) == SHAPE


def rope(tern, **k):
    a = dict(q=P, k=P, v=P, f32=1, qs=1024, ks=256, vs=256, pos=P, slots=P, inv=P, factor=1.0, rot=128, inter=0, T=2,
             q_heads=8, out=P, kc=P, vc=P)
    a.update(k)
    lay = layout(tern)
    return tern.lib().tern_rope_append(a["q"], a["k"], a["v"], a["f32"], a["qs"], a["ks"], a["vs"], a["pos"],
                                       a["slots"], a["inv"], a["factor"], a["rot"], a["inter"], a["T"], a["q_heads"],
                                       a["out"], a["kc"], a["vc"], ctypes.addressof(lay), None)


@pytest.mark.parametrize("bad,code", [(dict(rot=3), SHAPE), (dict(rot=130), SHAPE), (dict(T=-1), SHAPE),
                                      (dict(qs=1020), SHAPE), (dict(q_heads=-1), SHAPE), (dict(q=None), NULL),
                                      (dict(inv=None), NULL), (dict(kc=None), NULL), (dict(slots=None), NULL),
                                      (dict(k=P + 8), ALIGN), (dict(slots=P + 4), ALIGN), (dict(out=P + 2), ALIGN)])
def test_rope_refuses_arguments(tern, bad, code):
    assert rope(tern, **bad) == code


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot,base,factor,original", [(128, 10000.0, 4.0, 4096), (64, 1e6, 8.0, 32768),
                                                      (4, 10000.0, 1.0, 128), (2, 500.0, 2.0, 64)])
def test_rope_frequencies(tern, scaling, rot, base, factor, original):
    if scaling == "ntk" and rot == 2:
        pytest.skip("the base's exponent has no value for one pair")
    f, a = tern.rope_frequencies(rot, base, scaling, factor, original)
    want, wa = ref.rope_frequencies(rot, base, scaling, factor, original)
    assert f.shape == (rot // 2,) and f.dtype == np.float32
    # both sides compute in 64 bits; the result is rounded once to 24
    assert (np.abs(f - want) <= 2.0 ** -23 * want).all() and abs(a - wa) <= 2.0 ** -23 * wa


def test_rope_frequency_refusals(tern):
    for bad in [dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=64, base=1.0),
                dict(rot_dim=64, scaling="linear", factor=0.5), dict(rot_dim=64, scaling="yarn", factor=2.0),
                dict(rot_dim=64, scaling="yarn", factor=2.0, original_len=100, turns_fast=1.0, turns_slow=2.0)]:
        with pytest.raises(tern.TernError):
            tern.rope_frequencies(**bad)
    with pytest.raises(ValueError, match="scaling"):
        tern.rope_frequencies(64, scaling="other")


def test_binding_checks_shapes_before_pointers(tern):
    """CPU tensors: the shape checks come before the device checks."""
    kc = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16)
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16)
    t, n = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_cache"):
        tern.paged_attention(q, kc[0], kc[0], t, n)
    with pytest.raises(ValueError, match="k_cache"):
        tern.paged_attention(q, kc.transpose(2, 3), kc.transpose(2, 3), t, n)
    with pytest.raises(TypeError, match="k_cache"):
        tern.paged_attention(q, kc, kc, t, n)
    with pytest.raises(TypeError, match="k_cache"):
        tern.cache_evict(kc, kc, t, t, n, 4, 1, kc, kc, t, t)


def test_oracle_rope_turns_by_the_angle():
    """The oracle itself: a quarter turn, and norms that the rotation keeps."""
    x = np.zeros((1, 1, 4))
    x[0, 0] = [1, 2, 3, 4]
    y = ref.rope(x, [1], [np.pi / 2, 0.0], 1.0, True)[0, 0]
    assert np.allclose(y, [-2, 1, 3, 4])
    y = ref.rope(x, [1], [np.pi / 2, 0.0], 1.0, False)[0, 0]
    assert np.allclose(y, [-3, 2, 1, 4])
    r = np.random.default_rng(0).standard_normal((5, 2, 16))
    y = ref.rope(r, np.arange(5), ref.rope_frequencies(12, 100.0)[0], 2.0, False)
    assert np.allclose((y[..., :12] ** 2).sum(-1), 4 * (r[..., :12] ** 2).sum(-1)) and np.array_equal(y[..., 12:], r[..., 12:])


def test_oracle_attention_and_evict_on_small_cases():
    """One key: the output is its value.  Two equal keys: their mean.  A mass
    sums to the number of rows.  Ties go to the lowest index."""
    k = np.zeros((2, 1, 16, 4))
    v = np.random.default_rng(1).standard_normal(k.shape)
    q = np.random.default_rng(2).standard_normal((2, 1, 4))
    table = np.array([[1]])
    out, lse, _, _ = ref.attention(q, k, v, table, [2], [0, 2], 0.5)
    assert np.allclose(out[0, 0], v[1, 0, 0]) and np.allclose(out[1, 0], v[1, 0, :2].mean(0))
    assert np.allclose(lse[:, 0], [0, np.log(2)])
    m, added = ref.mass(q, k, table, [2], [0, 2], 0.5, 0, lse, 1.0, np.zeros((2, 1, 16)), np.zeros((2, 1, 16)))
    assert np.isclose(added.sum(), 2) and np.allclose(added[1, 0, :2], [1.5, 0.5])
    w = np.zeros((2, 1, 16))
    w[1, 0, :6] = [1, 0, 1, -0.0, 1, 9]
    assert ref.evict(w, table, [6], 4, 1) == [[[0, 2, 4, 5]]]
    assert ref.evict(w, table, [6], 5, 1) == [[[0, 1, 2, 4, 5]]]
