"""Arguments of the paged-cache calls that are refused before any device use.
Fake pointers: every call here is one that is refused."""
import ctypes

import pytest
import torch

P = 4096
SHAPE = 2


@pytest.fixture(scope="module")
def tern():
    from bit_gemv_gemm_gb300 import build
    build.build()
    import bit_gemv_gemm_gb300 as t
    return t


def layout(tern):
    return tern.CacheLayout(10, 16, 2, 128, 2 * 16 * 128, 16 * 128, 128)


@pytest.mark.parametrize("shift", [0, 4, 12, -12])
def test_evict_refuses_new_lengths_over_the_old(tern, shift):
    lay = layout(tern)
    at = ctypes.addressof(lay)
    assert tern.lib().tern_cache_evict(P, P, at, P, P, 100, P, 4, 100, 10, P, P, at, P, P, 7, P, P + shift, None) == SHAPE


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38, float("inf"), float("nan")])
def test_scales_without_a_finite_product_with_log2_e_are_refused(tern, scale):
    """The kernels keep scores in powers of two: a scale that is infinite there made NaN of every 0."""
    lay = layout(tern)
    at = ctypes.addressof(lay)
    assert tern.lib().tern_paged_attention(P, 1024, P, P, at, P, 4, P, P, 2, 2, 1, 8, scale, 0, P, P, P, 1 << 27,
                                           None) == SHAPE
    assert tern.lib().tern_attention_mass(P, 1024, P, at, P, 4, P, P, 2, 2, 1, 8, scale, 0, P, 1.0, P, P, None) == SHAPE


def test_strides_of_single_axes_say_nothing(tern):
    """A pool of one page, one head or both may come as a view with any stride there."""
    x = torch.zeros(4 * 16 * 64, dtype=torch.bfloat16)
    for shape, stride in (((4, 1, 16, 64), (1024, 0, 64, 1)), ((4, 1, 16, 64), (1024, 7, 64, 1)),
                          ((1, 4, 16, 64), (3, 1024, 64, 1)), ((1, 1, 64, 64), (0, 0, 64, 1))):
        v = x.as_strided(shape, stride)
        lay = tern._layout("k_cache", v.shape, v.stride())
        assert lay.page_stride >= 64 and lay.page_stride % 8 == 0 and lay.head_stride >= 64 and lay.head_stride % 8 == 0
        assert lay.slot_stride == 64
        dense = torch.zeros(shape, dtype=torch.bfloat16)
        tern._layout("v_cache", dense.shape, dense.stride(), (v.shape, v.stride()))
    with pytest.raises(ValueError, match="v_cache"):
        tern._layout("v_cache", (4, 2, 16, 64), (2048, 1024, 64, 1), ((4, 2, 16, 64), (2048, 64, 128, 1)))


def test_attention_workspaces_follow_the_need(tern):
    """One token takes less than a chunk, small heads less than large, and what a longer step needs is never less."""
    size = tern.paged_attention_workspace_bytes
    assert size(1, 1, 1, 32, 8, 128) < 8 << 20 < size(1, 512, 512, 32, 8, 128)
    for d in (64, 128, 256):
        steps = [size(2, 2 * n, n, 32, 8, d) for n in (0, 1, 4, 5, 32, 33, 4000)]
        assert steps == sorted(steps) and steps[-1] <= 1 << 27
        # max_new counts up to T, and is the average at least
        assert size(4, 4, 100, 32, 8, d) == size(4, 4, 4, 32, 8, d) and size(4, 80, 0, 32, 8, d) == size(4, 80, 20, 32, 8, d)
    assert size(1, 512, 512, 32, 8, 64) < size(1, 512, 512, 32, 8, 128) < size(1, 512, 512, 32, 8, 256)
