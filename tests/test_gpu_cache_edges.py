"""The paged-cache operators where their arguments are at their ends: windows
past every key, values that are not finite, streams of their own, groups that do
not fill a row tile.  Bounds as in test_gpu_cache.py, where they are derived."""
import pytest
import torch

from test_gpu_cache import Problem, check_attention, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tern():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_gemv_gemm_gb300 import build
    build.build()
    import bit_gemv_gemm_gb300 as t
    return t


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [4, 8])
def test_many_short_sequences_of_one_key_tile(tern, D, group):
    """Items of a single key tile, in which the second stream of the tiles kernel has no product."""
    lens = [1 + (37 * b) % 128 for b in range(700)]
    new = [min(L, 5 + (7 * b) % 11) for b, L in enumerate(lens)]
    p = Problem(2, lens, new, 2 * group, 2, D)
    a = run_attention(tern, p)
    check_attention(p, *a)
    for _ in range(20):
        b = run_attention(tern, p)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
