"""Frequencies of a context stretched by parts, against the published formula
written out here, where the slow end of the ramp lies past the last pair too."""
import math

import numpy as np
import pytest

from oracle import cache as ref


@pytest.fixture(scope="module")
def tern():
    from bit_gemv_gemm_gb300 import build
    build.build()
    import bit_gemv_gemm_gb300 as t
    return t


def by_parts(r, base, factor, original, fast, slow):
    """Pair i turns original * base^(-2 i / r) / (2 pi) times in the original length.  The correction
    range is [floor, ceil] of the indices of `fast` and `slow` turns, kept inside [0, r - 1]."""
    def index(turns):
        return r * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), r - 1)
    out = []
    for i in range(r // 2):
        f = base ** (-2 * i / r)
        stretched = min(max((i - lo) / (hi - lo if hi != lo else 0.001), 0), 1)
        out.append(f / factor * stretched + f * (1 - stretched))
    return np.array(out)


@pytest.mark.parametrize("r,base,factor,original", [(128, 1e4, 4.0, 4096), (128, 1e4, 4.0, 65536), (128, 1e4, 4.0, 131072),
                                                    (64, 1e4, 8.0, 131072), (64, 1e4, 8.0, 1 << 30), (128, 1e6, 8.0, 32768),
                                                    (16, 500.0, 2.0, 100000)])
@pytest.mark.parametrize("fast,slow", [(32.0, 1.0), (64.0, 4.0)])
def test_frequencies_by_parts(tern, r, base, factor, original, fast, slow):
    want = by_parts(r, base, factor, original, fast, slow)
    got, a = tern.rope_frequencies(r, base, "yarn", factor, original, fast, slow)
    # 64 bits, rounded once to 24
    assert (np.abs(got - want) <= 2.0 ** -23 * want).all() and abs(a - (0.1 * math.log(factor) + 1)) < 1e-6
    oracle, _ = ref.rope_frequencies(r, base, "yarn", factor, original, fast, slow)
    assert (np.abs(oracle - want) <= 2.0 ** -40 * want).all()


def test_a_pair_of_many_turns_is_not_divided(tern):
    """Every pair turns more than once in the original length: none is stretched in full."""
    f, _ = tern.rope_frequencies(128, 1e4, "yarn", 4.0, 131072)
    plain, _ = tern.rope_frequencies(128, 1e4)
    assert (f > 1.01 * plain / 4).all()
