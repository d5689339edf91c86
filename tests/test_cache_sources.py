"""What the sources of the cache operators must not hold."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gemv_gemm_gb300", "csrc")


def test_no_load_is_multicast():
    """The library is loaded by programs that use several GPUs, whose tensors may lie on a peer: a
    cluster's CTAs each fetch what they read."""
    files = glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    assert files
    for f in files:
        # string literals put together as the compiler does
        text = re.sub(r'"\s*"', "", open(f).read())
        for ptx in re.findall(r"cp\.async\.bulk[^;]*", text):
            assert "multicast" not in ptx, os.path.basename(f)
