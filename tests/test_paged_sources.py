"""What the sources of the paged cache's kernels may not hold.  No GPU needed."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_graph_causal_b200", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


CHAINED = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and "launch_chained(" in _code(f))


def test_there_are_chained_kernels():
    assert {"paged_append.cu", "paged_decode.cu", "paged_plan.cu"} <= set(CHAINED)


@pytest.mark.parametrize("name", CHAINED)
def test_chained_kernels_load_coherently(name):
    """These kernels are on the GPU while the one before them still writes what they will read:
    no load that takes memory for read-only as long as the kernel lives (__ldg, .nc, what the
    compiler makes of const __restrict__, and the row slices, which use __ldg)."""
    assert re.findall(r"__ldg\b|\.nc\b|__restrict__|\bSlice<", _code(name)) == []
