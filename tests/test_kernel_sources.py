"""Rules that the kernels' sources keep."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_w4a16_b200", "csrc")


def code(path):
    with open(path, encoding="utf-8") as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


WAITING = [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "pdl_wait_prior_grid" in code(p)]


def test_the_waiting_kernels_are_found():
    assert {os.path.basename(p) for p in WAITING} >= {"skinny.cu", "tile_gemm.cu", "quantize.cu", "verify.cu"}


@pytest.mark.parametrize("path", WAITING, ids=os.path.basename)
def test_no_read_only_loads_where_a_kernel_waits_for_the_previous_one(path):
    """A kernel that starts while the previous one still runs may not read its inputs through read-only
    loads: the data changes in its lifetime, and nothing keeps such a load behind the wait.  The compiler
    takes them for pointers marked __restrict__."""
    for word in ("__restrict__", "__ldg", "ld.global.nc"):
        assert word not in code(path), word
