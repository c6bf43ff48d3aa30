"""Kernels that follow one another by programmatic dependent launch and hold tensor
memory: each has its own, block-wide, before it lets the next kernel start, since
that one's blocks may allocate theirs before they wait for this one (were both to fit
on an SM, each would wait for the other)."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "quantized_moe_routed_gb300", "csrc")
UNITS = ["moe_kv_attend_tc.cu", "moe_linear_tc.cu", "moe_small.cu", "moe_tc.cu"]


def _source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_every_unit_that_allocates_is_looked_at():
    assert sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and "tc_alloc(" in _source(f)) == UNITS


@pytest.mark.parametrize("name", UNITS)
def test_tensor_memory_before_the_next_kernel(name):
    src = _source(name)
    at = src.index("tc_alloc(")
    assert src.count("tc_alloc(") == 1
    kernel = src[src.rindex("__global__", 0, at):]
    at = kernel.index("tc_alloc(")
    barrier = kernel.index("__syncthreads();", at)
    release = re.search(r"grid_release\(\)|griddepcontrol\.launch_dependents", kernel).start()
    assert at < barrier < release
