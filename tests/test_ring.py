"""The way out of the layer kernels' rings of copies (moe_ring.h), run on the host
against a model of barriers and copies: after it, nothing is in flight, and no wait
was for a phase that never comes.  And where it stands in the kernels: after the
block's last barrier, before tensor memory is given back."""
import os
import re
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "quantized_moe_routed_gb300", "csrc")


@pytest.fixture(scope="module")
def sim(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("ring") / "ring_sim")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, "-o", exe,
                    os.path.join(ROOT, "tests", "native", "ring_sim.cpp")], check=True)
    return lambda mode, seeds: subprocess.run([exe, mode, str(seeds)], check=True, capture_output=True, text=True).stdout.strip()


@pytest.mark.parametrize("mode", ["one", "halves"])
def test_nothing_is_left_in_flight(sim, mode):
    assert sim(mode, 20000) == "ok"


@pytest.mark.parametrize("mode", ["skipped", "early"])
def test_the_model_notices(sim, mode):
    assert sim(mode, 20000).startswith("seed")


@pytest.mark.parametrize("name", ["moe_kv_attend.cu", "moe_kv_attend_tc.cu", "moe_linear_tc.cu"])
def test_the_kernels_drain_after_their_last_barrier(name):
    src = open(os.path.join(CSRC, name)).read()
    kernel = src[src.index("__global__"):]
    kernel = kernel[:kernel.index("\n}\n")]
    drain = kernel.index("ring_drain")
    before = kernel[:drain]
    # between the block's barrier and the drain: no wait that could give up, no product, no copy
    last = before.rindex("__syncthreads();")
    assert not re.search(r"\bwait(_or_abort)?\(|mma_|tma2d|bulk_g2s", before[last:]), before[last:]
    assert before.count("ring_drain") == 0
    if "tc_alloc" in kernel:
        end = kernel[drain:]
        assert end.index("tc_commit(&ct->drained") < end.index("__syncthreads();") < end.index("tc_dealloc")
