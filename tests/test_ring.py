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


def _kernel(name):
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    kernel = src[src.index("__global__"):]
    return kernel[:kernel.index("\n}\n")]


_GOES_ON = r"\bwait(_or_abort)?\(|mma_|tma2d|bulk_g2s"  # a wait that could give up, a product, a copy


@pytest.mark.parametrize("name", ["moe_kv_attend.cu", "moe_linear_tc.cu"])
def test_the_kernels_drain_after_their_last_barrier(name):
    kernel = _kernel(name)
    drain = kernel.index("ring_drain")
    before = kernel[:drain]
    last = before.rindex("__syncthreads();")
    assert not re.search(_GOES_ON, before[last:]), before[last:]
    assert before.count("ring_drain") == 0
    if "tc_alloc" in kernel:
        end = kernel[drain:]
        assert end.index("tc_commit(&ct->drained") < end.index("__syncthreads();") < end.index("tc_dealloc")


def test_the_many_rows_attention_drains_where_all_warps_have_met():
    """Here every kind of warp comes to the barrier at its own end (code behind their
    common one costs the loops 4% of their time): each once, with nothing after it that
    could give up or start anything, and the drains only behind it."""
    kernel = _kernel("moe_kv_attend_tc.cu")
    meet = kernel[kernel.index("auto meet = [&] {"):]
    meet = meet[:meet.index("};")]
    assert '"bar.sync 2, %0;" ::"n"(kThreads)' in meet and "return aborted();" in meet
    rest = kernel[kernel.index("auto landed"):]
    rest = rest[rest.index("};"):]
    at = [m.start() for m in re.finditer(r"\bmeet\(\)", rest)]
    assert len(at) == 4  # converters, producers, issuers, softmax
    for a in at:
        # up to the end of the warp's branch
        tail = re.split(r"\n        \} else|\n    \} else|\n    \}\n", rest[a:])[0]
        assert not re.search(_GOES_ON, tail), tail
    for what in ("ring_drain(", "tc_commit(&ct->drained"):
        assert rest.count(what) == 1
        guard = rest[:rest.index(what)]
        assert re.search(r"if \(meet\(\) && (lane == 0|elect_one\(\))\) \{[^}]*$", guard), guard[-200:]
    assert rest.index("__syncthreads();") > max(at) and rest.rindex("tc_dealloc") > rest.rindex("__syncthreads();")
