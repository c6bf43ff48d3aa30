"""What the sampling and moving kernels keep outside their 64 registers (no GPU needed): around the passes over a
row, what the first block's decisions need; in the passes themselves little or nothing."""
import os
import re

import pytest

from quantized_moe_routed_gb300 import build as libbuild


@pytest.mark.parametrize("unit,most", [("moe_sample.cu", 512), ("moe_kv_move.cu", 32)])
def test_spills_stay_what_they_are(unit, most):
    libbuild.build()
    text = open(os.path.join(libbuild.BUILD, unit + ".log")).read()
    spills = [int(a) + int(b) for a, b in re.findall(r"(\d+) bytes spill stores, (\d+) bytes spill loads", text)]
    assert spills and max(spills) <= most, spills
