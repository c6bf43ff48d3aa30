"""Every status that include/moe_nvfp4.h declares has its name, in the library and in
the binding."""
import os
import re

from conftest import ROOT
from quantized_moe_routed_gb300 import binding
from quantized_moe_routed_gb300 import build as libbuild


def test_every_status_has_its_name():
    libbuild.build()
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_nvfp4.h")).read(), flags=re.S)
    declared = {int(v): n for n, v in re.findall(r"\b(MOE_OK|MOE_ERR_[A-Z_]+)\s*=\s*(\d+)", src)}
    assert len(declared) >= 12 and declared == binding.STATUS_NAMES
    lib = binding.load_library()
    for value, name in declared.items():
        assert lib.moe_status_string(value).decode() == name
    assert lib.moe_status_string(max(declared) + 1).decode() == "MOE_ERR_UNKNOWN"
