"""The layer operators' host side (moe_layer.cu) on the host, over a runtime that
only takes notes: calls on a cache of another device than the current one are refused
and queue nothing."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

from conftest import ROOT
from quantized_moe_routed_gb300 import binding, layer

A = 1 << 20  # stands for an aligned device pointer: never read


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    so = str(tmp_path_factory.mktemp("layer_host") / "liblayer_host.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", cuda,
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "quantized_moe_routed_gb300", "csrc"),
                    "-o", so, "-x", "c++", os.path.join(ROOT, "tests", "native", "layer_host.cpp")], check=True)
    lib = C.CDLL(so)
    for name, (res, args) in layer.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    lib.fake_queued.restype = lib.fake_message.restype = C.c_char_p
    return lib


@pytest.fixture
def cache(lib):
    lib.fake_device(1)
    out = C.c_void_p()
    d = layer.moe_kv_desc(4, 8, 2, 64, A, A, A, A, 0, 0, 0, None, 1)
    assert lib.moe_kv_create(C.byref(d), C.byref(out)) == binding.MOE_OK
    yield out
    lib.moe_kv_destroy(out)


CALLS = {
    "init": lambda lib, kv: lib.moe_kv_workspace_init(kv, A, 1 << 30, None),
    "append": lambda lib, kv: lib.moe_kv_append(kv, None, 0, A, 128, A, 128, None, C.byref(_batch()), A, None),
    "attend": lambda lib, kv: lib.moe_kv_attend(kv, A, 512, 1.0, A, C.byref(_batch()), A, None),
    "check": lambda lib, kv: lib.moe_kv_check(kv, A, None),
}


def _batch():
    return layer.moe_kv_batch(A, A, A, 1, 1, 1, 1)


@pytest.mark.parametrize("call", sorted(CALLS))
def test_a_cache_of_another_device_is_refused(lib, cache, call):
    lib.fake_clear()
    assert CALLS[call](lib, cache) == binding.MOE_OK
    assert lib.fake_queued() != b""
    lib.fake_clear()
    lib.fake_device(0)
    assert CALLS[call](lib, cache) == binding.MOE_ERR_INVALID_ARG
    assert lib.fake_queued() == b"" and b"device" in lib.fake_message()
