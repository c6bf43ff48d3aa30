"""The ABI of the operators for speculative decoding and sampling and their host-side
checks (no GPU needed): the binding prototypes what include/moe_speculate.h declares,
and arguments are refused before anything is queued."""
import ctypes as C
import os
import re

import pytest
import torch

from conftest import ROOT
from quantized_moe_routed_gb300 import MoeError, binding, layer, sample
from quantized_moe_routed_gb300 import build as libbuild

INVALID, MISALIGNED, SHAPE, OK = (binding.MOE_ERR_INVALID_ARG, binding.MOE_ERR_MISALIGNED, binding.MOE_ERR_UNSUPPORTED_SHAPE,
                                  binding.MOE_OK)
A = 1 << 20  # stands for an aligned device pointer: never read
M = 1 << 24  # apart from it


def _header():
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_speculate.h")).read(), flags=re.S)


def test_binding_prototypes_what_the_header_declares():
    libbuild.build()
    src = _header()
    declared = set(re.findall(r"\b(moe_[a-z_]+)\s*\(", src))
    assert declared == set(layer.SPECULATE_SIGNATURES), declared ^ set(layer.SPECULATE_SIGNATURES)
    lib = layer._library()
    for name in declared:
        args = re.search(r"\b" + name + r"\s*\(([^()]*)\)", src).group(1)
        assert len(args.split(",")) == len(layer.SPECULATE_SIGNATURES[name][1]), name
        assert hasattr(lib, name), name
    body = re.search(r"typedef struct \{([^{}]*)\}\s*moe_sample_desc;", src).group(1)
    names = re.findall(r"\*?\s*(\w+)\s*[,;]", body)
    assert names == [f for f, _ in layer.moe_sample_desc._fields_]
    for name, value in (("MOE_KV_MAX_TREE", layer.MAX_TREE), ("MOE_SAMPLE_MAX_VOCAB", layer.MAX_VOCAB)):
        assert re.search(r"#define\s+" + name + r"\s+" + str(value) + r"\b", src), name


@pytest.mark.parametrize("unit,regs", [("moe_sample.cu", 64), ("moe_kv_move.cu", 64)])
def test_kernels_fit_their_registers(unit, regs):
    # two blocks of 512 threads share an SM, four and more of 256
    libbuild.build()
    text = open(os.path.join(libbuild.BUILD, unit + ".log")).read()
    used = [int(r) for r in re.findall(r"Used (\d+) registers", text)]
    spills = [int(a) + int(b) for a, b in re.findall(r"(\d+) bytes spill stores, (\d+) bytes spill loads", text)]
    assert used and max(used) <= regs, used
    assert max(spills) <= 768, spills  # (around the passes: what the first block's decisions keep)


def _sample(logits=A, stride=100, bf16=0, T=2, V=100, u=A, t=None, k=None, p=None, mp=None, token=A, prob=None):
    d = layer.moe_sample_desc(logits, stride, bf16, T, V, u, t, 1.0, k, 0, p, 1.0, mp, 0.0, token, prob)
    return layer._library().moe_sample(C.byref(d), None)


@pytest.mark.parametrize("status,args", [
    (INVALID, dict(T=-1)), (INVALID, dict(T=(1 << 27) + 1)), (SHAPE, dict(V=0)), (SHAPE, dict(V=262145, stride=1 << 20)),
    (INVALID, dict(bf16=2)), (INVALID, dict(stride=99)), (INVALID, dict(logits=None)), (INVALID, dict(u=None)),
    (INVALID, dict(token=None)), (MISALIGNED, dict(logits=A + 2)), (MISALIGNED, dict(logits=A + 1, bf16=1)),
    (MISALIGNED, dict(u=A + 2)), (MISALIGNED, dict(t=A + 1)), (MISALIGNED, dict(k=A + 2)), (MISALIGNED, dict(p=A + 2)),
    (MISALIGNED, dict(mp=A + 2)), (MISALIGNED, dict(token=A + 2)), (MISALIGNED, dict(prob=A + 2))])
def test_sample_refuses(status, args):
    assert _sample(**args) == status
    assert binding.moe_last_error()


def test_empty_samples_need_no_pointers():
    assert _sample(T=0, logits=None, u=None, token=None) == OK
    assert layer._library().moe_sample(None, None) == INVALID


def test_null_handles_are_refused():
    lib = layer._library()
    batch = layer.moe_kv_batch(A, A, A, 1, 1, 1, 1)
    assert lib.moe_kv_append_tree(None, None, 0, A, 64, A, 64, None, C.byref(batch), A, A, None) == INVALID
    assert lib.moe_kv_attend_tree(None, A, 64, 1.0, A, C.byref(batch), A, A, None) == INVALID
    assert lib.moe_kv_compact(None, A, A, 1, M, C.byref(batch), A, None) == INVALID
    assert lib.moe_kv_fork(None, A, A, 1, A, A, 1, 1, M, M, A, None) == INVALID


def test_the_python_layer_refuses_host_tensors():
    x, u = torch.zeros((2, 64)), torch.zeros(2)
    for call in (lambda: sample(x, u), lambda: sample(x[0], u), lambda: sample(x.half(), u)):
        with pytest.raises(MoeError) as ei:
            call()
        assert ei.value.status == INVALID


# ----------------------------------------------------------------------------- over a runtime that only takes notes
@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    import shutil
    import subprocess
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    so = str(tmp_path_factory.mktemp("speculate_host") / "libspeculate_host.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", cuda,
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "quantized_moe_routed_gb300", "csrc"),
                    "-I", os.path.join(ROOT, "tests", "native"),
                    "-o", so, "-x", "c++", os.path.join(ROOT, "tests", "native", "speculate_host.cpp")], check=True)
    lib = C.CDLL(so)
    for name, (res, args) in {**layer.SIGNATURES, **layer.SPECULATE_SIGNATURES}.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    lib.fake_queued.restype = lib.fake_message.restype = C.c_char_p
    return lib


@pytest.fixture
def cache(lib):
    lib.fake_device(1)
    lib.fake_clear()
    out = C.c_void_p()
    d = layer.moe_kv_desc(4, 8, 2, 64, A, A, A, A, 0, 0, 0, None, 1)
    assert lib.moe_kv_create(C.byref(d), C.byref(out)) == OK
    yield out
    lib.moe_kv_destroy(out)


def _batch(q_off=A, kv_len=A, pages=A, max_pages=3, B=2, N=4, max_q=2):
    return C.byref(layer.moe_kv_batch(q_off, kv_len, pages, max_pages, B, N, max_q))


def _append(lib, kv, parent=A, batch=None, k=A):
    return lib.moe_kv_append_tree(kv, None, 0, k, 128, A, 128, None, batch or _batch(), parent, A, None)


def _attend(lib, kv, parent=A, batch=None, scale=1.0, o=A):
    return lib.moe_kv_attend_tree(kv, A, 512, scale, o, batch or _batch(), parent, A, None)


def _compact(lib, kv, keep=A, n_keep=A, K=4, out=M, batch=None, ws=A):
    return lib.moe_kv_compact(kv, keep, n_keep, K, out, batch or _batch(), ws, None)


def _fork(lib, kv, src=A, fresh=A, n=3, kv_len=A, pages=A, width=3, B=2, out=M, pages_out=2 * M, ws=A):
    return lib.moe_kv_fork(kv, src, fresh, n, kv_len, pages, width, B, out, pages_out, ws, None)


CALLS = {"append": (_append, b"launch_kv_append "), "attend": (_attend, b"launch_kv_attend_rows "),
         "compact": (_compact, b"launch_kv_compact "), "fork": (_fork, b"launch_kv_fork ")}


@pytest.mark.parametrize("call", sorted(CALLS))
def test_one_launch_on_the_caches_device_and_no_other(lib, cache, call):
    fn, launch = CALLS[call]
    assert fn(lib, cache) == OK
    assert lib.fake_queued() == b"claim " + launch
    lib.fake_clear()
    lib.fake_device(0)
    assert fn(lib, cache) == INVALID
    assert lib.fake_queued() == b"" and b"device" in lib.fake_message()


@pytest.mark.parametrize("status,fn,args", [
    (INVALID, _append, dict(parent=None)), (MISALIGNED, _append, dict(parent=A + 2)), (INVALID, _append, dict(k=None)),
    (SHAPE, _append, dict(batch=_batch(N=300, max_q=257))), (INVALID, _attend, dict(parent=None)),
    (MISALIGNED, _attend, dict(parent=A + 1)), (SHAPE, _attend, dict(batch=_batch(N=300, max_q=257))),
    (INVALID, _attend, dict(scale=float("inf"))), (INVALID, _attend, dict(o=None)),
    (INVALID, _compact, dict(keep=None)), (INVALID, _compact, dict(n_keep=None)), (INVALID, _compact, dict(out=None)),
    (INVALID, _compact, dict(K=-1)), (INVALID, _compact, dict(K=257)), (INVALID, _compact, dict(out=A)),
    (INVALID, _compact, dict(out=A + 4)), (MISALIGNED, _compact, dict(keep=A + 2)), (MISALIGNED, _compact, dict(out=M + 1)),
    (INVALID, _compact, dict(ws=None)), (INVALID, _compact, dict(batch=_batch(B=513))), (INVALID, _compact, dict(batch=_batch(N=-1))),
    (INVALID, _compact, dict(batch=_batch(pages=None))), (INVALID, _compact, dict(batch=_batch(max_pages=0))),
    (INVALID, _fork, dict(n=-1)), (INVALID, _fork, dict(n=513)), (INVALID, _fork, dict(B=0)), (INVALID, _fork, dict(B=-1)),
    (INVALID, _fork, dict(src=None)), (INVALID, _fork, dict(fresh=None)), (INVALID, _fork, dict(kv_len=None)),
    (INVALID, _fork, dict(pages=None)), (INVALID, _fork, dict(out=None)), (INVALID, _fork, dict(pages_out=None)),
    (INVALID, _fork, dict(pages_out=A + 8)), (INVALID, _fork, dict(out=2 * M + 8)), (INVALID, _fork, dict(width=0)),
    (MISALIGNED, _fork, dict(src=A + 2)), (MISALIGNED, _fork, dict(pages_out=2 * M + 2)), (INVALID, _fork, dict(ws=None))])
def test_refusals_queue_nothing(lib, cache, status, fn, args):
    assert fn(lib, cache, **args) == status
    assert lib.fake_queued() == b"" and lib.fake_message()


def test_empty_steps(lib, cache):
    empty = _batch(B=0, N=0, max_q=0, q_off=None, kv_len=None, pages=None)
    assert _append(lib, cache, batch=empty, parent=None, k=None) == OK
    assert _attend(lib, cache, batch=empty, parent=None) == OK
    assert _compact(lib, cache, batch=empty, keep=None, n_keep=None, out=None) == OK
    assert _fork(lib, cache, n=0, src=None, fresh=None, out=None, pages_out=None) == OK
    assert lib.fake_queued() == b""
    # sequences without new tokens keep their lengths: that is work
    assert _compact(lib, cache, batch=_batch(N=0, max_q=0), K=0, keep=None) == OK
    assert b"launch_kv_compact" in lib.fake_queued()
