"""The layer operators' ABI and host-side checks (no GPU needed): the binding
prototypes what include/moe_layer.h declares, arguments are refused before
anything is queued, and the kernels keep to their registers."""
import ctypes as C
import os
import re

import pytest
import torch

from conftest import ROOT
from quantized_moe_routed_gb300 import MoeError, Nvfp4Linear, add_rms_norm, binding, layer
from quantized_moe_routed_gb300 import build as libbuild

INVALID, MISALIGNED, SHAPE = (binding.MOE_ERR_INVALID_ARG, binding.MOE_ERR_MISALIGNED, binding.MOE_ERR_UNSUPPORTED_SHAPE)
A = 1 << 20  # stands for an aligned device pointer: never read


def _header():
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_layer.h")).read(), flags=re.S)


def test_binding_prototypes_what_the_header_declares():
    libbuild.build()
    src = _header()
    declared = set(re.findall(r"\b(moe_[a-z_]+)\s*\(", src))
    assert declared == set(layer.SIGNATURES), declared ^ set(layer.SIGNATURES)
    lib = layer._library()
    for name in declared:
        args = re.search(r"\b" + name + r"\s*\(([^()]*)\)", src).group(1)
        assert len(args.split(",")) == len(layer.SIGNATURES[name][1]), name
        assert hasattr(lib, name), name
    for struct in ("moe_kv_desc", "moe_kv_batch"):
        body = re.search(r"typedef struct \{([^{}]*)\}\s*" + struct + ";", src).group(1)
        names = re.findall(r"\*?\s*(\w+)\s*[,;]", body)
        assert names == [f for f, _ in getattr(layer, struct)._fields_], struct
    for name, value in (("MOE_KV_PAGE", layer.PAGE), ("MOE_KV_MAX_SEQS", layer.MAX_SEQS)):
        assert re.search(r"#define\s+" + name + r"\s+" + str(value) + r"\b", src), name


def _norm(x=A, f32=0, stride=256, r=None, r_out=None, w=A, eps=1e-6, y=A, q=None, qs=None, T=1, H=256):
    return layer._library().moe_norm(x, f32, stride, r, r_out, w, eps, y, q, qs, T, H, None)


@pytest.mark.parametrize("status,args", [
    (INVALID, dict(T=-1)), (SHAPE, dict(H=0)), (SHAPE, dict(H=12)), (SHAPE, dict(H=16392)), (SHAPE, dict(H=64, q=A, qs=A)),
    (INVALID, dict(f32=2)), (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(stride=255)),
    (INVALID, dict(y=None)), (INVALID, dict(q=A)), (INVALID, dict(qs=A)), (INVALID, dict(x=None)), (INVALID, dict(w=None)),
    (MISALIGNED, dict(x=A + 8)), (MISALIGNED, dict(r=A + 2)), (MISALIGNED, dict(stride=260)), (MISALIGNED, dict(q=A, qs=A + 2))])
def test_norm_refuses(status, args):
    assert _norm(**args) == status
    assert binding.moe_last_error()


def _linear(q=A, s=A, ts=A, N=16, K=64, x=A, stride=64, y=A, bf16=0, T=1):
    return layer._library().moe_linear(q, s, ts, N, K, x, stride, y, bf16, T, None)


@pytest.mark.parametrize("status,args", [
    (INVALID, dict(T=-1)), (INVALID, dict(T=1 << 22)), (SHAPE, dict(N=0)), (SHAPE, dict(K=0)), (SHAPE, dict(K=48, stride=48)),
    (SHAPE, dict(K=(1 << 22) + 32, stride=1 << 23)), (INVALID, dict(bf16=2)), (INVALID, dict(stride=63)),
    (INVALID, dict(q=None)), (INVALID, dict(s=None)), (INVALID, dict(ts=None)), (INVALID, dict(x=None)),
    (INVALID, dict(y=None)), (MISALIGNED, dict(q=A + 8)), (MISALIGNED, dict(s=A + 1)), (MISALIGNED, dict(ts=A + 2)),
    (MISALIGNED, dict(x=A + 2)), (MISALIGNED, dict(stride=68)), (MISALIGNED, dict(y=A + 2))])
def test_linear_refuses(status, args):
    assert _linear(**args) == status
    assert binding.moe_last_error()


def test_empty_steps_need_no_pointers():
    assert _norm(T=0, x=None, w=None, y=None) == binding.MOE_OK
    assert _linear(T=0, q=None, s=None, ts=None, x=None, y=None) == binding.MOE_OK


def _create(**change):
    f = dict(n_pages=4, q_heads=8, kv_heads=2, head_dim=64, k=A, v=A, ks=A, vs=A, rot_dim=64, inter=0, positions=16, rope=A,
             device=0)
    f.update(change)
    out = C.c_void_p()
    st = layer._library().moe_kv_create(C.byref(layer.moe_kv_desc(*f.values())), C.byref(out))
    assert not out
    return st


@pytest.mark.parametrize("status,change", [
    (SHAPE, dict(head_dim=96)), (SHAPE, dict(kv_heads=0)), (SHAPE, dict(kv_heads=3)), (SHAPE, dict(q_heads=1)),
    (SHAPE, dict(kv_heads=2048, q_heads=2048)), (SHAPE, dict(n_pages=0)), (SHAPE, dict(n_pages=1 << 24)),
    (SHAPE, dict(rot_dim=66)), (SHAPE, dict(rot_dim=3)), (SHAPE, dict(rot_dim=-2)), (INVALID, dict(inter=2)),
    (INVALID, dict(k=None)), (INVALID, dict(vs=None)), (INVALID, dict(rope=None)), (INVALID, dict(positions=0)),
    (MISALIGNED, dict(k=A + 8)), (MISALIGNED, dict(v=A + 4)), (MISALIGNED, dict(ks=A + 2)), (MISALIGNED, dict(rope=A + 4))])
def test_cache_refuses(status, change):
    assert _create(**change) == status
    assert binding.moe_last_error()


def test_null_handles_are_refused():
    lib = layer._library()
    batch = layer.moe_kv_batch(A, A, A, 1, 1, 1, 1)
    assert lib.moe_kv_create(None, None) == INVALID
    assert lib.moe_kv_workspace_bytes(None) == 0
    assert lib.moe_kv_workspace_init(None, A, 256, None) == INVALID
    assert lib.moe_kv_append(None, None, 0, A, 64, A, 64, None, C.byref(batch), A, None) == INVALID
    assert lib.moe_kv_attend(None, A, 64, 1.0, A, C.byref(batch), A, None) == INVALID
    assert lib.moe_kv_check(None, A, None) == INVALID
    lib.moe_kv_destroy(None)


def test_the_python_layer_refuses_host_tensors():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    for call in (lambda: add_rms_norm(x, w), lambda: add_rms_norm(x, w, outputs="fp8"), lambda: add_rms_norm(x[0], w),
                 lambda: Nvfp4Linear(torch.zeros((4, 16), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8),
                                     torch.ones(1))):
        with pytest.raises(MoeError) as ei:
            call()
        assert ei.value.status == INVALID


def test_rope_table_on_the_host():
    t = layer.rope_table(5, 8, theta=100.0, magnitude=2.0, device="cpu")
    assert t.shape == (5, 8) and t.dtype == torch.float32
    ang = 3 * 100.0 ** (-2 / 8)
    assert abs(float(t[3, 2]) - 2 * torch.cos(torch.tensor(ang)).item()) < 1e-6
    assert abs(float(t[3, 3]) - 2 * torch.sin(torch.tensor(ang)).item()) < 1e-6
    with pytest.raises(MoeError):
        layer.rope_table(5, 8, inv_freq=[1.0, 2.0], device="cpu")


@pytest.mark.parametrize("unit,regs", [("moe_norm.cu", 128), ("moe_linear.cu", 128), ("moe_linear_tc.cu", 128),
                                       ("moe_kv_append.cu", 64),
                                       ("moe_kv_attend.cu", 168), ("moe_kv_attend_tc.cu", 128)])
def test_kernels_fit_their_registers(unit, regs):
    # blocks of 512 threads have 128 registers a thread, of 384 have 168; two
    # append blocks share an SM.  A few values around the inner loops may spill.
    libbuild.build()
    text = open(os.path.join(libbuild.BUILD, unit + ".log")).read()
    used = [int(r) for r in re.findall(r"Used (\d+) registers", text)]
    spills = [int(a) + int(b) for a, b in re.findall(r"(\d+) bytes spill stores, (\d+) bytes spill loads", text)]
    assert used and max(used) <= regs, used
    assert max(spills) <= 512, spills
