"""moe_norm against its 64-bit definition.  bf16 outputs: half a bf16 step
(2^-8 relative) and the fp32 arithmetic (sum of H squares, a handful of
roundings: under 2^-16).  8-bit outputs: half an E4M3 step of the code plus the
same fp32 error; the block scale is the definition's unless the block's largest
lies within that error of 448 times a power of two."""
import pytest
import torch

import layer_reference as ref
from quantized_moe_routed_gb300 import MoeError, add_rms_norm, binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32 = 2.0 ** -16


def _inputs(T, H, x32, seed=0, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g) * gain
    x = x if x32 else x.bfloat16()
    r = (torch.randn((T, H), generator=g) * 3).bfloat16()
    w = (1 + 0.3 * torch.randn(H, generator=g)).bfloat16()
    return x, r, w


def _close_bf16(got, want):
    err = (got.cpu().double() - want).abs()
    assert bool((err <= (2.0 ** -8 + F32) * want.abs() + 1e-38).all()), float(err.max())


def _check_q(q, scale, y):
    T, H = y.shape
    b = y.view(T, H // 128, 128)
    amax = b.abs().amax(-1)
    lo, hi = ref.pow2_scale(amax * (1 - F32)), ref.pow2_scale(amax * (1 + F32))
    s = scale.cpu().double()
    assert bool(((s == lo) | (s == hi)).all())
    val = ref.e4m3(q.cpu().view(torch.uint8)).view(b.shape) * s[..., None]
    tol = ref.half_step(b / s[..., None]) * s[..., None] * (1 + 2.0 ** -10) + F32 * b.abs()
    assert bool(((val - b).abs() <= tol).all())


@pytest.mark.parametrize("T,H", [(1, 8), (1, 4096), (3, 264), (5, 128), (2, 16384), (7, 5120), (130, 1000), (300, 2048), (2, 12296)])
@pytest.mark.parametrize("x32", [False, True])
def test_norm_matches_the_definition(T, H, x32):
    x, r, w = _inputs(T, H, x32, seed=T + H)
    s, y = ref.norm(x, r, w, 1e-5)
    xd, rd, wd = x.to(DEV), r.to(DEV), w.to(DEV)
    ro = torch.empty_like(rd)
    outputs = "both" if H % 128 == 0 else "bf16"
    out = add_rms_norm(xd, wd, residual=rd, residual_out=ro, eps=1e-5, outputs=outputs)
    assert torch.equal(rd.cpu(), r)
    _close_bf16(ro, s)
    _close_bf16(out[0] if outputs == "both" else out, y)
    if outputs == "both":
        _check_q(out[1], out[2], y)
        q, sc = add_rms_norm(xd, wd, residual=rd, residual_out=ro, eps=1e-5, outputs="e4m3")
        assert torch.equal(q.view(torch.uint8), out[1].view(torch.uint8)) and torch.equal(sc, out[2])


def test_norm_in_place_residual_and_without():
    x, r, w = _inputs(4, 512, False, seed=5)
    s, y = ref.norm(x, r, w, 1e-6)
    rd = r.to(DEV)
    out = add_rms_norm(x.to(DEV), w.to(DEV), residual=rd)
    _close_bf16(rd, s)
    _close_bf16(out, y)
    out = add_rms_norm(x.to(DEV), w.to(DEV))
    _close_bf16(out, ref.norm(x, None, w, 1e-6)[1])


def test_norm_strided_rows_streams_and_empty():
    x, _, w = _inputs(6, 3 * 256, False, seed=8)
    xd = x.to(DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = add_rms_norm(xd[:, 256:512], w[:256].to(DEV), stream=st)
    st.synchronize()
    _close_bf16(out, ref.norm(x[:, 256:512], None, w[:256], 1e-6)[1])
    assert add_rms_norm(xd[:0], w.to(DEV)).shape == (0, 768)


@pytest.mark.parametrize("gain", [1e-30, 1e-12, 1e12])
def test_norm_small_and_large_rows(gain):
    x, _, w = _inputs(3, 256, True, seed=11, gain=gain)
    x[1] = 0
    s, y = ref.norm(x, None, w, 1e-6)
    out, q, sc = add_rms_norm(x.to(DEV), w.to(DEV), outputs="both")
    _close_bf16(out, y)
    _check_q(q, sc, y)
    assert bool((q[1].view(torch.uint8) == 0).all()) and bool((sc[1] == 2.0 ** -64).all())


def test_norm_nan_and_infinity_stay_in_their_rows():
    x, _, w = _inputs(4, 256, True, seed=12)
    y = ref.norm(x, None, w, 1e-6)[1]
    x[1, 7], x[2, 100] = float("nan"), float("inf")
    out, q, sc = add_rms_norm(x.to(DEV), w.to(DEV), outputs="both")
    _close_bf16(out[[0, 3]], y[[0, 3]])
    _check_q(q[[0, 3]], sc[[0, 3]], y[[0, 3]])
    assert bool(out[1].isnan().all()) and bool(out[2, 100].isnan())
    assert bool((q.view(torch.uint8)[1] & 127 == 127).all()) and int(q.view(torch.uint8)[2, 100]) & 127 == 127
    assert bool(sc.isfinite().all())


def test_norm_is_bitwise_reproducible_and_captures():
    x, r, w = (t.to(DEV) for t in _inputs(33, 4096, False, seed=3))
    ro = torch.empty_like(r)
    first = add_rms_norm(x, w, residual=r, residual_out=ro, outputs="both")
    out = [torch.empty_like(t) for t in first]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        add_rms_norm(x, w, residual=r, residual_out=ro, outputs="both", out=out[0], out_q=out[1], out_scale=out[2])
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, out):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_norm_refusals():
    x, r, w = (t.to(DEV) for t in _inputs(4, 256, False))
    big = torch.zeros((1, 16392), dtype=torch.bfloat16, device=DEV)
    flat = torch.zeros(4 * 256 + 8, dtype=torch.bfloat16, device=DEV)
    cases = [(lambda: add_rms_norm(x[:, :252], w[:252]), binding.MOE_ERR_UNSUPPORTED_SHAPE),
             (lambda: add_rms_norm(big, big[0]), binding.MOE_ERR_UNSUPPORTED_SHAPE),
             (lambda: add_rms_norm(x[:, :136].contiguous(), w[:136], outputs="e4m3"), binding.MOE_ERR_UNSUPPORTED_SHAPE),
             (lambda: add_rms_norm(flat[4:4 + 1024].view(4, 256), w), binding.MOE_ERR_MISALIGNED),
             (lambda: add_rms_norm(x.half(), w), binding.MOE_ERR_INVALID_ARG),
             (lambda: add_rms_norm(x, w[:128]), binding.MOE_ERR_INVALID_ARG),
             (lambda: add_rms_norm(x, w, residual=r[:2]), binding.MOE_ERR_INVALID_ARG),
             (lambda: add_rms_norm(x, w, eps=-1.0), binding.MOE_ERR_INVALID_ARG),
             (lambda: add_rms_norm(x, w, residual_out=r), binding.MOE_ERR_INVALID_ARG),
             (lambda: add_rms_norm(x.t(), w), binding.MOE_ERR_INVALID_ARG),
             (lambda: add_rms_norm(x, w, outputs="fp8"), binding.MOE_ERR_INVALID_ARG)]
    for call, status in cases:
        with pytest.raises(MoeError) as ei:
            call()
        assert ei.value.status == status
