"""moe_linear against its 64-bit definition.  The weights are exact and so is x
(8 significant bits, down to 2^-28 of its chunk's largest), so what is left is
the fp32 sums: K / 16 tensor-core steps, the chunks' and the warps' sums, each
within 2^-22 of the sum of magnitudes so far."""
import pytest
import torch

import layer_reference as ref
from quantized_moe_routed_gb300 import MoeError, Nvfp4Linear, binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _weights(N, K, seed, signed_scales=False):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = torch.randint(1, 0x7F, (N, K // 16), generator=g, dtype=torch.uint8)
    if signed_scales:
        s |= torch.randint(0, 2, s.shape, generator=g, dtype=torch.uint8) << 7
    ts = torch.rand(N, generator=g) * 0.01 + 1e-4
    return q, s, ts


def _check(y, x, q, s, ts, bf16=False):
    w = ref.nvfp4(q, s) * ts.double()[:, None]
    want, mag = x.double() @ w.T, x.double().abs() @ w.abs().T
    tol = 2.0 ** -22 * (q.shape[1] / 8 + 16) * mag + (2.0 ** -8 * want.abs() if bf16 else 0) + 1e-38
    err = (y.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("T", [1, 2, 8, 9, 16, 17, 24, 25, 60])
@pytest.mark.parametrize("N,K", [(1, 32), (16, 64), (33, 160), (256, 4096), (1000, 1056)])
def test_linear_matches_the_definition(T, N, K):
    q, s, ts = _weights(N, K, seed=T + N + K, signed_scales=T == 9)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).bfloat16()
    lin = Nvfp4Linear(q.to(DEV), s.to(DEV), ts.to(DEV))
    _check(lin(x.to(DEV)), x, q, s, ts)
    _check(lin(x.to(DEV), dtype=torch.bfloat16), x, q, s, ts, bf16=True)


@pytest.mark.parametrize("T", [1, 12, 24])
def test_linear_many_rows(T):
    N, K = 20003, 512
    q, s, ts = _weights(N, K, seed=2)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(1)).bfloat16()
    _check(Nvfp4Linear(q.to(DEV), s.to(DEV), ts.to(DEV))(x.to(DEV)), x, q, s, ts)


@pytest.mark.parametrize("gain", [1e-34, 1e-20, 1e6, 1e30])
def test_linear_range_of_x(gain):
    """Tokens and chunks of very different magnitude, a zero token, a zero chunk."""
    q, s, ts = _weights(48, 512, seed=4)
    x = torch.randn((5, 512), generator=torch.Generator().manual_seed(1))
    x[1] *= gain
    x[2, 128:256] *= gain
    x[3] = 0
    x[4, :128] = 0
    x = x.bfloat16()
    y = Nvfp4Linear(q.to(DEV), s.to(DEV), ts.to(DEV))(x.to(DEV))
    _check(y, x, q, s, ts)
    assert bool((y[3] == 0).all())


def test_linear_nan_and_infinity_stay_in_their_token():
    q, s, ts = _weights(32, 256, seed=4)
    x = torch.randn((4, 256), generator=torch.Generator().manual_seed(1)).bfloat16()
    clean = x.clone()
    x[1, 9], x[2, 200] = float("nan"), float("inf")
    y = Nvfp4Linear(q.to(DEV), s.to(DEV), ts.to(DEV))(x.to(DEV))
    _check(y[[0, 3]], clean[[0, 3]], q, s, ts)
    assert bool(y[1].isnan().all()) and bool((~y[2].isfinite()).all())


def test_linear_strided_x_one_scale_stream_and_empty():
    q, s, ts = _weights(64, 128, seed=6)
    x = torch.randn((6, 384), generator=torch.Generator().manual_seed(1)).bfloat16()
    lin = Nvfp4Linear(q.to(DEV), s.to(DEV), ts[:1].to(DEV))
    xd = x.to(DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = lin(xd[:, 128:256], stream=st)
    st.synchronize()
    _check(y, x[:, 128:256], q, s, ts[:1].expand(64))
    assert lin(xd[:0, :128]).shape == (0, 64)


def test_linear_is_bitwise_reproducible_and_independent_of_the_batch():
    q, s, ts = (t.to(DEV) for t in _weights(512, 2048, seed=7))
    lin = Nvfp4Linear(q, s, ts)
    x = torch.randn((8, 2048), generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    y = lin(x)
    out = torch.empty_like(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin(x, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, out)


def test_linear_refusals():
    q, s, ts = (t.to(DEV) for t in _weights(16, 64, seed=1))
    lin = Nvfp4Linear(q, s, ts)
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV)
    flat = torch.zeros(256, dtype=torch.bfloat16, device=DEV)
    inv, mis = binding.MOE_ERR_INVALID_ARG, binding.MOE_ERR_MISALIGNED
    cases = [(lambda: lin(x[:, :32]), inv), (lambda: lin(x.float()), inv), (lambda: lin(x.cpu()), inv),
             (lambda: lin(x, dtype=torch.float16), inv), (lambda: lin(x, out=torch.empty((2, 15), device=DEV)), inv),
             (lambda: lin(flat[4:132].view(2, 64)), mis), (lambda: lin(torch.as_strided(flat, (2, 64), (68, 1))), mis),
             (lambda: Nvfp4Linear(q, s[:, :2].contiguous(), ts), inv), (lambda: Nvfp4Linear(q, s, ts[:3]), inv),
             (lambda: Nvfp4Linear(q[:, :8].contiguous(), s[:, :1].contiguous(), ts)(x[:, :16].contiguous()),
              binding.MOE_ERR_UNSUPPORTED_SHAPE)]
    for call, status in cases:
        with pytest.raises(MoeError) as ei:
            call()
        assert ei.value.status == status
