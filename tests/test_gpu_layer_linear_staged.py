"""moe_linear where x is staged in shared memory (more tiles of 16 rows than a block
each, lengths or scales that the tensor-core kernel does not take): against the
64-bit definition with the bound of test_gpu_layer_linear.py.  On 152 SMs the sizes
below take, in turn: warps that share a tile's K (sums added across warps); x in
pieces, two in shared memory, for one tile a warp and for two; two tiles a warp
with 8, 16 and 24 tokens; two passes of a block over K, with x staged once and again;
tokens in two groups; a last tile of few rows, a last chunk of K that is not whole."""
import pytest
import torch

from quantized_moe_routed_gb300 import Nvfp4Linear
from test_gpu_layer_linear import _weights
from test_gpu_layer_linear_tc import _check_rows, _linear, _x

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

CASES = [
    # N, K, tokens
    (8192, 4096, (1, 3, 8)),            # four warps a tile
    (12000, 1056, (1, 8, 16, 24)),      # two, and a last chunk of 32
    (9731, 96, (2, 24)),                # one chunk of K in all
    (20003, 8224, (8, 16, 24)),         # x whole for 8 tokens, in pieces for more; one tile a warp
    (40000, 544, (5, 12, 24)),          # two tiles a warp, x whole
    (50001, 2112, (8, 16, 24)),         # two tiles a warp, x in pieces for 16 and 24
    (100003, 1056, (1, 16, 24, 40)),    # two passes, x whole
    (100003, 4128, (1, 16, 24, 40)),    # two passes, x in pieces
]


@pytest.mark.parametrize("N,K,tokens", CASES)
def test_staged_products(N, K, tokens):
    w = _weights(N, K, seed=N + K, signed_scales=True)
    lin = _linear(w)
    for T in tokens:
        x = _x(T, K, seed=T)
        y = lin(x.to(DEV))
        assert bool(torch.isfinite(y).all())
        _check_rows(y, x, w)
        _check_rows(lin(x.to(DEV), dtype=torch.bfloat16), x, w, bf16=True)
        assert torch.equal(lin(x.to(DEV)), y)


@pytest.mark.parametrize("N,K,tokens", [(20003, 4096, (1, 16, 24)), (50001, 2048, (16, 24)), (100003, 2048, (8, 24))])
def test_scales_that_are_not_16_byte_aligned(N, K, tokens):
    """Sizes that the tensor-core kernel would take otherwise."""
    w = _weights(N, K, seed=N + K)
    buf = torch.zeros(w[1].numel() + 16, dtype=torch.uint8, device=DEV)
    s = buf[6:6 + w[1].numel()].view(w[1].shape)
    s.copy_(w[1])
    lin = Nvfp4Linear(w[0].to(DEV), s, w[2].to(DEV))
    for T in tokens:
        x = _x(T, K, seed=T)
        _check_rows(lin(x.to(DEV)), x, w)


@pytest.mark.parametrize("T", [1, 24])
def test_range_and_nan_in_pieces(T):
    """Chunks of very different magnitude in the pieces, zero tokens, a NaN that stays in its token."""
    N, K = 50001, 2112
    w = _weights(N, K, seed=5)
    x = _x(T, K).float()
    x[0, 128:256] *= 1e-20
    x[0, 1024:1152] *= 1e6
    if T > 1:
        x[1] *= 1e-34
        x[2] = 0
    x = x.bfloat16()
    dirty = x.clone()
    if T > 1:
        dirty[3, 2100] = float("nan")
    y = _linear(w)(dirty.to(DEV))
    keep = [t for t in range(T) if t != 3]
    _check_rows(y[keep], x[keep], w)
    if T > 1:
        assert bool(y[3].isnan().all()) and bool((y[2] == 0).all())
