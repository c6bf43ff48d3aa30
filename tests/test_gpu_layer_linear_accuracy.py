"""How exact moe_linear's sums are, in the norm: each token's outputs against the
64-bit definition, for normal weights as an NVFP4 quantiser leaves them.  The operands
are exact, so this is the sums alone: tensor-core additions over 128 (staged and few-tiles
kernels) or 512 elements of K, from there on additions in fp32 that round.  The
latter are off by 2^-25 / sqrt(3) of the sum so far each, of either sign: 64 of them by
1.4e-7; the former by 1.1e-7 of the result at these lengths.  Together under 3e-7; sums
on the tensor cores over all of K = 4096 are off by 1e-6.

And a token's bits in a batch against its bits alone, where one kernel serves both."""
import pytest
import torch

import layer_reference as ref
from quantized_moe_routed_gb300 import Nvfp4Linear
from quantized_moe_routed_gb300.inputs import quantize_nvfp4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _weights(N, K, seed):
    g = torch.Generator().manual_seed(seed)
    q, s, _ = quantize_nvfp4(torch.randn((N, K), generator=g) * 0.02)
    return q, s, (1 + torch.rand(N, generator=g)) * 1e-3


# few tiles, staged (a tile by several warps, x in pieces), tensor cores (one, two, four tiles a block)
@pytest.mark.parametrize("N,K,T", [
    (256, 4096, 16), (4096, 4096, 1), (2048, 8192, 24), (8192, 4096, 8), (12000, 4128, 16), (12161, 4096, 24), (12161, 8192, 1),
    (19457, 4096, 24), (40003, 4096, 1), (40003, 4096, 24), (40003, 4096, 40), (40003, 8192, 16)])
def test_sums_in_the_norm(N, K, T):
    q, s, ts = _weights(N, K, seed=N + K)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).bfloat16()
    y = Nvfp4Linear(q.to(DEV), s.to(DEV), ts.to(DEV))(x.to(DEV))
    pick = torch.randperm(N, generator=torch.Generator().manual_seed(0))[:4000]
    want = (x.to(DEV).double() @ (ref.nvfp4(q[pick], s[pick]) * ts[pick].double()[:, None]).to(DEV).T)
    err = (y[:, pick.to(DEV)].double() - want).norm(dim=1) / want.norm(dim=1)
    assert float(err.max()) < 3e-7, float(err.max())


@pytest.mark.parametrize("T", [2, 8, 9, 17, 24, 30])
def test_a_token_alone_and_in_a_batch(T):
    """512 rows are a block a tile for any number of tokens."""
    q, s, ts = (t.to(DEV) for t in _weights(512, 2048, seed=7))
    lin = Nvfp4Linear(q, s, ts)
    x = torch.randn((T, 2048), generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    y = lin(x)
    for t in range(T):
        assert torch.equal(y[t], lin(x[t:t + 1])[0])
