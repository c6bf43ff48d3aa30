"""moe_linear where the weights have many rows (the tensor-core kernel): against
the 64-bit definition with the bound of test_gpu_layer_linear.py, whose K / 16
sums these are too; x is exact down to 2^-31 of its token's largest element, and
what is smaller is off by 2^-39 of that largest an element."""
import pytest
import torch

from quantized_moe_routed_gb300 import Nvfp4Linear
from test_gpu_layer_linear import _check, _weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _pick(N):
    """Rows to compare: the ends, and some of every block's."""
    g = torch.Generator().manual_seed(0)
    return torch.unique(torch.cat([torch.arange(600), torch.randint(0, N, (1200,), generator=g), torch.arange(N - 600, N)]))


def _check_rows(y, x, w, pick=None, bf16=False):
    pick = _pick(w[0].shape[0]) if pick is None else pick
    _check(y[:, pick.to(DEV)], x, *(t[pick] for t in w), bf16=bf16)


def _linear(w):
    return Nvfp4Linear(*(t.to(DEV) for t in w))


@pytest.fixture(scope="module")
def many():
    w = _weights(50001, 1024, seed=11, signed_scales=True)
    return w, _linear(w)


def _x(T, K, seed=1):
    return torch.randn((T, K), generator=torch.Generator().manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 130])
def test_tokens(many, T):
    w, lin = many
    x = _x(T, 1024)
    y = lin(x.to(DEV))
    assert bool(torch.isfinite(y).all())
    _check_rows(y, x, w)
    _check_rows(lin(x.to(DEV), dtype=torch.bfloat16), x, w, bf16=True)


# one tile a block, two, four of fewer rows, four, several waves
@pytest.mark.parametrize("N,K", [(12161, 4096), (19457, 4096), (40001, 2048), (77824, 1024), (155649, 512)])
@pytest.mark.parametrize("T", [1, 24, 40])
def test_rows_and_lengths(N, K, T):
    w = _weights(N, K, seed=N)
    x = _x(T, K)
    y = _linear(w)(x.to(DEV))
    assert bool(torch.isfinite(y).all())
    _check_rows(y, x, w)


def test_long_rows_and_repeats():
    w = _weights(10001, 8192, seed=3)
    lin = _linear(w)
    x = _x(20, 8192).to(DEV)
    y = lin(x)
    _check_rows(y, x.cpu(), w)
    for _ in range(20):
        assert torch.equal(lin(x), y)


@pytest.mark.parametrize("gain", [1e-34, 1e-20, 1e6, 1e30])
def test_range_of_x(many, gain):
    w, lin = many
    x = _x(5, 1024).float()
    x[1] *= gain
    x[2, 128:256] *= gain
    x[3] = 0
    x[4, :128] = 0
    x = x.bfloat16()
    y = lin(x.to(DEV))
    _check_rows(y, x, w)
    assert bool((y[3] == 0).all())


def test_nan_and_infinity_stay_in_their_token(many):
    w, lin = many
    x = _x(18, 1024)
    clean = x.clone()
    x[1, 9], x[2, 200], x[17, 500] = float("nan"), float("inf"), float("nan")
    y = lin(x.to(DEV))
    keep = [t for t in range(18) if t not in (1, 2, 17)]
    _check_rows(y[keep], clean[keep], w)
    assert bool(y[[1, 17]].isnan().all()) and bool((~y[2].isfinite()).any())


def test_strides_alignment_streams_and_graphs(many):
    w, lin = many
    wide = _x(6, 2048)
    st = torch.cuda.Stream()
    xd = wide.to(DEV)
    st.wait_stream(torch.cuda.current_stream())
    y = lin(xd[:, 512:1536], stream=st)
    st.synchronize()
    _check_rows(y, wide[:, 512:1536], w)
    out = torch.empty_like(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin(xd[:, 512:1536], out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)
    # scales that are not 16-byte aligned take the other kernel: the same product
    buf = torch.zeros(w[1].numel() + 16, dtype=torch.uint8, device=DEV)
    off = buf[2:2 + w[1].numel()].view(w[1].shape)
    off.copy_(w[1])
    other = Nvfp4Linear(w[0].to(DEV), off, w[2].to(DEV))(xd[:, 512:1536])
    _check_rows(other, wide[:, 512:1536], w)
