"""moe_kv_attend over long runs of one tile: what the tensor cores' additions cut off
must not grow with the length.  Values are positive, each head dim of its own size, so
that every addition cuts the same way; batches have about as many tiles as the GPU
has SMs or more, so that a block keeps a tile for long, and all sequences read the
same pages (the cache stays small).  sum(err * o) / sum(o * o) is what the output has
lost: a bf16 output's own rounding, 2^-8 of an element at most, has either sign and
averages out over the elements that differ (2^-13 where all weights are about equal and
the sequences' outputs alike, far less else).

128 rows: 1024 additions of 16 tokens in a run at most, each cutting less than 2^-23 of
the sum so far, which is half of the last on average: under 2^-13, and as much again for
the other steps (weights, runs and tiles joined): 2^-12.  One run over 262144 tokens
loses 1.6e-3.

8 and 16 rows: a warp's run has an addition for 128 tokens of the tile: 2^-12 holds up to
131072 tokens by the same count."""
import pytest
import torch

from quantized_moe_routed_gb300 import KVCache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _values(L, D, gain, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = (L + 63) // 64
    e4 = torch.float8_e4m3fn
    k = (torch.randn((n, 1, 64, D), generator=g, device=DEV) * gain).clamp(-448, 448).to(e4)
    size = 0.5 + torch.rand((1, 1, D, 1), generator=g, device=DEV)
    v = (torch.rand((n, 1, D, 64), generator=g, device=DEV).square() * size * 250).to(e4)
    return k, v, g


def _lost(lengths, n, G, D, gain, seed=0):
    """What the outputs of each sequence's last token have lost."""
    top = max(lengths)
    k, v, g = _values(top, D, gain, seed)
    B, pages = len(lengths), k.shape[0]
    sc = torch.full((pages, 1), 2.0 ** -6, device=DEV)
    cache = KVCache(pages, G, 1, D, buffers=dict(k=k.view(torch.uint8), v=v.view(torch.uint8), k_scale=sc, v_scale=sc.clone()))
    ws = cache.new_workspace()
    q = torch.randn((B * n, G, D), generator=g, device=DEV).bfloat16()
    ids = torch.arange(pages, dtype=torch.int32, device=DEV)[None].expand(B, -1).contiguous()
    args = ((torch.arange(B + 1, device=DEV) * n).int(), torch.tensor(lengths, dtype=torch.int32, device=DEV), ids, ws, n)
    out = cache.attend(q, *args)
    assert torch.equal(cache.attend(q, *args), out)
    assert cache.check(ws) == 0
    kk, vv = k.double().reshape(-1, D) / 64, v.double().transpose(2, 3).reshape(-1, D) / 64
    num = den = err2 = 0.0
    for b in range(0, B, max(1, B // 20)):
        L, r = lengths[b], (b + 1) * n - 1
        o = torch.softmax(q[r].double() @ kk[:L].T * D ** -0.5, -1) @ vv[:L]
        e = out[r].double() - o
        num, den, err2 = num + float((e * o).sum()), den + float((o * o).sum()), err2 + float((e * e).sum())
    assert (err2 / den) ** 0.5 < 2.0 ** -9
    return num / den


RAGGED = [262144 - 1000 * b for b in range(100)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gain", [1.0, 60.0, 240.0])
@pytest.mark.parametrize("lengths", [[262144] * 152, RAGGED, [40000, 100, 16384, 16385, 24576, 24705, 32768, 33000] * 60],
                         ids=["a tile a block", "cut tiles", "several tiles a block"])
def test_many_rows(D, gain, lengths):
    assert abs(_lost(lengths, 4, 32, D, gain)) < 2.0 ** -12


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [8, 16])
def test_few_rows(D, G):
    assert abs(_lost([131072] * 152, 1, G, D, 60.0)) < 2.0 ** -12
