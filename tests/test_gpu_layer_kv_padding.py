"""moe_kv_attend on batches with sequences that see nothing: lengths of zero, and
more new tokens than the sequence holds, as the padding of a captured batch has
them.  Many in a row give a block one tile after another without a step; such
tiles are zeros, the tiles between them are what they are without the padding, and
no wait runs out, whatever the warps' pace."""
import pytest
import torch

from test_gpu_layer_kv import Step, _cache, _check_attend, _pool

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _attend(step, bufs, Hq, q, calls):
    """The output of `calls` equal calls, and the workspace's status."""
    Hkv, D = bufs[0].shape[1], bufs[0].shape[3]
    cache = _cache(bufs, Hq, Hkv, D)
    ws = cache.new_workspace()
    args = (*step.dev(), ws, step.max_q)
    qd = q.to(DEV)
    first = cache.attend(qd, *args)
    out = torch.empty_like(first)
    for _ in range(calls - 1):
        out.fill_(float("nan"))
        cache.attend(qd, *args, out=out)
        assert torch.equal(out, first)
    return first, cache.check(ws)


# new tokens of a padding sequence and query heads on 2 of kv: tiles of 8, 16 and 128 rows
# (one, one, and one to five a sequence)
@pytest.mark.parametrize("n,Hq", [(1, 8), (4, 8), (20, 8), (32, 8), (150, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_batch_of_padding_only(n, Hq, D):
    step = Step([n] * 300, [0] * 150 + [0, 1] * 75, seed=n)
    bufs = _pool(step, 2, D, seed=n)
    q = torch.randn((step.N, Hq, D), generator=torch.Generator().manual_seed(n)).bfloat16()
    out, status = _attend(step, bufs, Hq, q, 100)
    assert status == 0
    see = [int(step.q_off[b]) + n - 1 for b in range(300) if step.L[b] == 1]  # the last token of these sees itself
    rest = torch.ones(step.N, dtype=torch.bool)
    rest[see] = False
    assert bool((out[rest.to(DEV)] == 0).all())
    _check_attend(step, bufs, q, out, D ** -0.5)


@pytest.mark.parametrize("n", [20, 40, 150])
@pytest.mark.parametrize("D", [64, 128])
def test_padding_between_live_sequences(n, D):
    live = {3: 700, 40: 65, 41: 130, 90: 1, 199: 300}
    step = Step([n] * 200, [live.get(b, 0) for b in range(200)], seed=n)
    bufs = _pool(step, 2, D, seed=n)
    q = torch.randn((step.N, 8, D), generator=torch.Generator().manual_seed(n)).bfloat16()
    out, status = _attend(step, bufs, 8, q, 100)
    assert status == 0
    _check_attend(step, bufs, q, out, D ** -0.5)
    empty = torch.tensor([b not in live for b in range(200)]).repeat_interleave(n)
    assert bool((out[empty.to(DEV)] == 0).all())


@pytest.mark.parametrize("n", [1, 4, 40])
def test_rows_outside_every_sequence_are_left_alone(n):
    """A step's arrays may be longer than its sequences (padding of a captured batch),
    in front and behind: those rows are not read, and not written."""
    step = Step([n, n], [n + 70, n], seed=n)
    bufs = _pool(step, 2, 128, seed=n)
    q_off, kv_len, pages = step.dev()
    N = step.N + 5
    g = torch.Generator().manual_seed(n)
    qkv = torch.randn((N, 12, 128), generator=g).bfloat16()
    qkv[:2], qkv[-3:] = float("nan"), float("nan")
    q, k, v = qkv.to(DEV).split((8, 2, 2), dim=1)
    cache, alone = _cache(bufs, 8, 2, 128), _cache(bufs, 8, 2, 128)
    ws = cache.new_workspace()
    q_out, out = (torch.full((N, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache.append(k, v, q_off + 2, kv_len, pages, ws, n, q=q, q_out=q_out)
    cache.attend(q_out, q_off + 2, kv_len, pages, ws, n, out=out)
    assert cache.check(ws) == 0
    want_q = alone.append(k[2:-3], v[2:-3], q_off, kv_len, pages, ws, n, q=q[2:-3])
    want = alone.attend(want_q, q_off, kv_len, pages, ws, n)
    for got, inner in ((q_out, want_q), (out, want)):
        assert torch.equal(got[2:-3], inner)
        assert bool((got[:2] == 7).all()) and bool((got[-3:] == 7).all())
    assert torch.equal(cache.k, alone.k) and torch.equal(cache.v, alone.v)
