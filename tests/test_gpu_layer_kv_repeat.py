"""moe_kv_attend run again and again: the same bits every time on batches whose
tiles are cut between blocks, and pages that are all out of range (a block then has
nothing to wait for, and its warps run ahead of each other as far as they can)."""
import pytest
import torch

import layer_reference as ref
from quantized_moe_routed_gb300 import KVCache, binding
from test_gpu_layer_kv import Step, _cache, _check_attend, _gather, _pool

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _lengths(seed, B, top):
    return torch.randint(1, top, (B,), generator=torch.Generator().manual_seed(seed)).tolist()


# new tokens of each sequence, lengths, query heads on 2 of kv: rows of 8, 16, 128
CASES = [([1] * 96, _lengths(1, 96, 5000), 8), ([1] * 7, _lengths(2, 7, 30000), 16), ([3] * 40, _lengths(3, 40, 3000), 8),
         ([5] * 24, [5 + n for n in _lengths(4, 24, 4000)], 8), ([1, 300, 17, 1, 64, 129], [9000, 1300, 2500, 1, 64, 700], 16)]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("D", [64, 128])
def test_the_same_bits_every_time(case, D):
    ql, L, Hq = CASES[case]
    step = Step(ql, L, seed=case)
    bufs = _pool(step, 2, D, seed=case)
    cache = _cache(bufs, Hq, 2, D)
    q = torch.randn((step.N, Hq, D), generator=torch.Generator().manual_seed(case)).bfloat16().to(DEV)
    ws = cache.new_workspace()
    args = (*step.dev(), ws, step.max_q)
    first = cache.attend(q, *args)
    assert bool(torch.isfinite(first).all())
    out = torch.empty_like(first)
    for _ in range(30):
        out.fill_(float("nan"))
        cache.attend(q, *args, out=out)
        assert torch.equal(out, first)
    assert cache.check(ws) == 0


@pytest.mark.parametrize("case", range(len(CASES)))
def test_pages_that_are_all_out_of_range(case):
    ql, L, Hq = CASES[case]
    step = Step(ql, L, seed=case)
    cache = _cache(_pool(step, 2, 128, seed=case), Hq, 2, 128)
    q = torch.randn((step.N, Hq, 128), generator=torch.Generator().manual_seed(case)).bfloat16().to(DEV)
    q_off, kv_len, pages = step.dev()
    ws = cache.new_workspace()
    good = cache.attend(q, q_off, kv_len, pages, ws, step.max_q)
    for bad in (-1, step.n_pages, 2 ** 31 - 1, -2 ** 31):
        for _ in range(5):
            out = cache.attend(q, q_off, kv_len, torch.full_like(pages, bad), ws, step.max_q)
            assert bool((out == 0).all())
        assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX
    # and in turn with good ones, every other page: nothing is left over from call to call
    mixed = pages.clone()
    mixed[:, 1::2] = -7
    a = cache.attend(q, q_off, kv_len, mixed, ws, step.max_q)
    assert torch.equal(cache.attend(q, q_off, kv_len, pages, ws, step.max_q), good)
    assert torch.equal(cache.attend(q, q_off, kv_len, mixed, ws, step.max_q), a)
    assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX and cache.check(ws) == 0


def test_one_long_sequence_beside_many_short():
    step = Step([1] * 64, [60001] + [n for n in _lengths(9, 63, 100)], seed=3)
    bufs = _pool(step, 1, 64, seed=3)
    cache = _cache(bufs, 4, 1, 64)
    q = torch.randn((64, 4, 64), generator=torch.Generator().manual_seed(3)).bfloat16()
    ws = cache.new_workspace()
    out = cache.attend(q.to(DEV), *step.dev(), ws, 1)
    assert cache.check(ws) == 0
    _check_attend(step, bufs, q, out, 64 ** -0.5)


@pytest.mark.parametrize("n,Hq", [(1, 4), (5, 4), (9, 8), (100, 4), (40, 32)])
@pytest.mark.parametrize("D", [64, 128])
def test_bad_pages_count_as_tokens_that_nothing_sees(n, Hq, D):
    """The same as the sequence without those pages' tokens."""
    step = Step([n], [700], seed=n)
    bufs = _pool(step, 2, D, seed=n)
    cache = _cache(bufs, Hq, 2, D)
    q = torch.randn((n, Hq, D), generator=torch.Generator().manual_seed(n)).bfloat16()
    pages, ws = step.pages.clone(), cache.new_workspace()
    bad = [0, 3, 4, 7]
    pages[0, bad] = torch.tensor([-1, step.n_pages, 1 << 30, -(1 << 31)], dtype=torch.int32)
    out = cache.attend(q.to(DEV), step.q_off.to(DEV), step.kv_len.to(DEV), pages.to(DEV), ws, n)
    assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX
    rest = Step([n], [700 - 64 * len(bad)], seed=n)
    rest.pages = step.pages[:, [i for i in range(step.pages.shape[1]) if i not in bad]]
    _check_attend(rest, bufs, q, out, D ** -0.5)


@pytest.mark.parametrize("gain", [1, 3, 5])
@pytest.mark.parametrize("n,Hq,Hkv,D", [(16, 64, 8, 128), (16, 64, 8, 64), (200, 16, 4, 128), (1, 64, 8, 128)])
def test_rows_whose_maximum_moves_now_and_then(n, Hq, Hkv, D, gain):
    """Long sequences and scores of several units: some row's running maximum moves
    far, and its accumulators are rescaled between products that are in flight."""
    L = [16400, 9488, 2576, 12048, 5136, 14608, 7696, 784]
    for seed in range(6):
        step = Step([n] * len(L), L, seed=seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        k, v = ((torch.randn(s, generator=g, device=DEV) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for s in ((step.n_pages, Hkv, 64, D), (step.n_pages, Hkv, D, 64)))
        sc = torch.full((step.n_pages, Hkv), 2.0 ** -6, device=DEV)
        cache = KVCache(step.n_pages, Hq, Hkv, D, buffers=dict(k=k, v=v, k_scale=sc, v_scale=sc.clone()))
        q = (torch.randn((step.N, Hq, D), generator=g, device=DEV) * gain).bfloat16()
        ws = cache.new_workspace()
        args = (*step.dev(), ws, n)
        first = cache.attend(q, *args)
        assert sum(not torch.equal(cache.attend(q, *args), first) for _ in range(100)) == 0
        assert cache.check(ws) == 0
        # one sequence and kv head against the definition
        b, h, G = 7, Hkv - 1, Hq // Hkv
        kk, vv = _gather(step, [t.cpu() for t in (k, v, sc, sc)], b, h)
        got = first[b * n:(b + 1) * n, h * G:].cpu().double()
        want = ref.attend(q[b * n:(b + 1) * n, h * G:].cpu(), kk, vv, n, L[b], D ** -0.5)[0]
        assert float((got - want).norm() / want.norm()) < 2 ** -6
