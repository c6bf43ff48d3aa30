"""The cache's moves: moe_kv_compact and moe_kv_fork against their definitions.  Codes are
exact: they stay, or are E4M3's nearest to code * (ratio of scales), a product whose
fp32 rounding is none for powers of two."""
import pytest
import torch

import layer_reference as ref
import speculate_reference as spec
import test_gpu_layer_kv as base
from quantized_moe_routed_gb300 import KVCache, MoeError, binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 64


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def _table(keeps):
    K = max([len(k) for k in keeps] + [1])
    t = torch.full((len(keeps), K), -7, dtype=torch.int32)     # entries behind the kept ones are not read
    for b, k in enumerate(keeps):
        t[b, :len(k)] = torch.tensor(k, dtype=torch.int32)
    return t.to(DEV), torch.tensor([len(k) for k in keeps], dtype=torch.int32, device=DEV)


def _values(cache):
    return ref.e4m3(cache.k.cpu()), ref.e4m3(cache.v.cpu()), cache.k_scale.cpu().double(), cache.v_scale.cpu().double()


def _same(a, b):
    return all(bool(((x == y) | (x.isnan() & y.isnan())).all()) for x, y in zip(a, b))


COMPACT = [
    # ql, L, kept, Hkv, D
    ([1], [1], [[0]], 1, 64), ([1], [64], [[]], 2, 128), ([5], [5], [[0, 2, 4]], 2, 128), ([16], [4017], [[0, 3, 7, 15]], 8, 128),
    ([8, 0, 3], [70, 9, 64], [[1, 2, 3, 7], [], [2]], 4, 64), ([8], [200], [[0, 1, 2]], 2, 64),
    ([70], [134], [[0, 1, 66, 69]], 2, 128), ([130], [140], [list(range(60, 130))], 2, 64),
    ([256], [319], [list(range(0, 256, 2))], 1, 128), ([256, 60], [256, 124], [list(range(256)), [59]], 3, 64),
    ([200], [1000], [list(range(1, 200))], 2, 128), ([100], [130], [[99]], 1, 64), ([65, 2], [129, 66], [[64], [1]], 2, 128),
]


@pytest.mark.parametrize("exps", [(-7, -6), (-8, -4), (-30, 20)])
@pytest.mark.parametrize("case", range(len(COMPACT)))
def test_compact_matches_the_definition(case, exps):
    ql, L, keeps, Hkv, D = COMPACT[case]
    step = base.Step(ql, L, seed=case)
    bufs = base._pool(step, Hkv, D, seed=case, exps=exps)
    base._stale(step, bufs[0])
    cache = base._cache(bufs, 2 * Hkv, Hkv, D)
    ws = cache.new_workspace()
    keep, n_keep = _table(keeps)
    q_off, kv_len, pages = step.dev()
    before = kv_len.clone()
    out = cache.compact(keep, n_keep, q_off, kv_len, pages, ws, max_q=step.max_q)
    assert cache.check(ws) == 0 and torch.equal(kv_len, before)
    *want, lens = spec.compact(bufs, step.pages, step.q_off.tolist(), L, keeps, [len(k) for k in keeps])
    assert out.tolist() == lens
    assert _same(_values(cache), want)


def test_compact_keeps_bits_where_the_scale_stays():
    """A token's NaN key codes and -0 move as they are."""
    Hkv, D = 2, 128
    step = base.Step([10], [74], seed=1)
    bufs = base._pool(step, Hkv, D, seed=1, exps=(-6, -5))
    page = int(step.pages[0, 1])
    bufs[0][page, :, 7] = 0xFF
    bufs[0][page, :, 8, :64] = 0x80
    bufs[1][page, :, :, 8] = 0x80
    cache = base._cache(bufs, 2, Hkv, D)
    ws = cache.new_workspace()
    keep, n_keep = _table([[0, 7, 8]])
    out = cache.compact(keep, n_keep, *step.dev(), ws, max_q=10)
    assert out.tolist() == [67]
    k, v = cache.k.cpu(), cache.v.cpu()
    assert torch.equal(k[page, :, 1:3], bufs[0][page, :, 7:9]) and torch.equal(v[page, :, :, 1:3], bufs[1][page, :, :, 7:9])
    assert torch.equal(k[page, :, 3:], bufs[0][page, :, 3:]) and torch.equal(v[page, :, :, 3:], bufs[1][page, :, :, 3:])


@pytest.mark.parametrize("scales", ["odd", "zero"])
def test_compact_scales_that_are_no_powers_of_two_or_none(scales):
    step = base.Step([70], [130], seed=2)
    bufs = list(base._pool(step, 2, 64, seed=2))
    g = torch.Generator().manual_seed(3)
    bufs[2], bufs[3] = (2.0 ** (-8 + 3 * torch.rand(bufs[2].shape, generator=g)) for _ in range(2))
    if scales == "zero":  # a page that was never written: its codes move as they are
        bufs[2][step.pages[0, 2].long()] = 0
        bufs[3][step.pages[0, 2].long()] = 0
    cache = base._cache(bufs, 2, 2, 64)
    ws = cache.new_workspace()
    keep, n_keep = _table([[0, 30, 68, 69]])   # positions 60, 90, 128, 129
    cache.compact(keep, n_keep, *step.dev(), ws, max_q=70)
    assert cache.check(ws) == 0
    got = _values(cache)
    assert not bool(got[1].isnan().any())
    if scales == "odd":  # a product rounded to fp32 before E4M3: within half a step and 2^-24
        *want, _ = spec.compact(bufs, step.pages, [0, 70], [130], [[0, 30, 68, 69]], [4])
        assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
        for a, b in zip(got[:2], want[:2]):
            assert float((a != b).double().mean()) < 1e-3
            assert bool(((a - b).abs() <= 2 * ref.half_step(b) * (1 + 2.0 ** -20)).all())


def test_compact_bad_sequences_are_left_and_flagged():
    ql, L, Hkv, D = [6, 6, 6], [70, 130, 66], 2, 64
    step = base.Step(ql, L, seed=3)
    bufs = base._pool(step, Hkv, D, seed=3)
    keeps = [[0, 2, 5], [1, 3], [2]]
    keep, n_keep = _table(keeps)
    q_off, kv_len, pages = step.dev()
    good = base._cache(bufs, 2, Hkv, D)
    ws = good.new_workspace()
    good.compact(keep, n_keep, q_off, kv_len, pages, ws, max_q=6)
    assert good.check(ws) == 0
    mine = [step.pages[b, :(n + 63) // 64].long() for b, n in enumerate(L)]

    def run(keep=keep, n_keep=n_keep, q_off=q_off, kv_len=kv_len, pages=pages, lens=(67, 130, 61)):
        cache = base._cache(bufs, 2, Hkv, D)
        out = cache.compact(keep, n_keep, q_off, kv_len, pages, ws, max_q=6)
        assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX and cache.check(ws) == 0
        assert out.tolist() == list(lens)
        for b in (0, 2):
            assert torch.equal(cache.k[mine[b]], good.k[mine[b]]) and torch.equal(cache.v[mine[b]], good.v[mine[b]])
        assert torch.equal(cache.k[mine[1]].cpu(), bufs[0][mine[1]]) and torch.equal(cache.v[mine[1]].cpu(), bufs[1][mine[1]])
        assert torch.equal(cache.k_scale[mine[1]].cpu(), bufs[2][mine[1]])

    for row in ([3, 1], [1, 1], [-1, 2], [0, 6], [0, 2 ** 31 - 1]):
        k = keep.clone()
        k[1, :2] = i32(*row)
        run(keep=k)
    for m in (-1, 4, 7, 2 ** 31 - 1):
        run(n_keep=i32(3, m, 1))
    for n in (-3, 10 ** 9, 5):
        run(kv_len=i32(70, n, 66), lens=(67, n, 61))
    for bad in (-1, step.n_pages, 2 ** 31 - 1):
        p = pages.clone()
        p[1, 1] = bad                 # positions 124 ..: the page that the kept ones come from and go to
        run(pages=p)


def test_compact_long_steps_are_refused_on_the_device():
    step = base.Step([300, 4], [300, 70], seed=4)
    bufs = base._pool(step, 1, 64, seed=4)
    cache = base._cache(bufs, 1, 1, 64)
    ws = cache.new_workspace()
    out = cache.compact(i32(5, 6).view(2, 1), i32(1, 0), *step.dev(), ws, max_q=4)
    assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX
    assert out.tolist() == [300, 66] and torch.equal(cache.k.cpu(), bufs[0])


def test_compact_streams_and_graphs():
    """A captured compaction of what a step appends, replayed."""
    step = base.Step([12, 3], [100, 67], seed=5)
    bufs = base._pool(step, 2, 128, seed=5)
    keeps = [[0, 4, 11], [1]]
    keep, n_keep = _table(keeps)
    *want, lens = spec.compact(bufs, step.pages, step.q_off.tolist(), step.L, keeps, [3, 1])
    cache = base._cache(bufs, 2, 2, 128)
    ws = cache.new_workspace()
    args = step.dev()
    start = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    out = torch.zeros(2, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.compact(keep, n_keep, *args, ws, max_q=12, kv_len_out=out)
    for stream in (None, torch.cuda.Stream()):
        for t, s in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), start):
            t.copy_(s)
        torch.cuda.synchronize()
        if stream is None:
            g.replay()
        else:
            cache.compact(keep, n_keep, *args, ws, max_q=12, kv_len_out=out, stream=stream)
        torch.cuda.synchronize()
        assert out.tolist() == lens and _same(_values(cache), want)


# ----------------------------------------------------------------------------- fork
def _pool_of(L, Hkv, D, C, seed):
    step = base.Step([0] * len(L), L, seed=seed, spare=C + 2, max_pages=max((n + 63) // 64 for n in L) + 1)
    bufs = base._pool(step, Hkv, D, seed=seed)
    used = set(step.pages.flatten().tolist())
    free = [p for p in range(step.n_pages) if p not in used]
    return step, bufs, free


FORK = [
    # L, src, which children get a page, Hkv, D
    ([1], [0], [True], 1, 64), ([100], [0, 0, 0], [False, True, True], 8, 128), ([64, 70], [1, 0, 1], [True, True, False], 2, 64),
    ([128, 1, 63], [2, 2, 1, 0, 0], [True] * 5, 4, 128), ([0, 5], [0, 0, 1], [True, True, True], 2, 128),
    ([300] * 40, [i // 3 for i in range(100)], [i % 3 > 0 for i in range(100)], 2, 64),
]


@pytest.mark.parametrize("case", range(len(FORK)))
def test_fork_matches_the_definition(case):
    L, src, own, Hkv, D = FORK[case]
    step, bufs, free = _pool_of(L, Hkv, D, len(src), case)
    cache = base._cache(bufs, Hkv, Hkv, D)
    ws = cache.new_workspace()
    fresh = [free[c] if o else -1 for c, o in enumerate(own)]
    _, kv_len, pages = step.dev()
    p, n = cache.fork(i32(*src), i32(*fresh), kv_len, pages, ws)
    assert cache.check(ws) == 0
    k, v, ks, vs = (t.clone() for t in bufs)
    want = step.pages[torch.tensor(src)].clone()
    for c, (s, f) in enumerate(zip(src, fresh)):
        if f >= 0:
            if L[s] % PAGE:
                for t in (k, v, ks, vs):
                    t[f] = t[int(step.pages[s, L[s] // PAGE])]
            want[c, L[s] // PAGE] = f
    assert torch.equal(p.cpu(), want) and n.tolist() == [L[s] for s in src]
    for a, b in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), (k, v, ks, vs)):
        assert torch.equal(a.cpu(), b)


def test_fork_of_a_full_table_and_of_nothing():
    step, bufs, free = _pool_of([128], 2, 64, 2, 1)
    cache = base._cache(bufs, 2, 2, 64)
    ws = cache.new_workspace()
    pages = step.dev()[2][:, :2].contiguous()
    p, n = cache.fork(i32(0), i32(free[0]), i32(128), pages, ws)     # no place for a next token
    assert cache.check(ws) == 0 and torch.equal(p, pages) and n.tolist() == [128] and torch.equal(cache.k.cpu(), bufs[0])
    p, n = cache.fork(i32(), i32(), i32(128), pages, ws)
    assert p.shape == (0, 2) and n.shape == (0,)


def test_fork_bad_children_are_flagged_and_empty():
    L = [100, 30]
    step, bufs, free = _pool_of(L, 2, 64, 4, 2)
    _, kv_len, pages = step.dev()
    ws = base._cache(bufs, 2, 2, 64).new_workspace()

    def run(src, fresh, bad, kv_len=kv_len, pages=pages):
        cache = base._cache(bufs, 2, 2, 64)
        p, n = cache.fork(i32(*src), i32(*fresh), kv_len, pages, ws)
        assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX and cache.check(ws) == 0
        for c in range(len(src)):
            if c in bad:
                assert bool((p[c] == -1).all()) and int(n[c]) == 0
            else:
                assert int(n[c]) == L[src[c]] and int(p[c, L[src[c]] // PAGE]) == fresh[c]
                tail = int(step.pages[src[c], L[src[c]] // PAGE])
                assert torch.equal(cache.k[fresh[c]].cpu(), bufs[0][tail])

    for s in (-1, 2, 2 ** 31 - 1):
        run([0, s], free[:2], {1})
    run([0, 1], [free[0], step.n_pages], {1})
    run([0, 1, 0], [free[0], free[1], free[0]], {2})              # a page given twice: to the first
    for n in (-1, 10 ** 9):
        run([1, 0, 1], free[:3], {1}, kv_len=i32(n, 30))
    for page in (-1, step.n_pages):
        p = pages.clone()
        p[0, 1] = page
        run([1, 0], free[:2], {1}, pages=p)


def test_fork_children_go_on_alone():
    """Children of one prompt append different tokens: each attends to its own."""
    Hq, Hkv, D, L, C = 4, 2, 128, 100, 3
    step, bufs, free = _pool_of([L], Hkv, D, C, 3)
    cache = base._cache(bufs, Hq, Hkv, D)
    ws = cache.new_workspace()
    pages, kv_len = cache.fork(i32(0, 0, 0), i32(-1, free[0], free[1]), i32(L), step.dev()[2], ws)
    qkv = torch.randn((C, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    q, k, v = qkv.split((Hq, Hkv, Hkv), dim=1)
    q_off = i32(0, 1, 2, 3)
    cache.append(k, v, q_off, kv_len + 1, pages, ws, max_q=1)
    out = cache.attend(q, q_off, kv_len + 1, pages, ws, max_q=1)
    assert cache.check(ws) == 0
    for c in range(C):
        alone = base._cache(bufs, Hq, Hkv, D)
        one = (i32(0, 1), i32(L + 1), step.dev()[2], ws)
        alone.append(k[c:c + 1], v[c:c + 1], *one, max_q=1)
        assert torch.equal(alone.attend(q[c:c + 1], *one, max_q=1)[0], out[c])


def test_moves_in_a_pool_past_32_bit_offsets():
    Hkv, D, base_page = 8, 128, 66000
    small = base.Step([9], [70], seed=8)
    bufs = base._pool(small, Hkv, D, seed=8)
    n = small.n_pages + base_page
    big = dict(k=torch.empty((n, Hkv, PAGE, D), dtype=torch.uint8, device=DEV),
               v=torch.empty((n, Hkv, D, PAGE), dtype=torch.uint8, device=DEV),
               k_scale=torch.empty((n, Hkv), dtype=torch.float32, device=DEV),
               v_scale=torch.empty((n, Hkv), dtype=torch.float32, device=DEV))
    assert big["k"].numel() > 2 ** 32
    for name, t in zip(("k", "v", "k_scale", "v_scale"), bufs):
        big[name][base_page:] = t.to(DEV)
    keep, n_keep = _table([[0, 5, 8]])
    used = small.pages[0].tolist()
    free = next(p for p in range(small.n_pages) if p not in used)
    res = []
    for cache, shift in ((KVCache(n, Hkv, Hkv, D, buffers=big), base_page), (base._cache(bufs, Hkv, Hkv, D), 0)):
        ws = cache.new_workspace()
        q_off, kv_len, pages = small.dev()
        lens = cache.compact(keep, n_keep, q_off, kv_len, pages + shift, ws, max_q=9)
        p, _ = cache.fork(i32(0), i32(free + shift), lens, pages + shift, ws)
        assert cache.check(ws) == 0
        res.append((p - shift, lens))
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert torch.equal(big["k"][base_page:], cache.k) and torch.equal(big["v"][base_page:], cache.v)


def test_refusals():
    cache = KVCache(4, 4, 2, 64)
    ws = cache.new_workspace()
    pages = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
    step = (i32(0, 2), i32(2), pages, ws)
    both = i32(2, 0)
    inv = binding.MOE_ERR_INVALID_ARG
    cases = [
        lambda: cache.compact(i32(0), i32(1), *step, max_q=2), lambda: cache.compact(i32(0, 1).view(2, 1), i32(1), *step, max_q=2),
        lambda: cache.compact(i32(0).view(1, 1), i32(1, 1), *step, max_q=2),
        lambda: cache.compact(i32(0).view(1, 1).long(), i32(1), *step, max_q=2),
        lambda: cache.compact(i32(0).view(1, 1), i32(1).cpu(), *step, max_q=2),
        lambda: cache.compact(torch.zeros((1, 257), dtype=torch.int32, device=DEV), i32(1), *step, max_q=2),
        lambda: cache.compact(i32(0).view(1, 1), i32(1), *step, max_q=2, kv_len_out=step[1]),
        lambda: cache.compact(i32(0).view(1, 1), i32(1), *step, max_q=2, kv_len_out=i32(0, 0)),
        lambda: cache.compact(i32(0).view(1, 1), i32(1), *step[:3], ws[:256], max_q=2),
        lambda: cache.fork(i32(0), i32(1, 2), i32(2), pages, ws), lambda: cache.fork(i32(0).view(1, 1), i32(1), i32(2), pages, ws),
        lambda: cache.fork(i32(0), i32(1), i32(2, 2), pages, ws), lambda: cache.fork(i32(0), i32(1), i32(2), pages.long(), ws),
        lambda: cache.fork(i32(0), i32(1), i32(2), pages, ws, pages_out=pages),
        lambda: cache.fork(i32(0), i32(1), both[:1], pages, ws, kv_len_out=both[:1]),
        lambda: cache.fork(i32(0), i32(1), i32(2), pages, ws, pages_out=pages.repeat(2, 1)),
        lambda: cache.fork(i32(0), i32(1), i32(2), pages[:, :0], ws), lambda: cache.fork(i32(0), i32(1), i32(), pages[:0], ws),
        lambda: cache.fork(torch.zeros(513, dtype=torch.int32, device=DEV), torch.zeros(513, dtype=torch.int32, device=DEV), i32(2),
                           pages, ws),
    ]
    for i, call in enumerate(cases):
        with pytest.raises(MoeError) as ei:
            call()
        assert ei.value.status == inv, i
    assert cache.check(ws) == 0
