"""moe_kv_append and moe_kv_attend against their 64-bit definitions.

append: value codes and scales are exact (values are not rotated).  Keys and
queries are rotated in fp32: three roundings, under 2^-22 (|a| + |b|) for pair
(a, b), then half an E4M3 step (a code) or half a bf16 step (a query).

attend: the output is rounded to bf16 (2^-8 relative).  Before that a weight is
off by 2^-9 (two E4M3 digits), by its score's error ds (relative), and by 2^-18
of the row's largest weight x v (the digits' smallest step).  ds: products of
fp32 sums, 2^-20 of the sum of magnitudes, and what q's digits leave out, 2^-18
of q's largest a product.  So, with A = sum w |v| / sum w, n visible tokens, ln
the weights' sum over the largest weight and vmax the largest visible |v|:
    |error| <= 2^-8 |o| + (2^-9 + 2 ds) A + 2^-18 n vmax / ln
"""
import math

import pytest
import torch

import layer_reference as ref
from quantized_moe_routed_gb300 import KVCache, MoeError, binding, rope_table

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 64


class Step:
    """Sequences with ql new tokens and lengths L, their pages shuffled over a pool."""

    def __init__(self, ql, L, seed=0, spare=3, max_pages=None, base=0):
        self.ql, self.L, self.N = ql, L, sum(ql)
        g = torch.Generator().manual_seed(seed)
        need = [max(0, (n + PAGE - 1) // PAGE) for n in L]
        self.n_pages = sum(need) + spare + base
        perm = torch.randperm(sum(need) + spare, generator=g) + base
        width = max_pages or max(need + [1])
        self.pages = torch.full((len(ql), width), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.pages[b, :m] = perm[at:at + m]
            at += m
        off = [0]
        for n in ql:
            off.append(off[-1] + n)
        self.q_off = torch.tensor(off, dtype=torch.int32)
        self.kv_len = torch.tensor(L, dtype=torch.int32)
        self.max_q = max(ql)

    def dev(self):
        return self.q_off.to(DEV), self.kv_len.to(DEV), self.pages.to(DEV)


def _pool(step, Hkv, D, seed, exps=(-8, -4)):
    """Random codes everywhere (no NaN in v; k's unused slots hold NaN codes)."""
    g = torch.Generator().manual_seed(seed)
    k = (torch.randn((step.n_pages, Hkv, PAGE, D), generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    v = (torch.randn((step.n_pages, Hkv, D, PAGE), generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    ks = 2.0 ** torch.randint(exps[0], exps[1], (step.n_pages, Hkv), generator=g).float()
    vs = 2.0 ** torch.randint(exps[0], exps[1], (step.n_pages, Hkv), generator=g).float()
    return k, v, ks, vs


def _stale(step, k):
    """NaN codes in the slots of k past each sequence's length, and in spare pages."""
    used = torch.zeros((k.shape[0], PAGE), dtype=torch.bool)
    for b, n in enumerate(step.L):
        for t in range(n):
            used[step.pages[b, t // PAGE], t % PAGE] = True
    k[~used[:, None, :].expand(-1, k.shape[1], -1)] = 0x7F


def _cache(bufs, Hq, Hkv, D, rope=None, inter=False):
    k, v, ks, vs = (t.to(DEV) for t in bufs)
    return KVCache(k.shape[0], Hq, Hkv, D, rope=rope, interleaved=inter,
                   buffers=dict(k=k, v=v, k_scale=ks, v_scale=vs))


def _gather(step, bufs, b, h):
    """Sequence b's keys and values of kv head h, float64 [L, D]."""
    k, v, ks, vs = bufs
    L = step.L[b]
    ids = step.pages[b, :(L + PAGE - 1) // PAGE].long()
    kk = ref.e4m3(k[ids, h]) * ks[ids, h].double()[:, None, None]
    vv = (ref.e4m3(v[ids, h]) * vs[ids, h].double()[:, None, None]).transpose(1, 2)
    return kk.reshape(-1, k.shape[3])[:L], vv.reshape(-1, k.shape[3])[:L]


def _check_attend(step, bufs, q, out, scale, skip=()):
    Hq, D = q.shape[1:]
    Hkv = bufs[0].shape[1]
    G = Hq // Hkv
    out = out.cpu().double()
    for b, (n, L) in enumerate(zip(step.ql, step.L)):
        if n == 0 or b in skip:
            continue
        r0 = int(step.q_off[b])
        for h in range(Hkv):
            k, v = _gather(step, bufs, b, h)
            qq = q[r0:r0 + n, h * G:(h + 1) * G]
            want, A, ln, vm = ref.attend(qq, k, v, n, L, scale)
            ka = k.abs().amax(0) if L else torch.zeros(D, dtype=torch.float64)
            mag = (qq.double().abs() * ka).sum(-1)
            ds = abs(scale) * (2.0 ** -20 * mag + 2.0 ** -18 * qq.double().abs().amax(-1) * ka.sum())
            seen = torch.clamp(L - n + torch.arange(n).double() + 1, 0, L)[:, None]
            tol = (2.0 ** -8 * want.abs() + (2.0 ** -9 + 2 * ds)[..., None] * A +
                   (2.0 ** -18 * seen * vm / ln)[..., None] + 1e-37)
            err = (out[r0:r0 + n, h * G:(h + 1) * G] - want).abs()
            assert bool((err <= tol).all()), (b, h, float((err / tol).max()))


ATTEND = [
    # ql, L, Hq, Hkv, D
    ([1], [1], 1, 1, 64), ([1], [64], 4, 2, 128), ([1], [65], 8, 1, 128), ([1], [4000], 8, 2, 128),
    ([1, 1, 1, 1], [1, 63, 128, 700], 24, 8, 64), ([1, 0, 1], [129, 77, 2], 12, 4, 128),
    ([1] * 9, [130, 1, 64, 65, 200, 3, 127, 511, 90], 16, 1, 128), ([1], [300], 32, 1, 64),
    ([1], [300], 33, 1, 128), ([3], [3], 8, 8, 128), ([3, 1, 2], [3, 70, 200], 8, 8, 64),
    ([5, 2], [64, 66], 16, 4, 128), ([16, 16], [400, 16], 8, 2, 128), ([16, 7], [300, 90], 8, 2, 64),
    ([33], [40], 4, 4, 128), ([130], [130], 4, 1, 128), ([100, 1, 0, 64], [250, 900, 5, 64], 12, 4, 64),
    ([70, 3], [500, 80], 20, 4, 128), ([300], [301], 2, 1, 128),
]


@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend_matches_the_definition(case):
    ql, L, Hq, Hkv, D = ATTEND[case]
    step = Step(ql, L, seed=case)
    bufs = _pool(step, Hkv, D, seed=case)
    _stale(step, bufs[0])
    q = torch.randn((step.N, Hq, D), generator=torch.Generator().manual_seed(case)).bfloat16()
    cache = _cache(bufs, Hq, Hkv, D)
    ws = cache.new_workspace()
    out = cache.attend(q.to(DEV), *step.dev(), ws, max_q=step.max_q)
    assert cache.check(ws) == 0
    _check_attend(step, bufs, q, out, 1 / math.sqrt(D))
    again = cache.attend(q.to(DEV), *step.dev(), ws, max_q=step.max_q)
    assert torch.equal(out, again)


@pytest.mark.parametrize("max_q", [1, 3, 8, 40, 60])
def test_attend_tiles_do_not_change_the_answer(max_q):
    """max_q only chooses tiles: every choice covers every row."""
    ql, L, Hq, Hkv, D = [60, 1, 9], [200, 333, 9], 8, 2, 128
    step = Step(ql, L, seed=1)
    bufs = _pool(step, Hkv, D, seed=1)
    q = torch.randn((step.N, Hq, D), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache = _cache(bufs, Hq, Hkv, D)
    ws = cache.new_workspace()
    out = cache.attend(q.to(DEV), *step.dev(), ws, max_q=max_q)
    _check_attend(step, bufs, q, out, 1 / math.sqrt(D))


@pytest.mark.parametrize("n,Hq", [(1, 8), (9, 8), (40, 8)])
def test_attend_rows_that_see_nothing_are_zero(n, Hq):
    """Lengths of zero, and more new tokens than the sequence holds."""
    step = Step([n, n, n], [0, max(n - 3, 0), 64], seed=2)
    bufs = _pool(step, 2, 128, seed=2)
    q = torch.randn((step.N, Hq, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache = _cache(bufs, Hq, 2, 128)
    ws = cache.new_workspace()
    out = torch.full((step.N, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    cache.attend(q.to(DEV), *step.dev(), ws, max_q=n, out=out)
    assert bool((out[:n] == 0).all())
    _check_attend(step, bufs, q, out, 1 / math.sqrt(128))


@pytest.mark.parametrize("n", [1, 9, 40, 70])
@pytest.mark.parametrize("scale", [0.0, -0.1, 1.5])
def test_attend_softmax_scale(n, scale):
    """No scale at all (equal weights), a negative one, one that leaves a few weights."""
    step = Step([n, n], [200, n], seed=12)
    bufs = _pool(step, 2, 128, seed=12)
    _stale(step, bufs[0])
    q = torch.randn((2 * n, 8, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache = _cache(bufs, 8, 2, 128)
    ws = cache.new_workspace()
    out = cache.attend(q.to(DEV), *step.dev(), ws, max_q=n, scale=scale)
    _check_attend(step, bufs, q, out, scale)


@pytest.mark.parametrize("n", [1, 6, 40])
def test_attend_scales_of_very_different_size(n):
    """Pages whose v differ by 2^50, scores up to large ones, a custom scale."""
    step = Step([n], [900], seed=3)
    bufs = _pool(step, 2, 128, seed=3, exps=(-30, 20))
    bufs[2].fill_(2.0 ** -7)
    q = (torch.randn((n, 4, 128), generator=torch.Generator().manual_seed(1)) * 3).bfloat16()
    q[0, 0] *= 1e-30
    q[0, 1] = 0
    cache = _cache(bufs, 4, 2, 128)
    ws = cache.new_workspace()
    for scale in (0.05, 0.3):
        out = cache.attend(q.to(DEV), *step.dev(), ws, max_q=n, scale=scale)
        _check_attend(step, bufs, q, out, scale)


@pytest.mark.parametrize("n", [1, 20])
def test_attend_scales_that_are_no_powers_of_two(n):
    step = Step([n], [500], seed=4)
    bufs = list(_pool(step, 2, 64, seed=4))
    g = torch.Generator().manual_seed(9)
    bufs[2], bufs[3] = (2.0 ** (-8 + 3 * torch.rand(bufs[2].shape, generator=g)) for _ in range(2))
    q = torch.randn((n, 6, 64), generator=g).bfloat16()
    cache = _cache(bufs, 6, 2, 64)
    ws = cache.new_workspace()
    out = cache.attend(q.to(DEV), *step.dev(), ws, max_q=n)
    _check_attend(step, bufs, q, out, 1 / 8)


@pytest.mark.parametrize("n", [1, 12])
def test_attend_nan_and_infinite_queries_stay_in_their_row(n):
    step = Step([n], [100], seed=5)
    bufs = _pool(step, 1, 128, seed=5)
    q = torch.randn((n, 8, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    clean = q.clone()
    q[0, 3, 5], q[0, 4, 6] = float("nan"), float("inf")
    cache = _cache(bufs, 8, 1, 128)
    ws = cache.new_workspace()
    out = cache.attend(q.to(DEV), *step.dev(), ws, max_q=n)
    assert bool(out[0, 3:5].isnan().all())
    out[0, 3:5] = cache.attend(clean.to(DEV), *step.dev(), ws, max_q=n)[0, 3:5]
    _check_attend(step, bufs, clean, out, 1 / math.sqrt(128))


def test_attend_bad_pages_lengths_and_offsets_are_flagged():
    ql, L = [1, 1, 1], [130, 200, 70]
    step = Step(ql, L, seed=6)
    bufs = _pool(step, 2, 128, seed=6)
    q = torch.randn((3, 4, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache = _cache(bufs, 4, 2, 128)
    ws = cache.new_workspace()
    q_off, kv_len, pages = step.dev()
    for bad in (-1, step.n_pages, 2 ** 30):
        p = pages.clone()
        p[1, 1] = bad
        out = cache.attend(q.to(DEV), q_off, kv_len, p, ws, max_q=1)
        assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX and cache.check(ws) == 0
        _check_attend(step, bufs, q, out, 1 / math.sqrt(128), skip=(1,))
        assert bool(out[1].isfinite().all())
    for lens in ([130, -4, 70], [130, 2 ** 31 - 1, 70]):
        out = cache.attend(q.to(DEV), q_off, torch.tensor(lens, dtype=torch.int32, device=DEV), pages, ws, max_q=1)
        assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX
        _check_attend(step, bufs, q, out, 1 / math.sqrt(128), skip=(1,))
        assert bool((out[1] == 0).all())
    for off in ([0, 1, 2, 9], [0, 1, 0, 3], [-5, 1, 2, 3]):
        cache.attend(q.to(DEV), torch.tensor(off, dtype=torch.int32, device=DEV), kv_len, pages, ws, max_q=1)
        assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX
    out = cache.attend(q.to(DEV), q_off, kv_len, pages, ws, max_q=1)
    assert cache.check(ws) == 0
    _check_attend(step, bufs, q, out, 1 / math.sqrt(128))


def test_attend_strided_queries_streams_and_graphs():
    step = Step([1, 4], [500, 60], seed=7)
    bufs = _pool(step, 2, 128, seed=7)
    qkv = torch.randn((5, 12, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache = _cache(bufs, 8, 2, 128)
    ws = cache.new_workspace()
    args = step.dev()
    qd = qkv.to(DEV)
    torch.cuda.synchronize()
    first = cache.attend(qd[:, :8], *args, ws, max_q=4)
    _check_attend(step, bufs, qkv[:, :8], first, 1 / math.sqrt(128))
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [cache.attend(qd[:, :8], *args, ws, max_q=4, stream=streams[i % 3]) for i in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    out = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attend(qd[:, :8], *args, ws, max_q=4, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)


def test_attend_and_append_in_a_pool_past_32_bit_offsets():
    """Pages whose codes lie past 2^32 bytes of the pool."""
    Hkv, D = 8, 128
    step = Step([2, 1], [130, 65], seed=8, base=66000)
    small = Step([2, 1], [130, 65], seed=8)
    bufs = _pool(small, Hkv, D, seed=8)
    q = torch.randn((3, 16, D), generator=torch.Generator().manual_seed(1)).bfloat16()
    kv = torch.randn((3, 2 * Hkv, D), generator=torch.Generator().manual_seed(2)).bfloat16()
    n = step.n_pages
    big = dict(k=torch.empty((n, Hkv, PAGE, D), dtype=torch.uint8, device=DEV),
               v=torch.empty((n, Hkv, D, PAGE), dtype=torch.uint8, device=DEV),
               k_scale=torch.empty((n, Hkv), dtype=torch.float32, device=DEV),
               v_scale=torch.empty((n, Hkv), dtype=torch.float32, device=DEV))
    assert big["k"].numel() > 2 ** 32
    for name, t in zip(("k", "v", "k_scale", "v_scale"), bufs):
        big[name][66000:] = t.to(DEV)
    a, b = KVCache(n, 16, Hkv, D, buffers=big), _cache(bufs, 16, Hkv, D)
    res = []
    for cache, st in ((a, step), (b, small)):
        ws = cache.new_workspace()
        kvd = kv.to(DEV)
        cache.append(kvd[:, :Hkv], kvd[:, Hkv:], *st.dev(), ws, max_q=2)
        res.append(cache.attend(q.to(DEV), *st.dev(), ws, max_q=2))
        assert cache.check(ws) == 0
    assert torch.equal(*res)
    assert torch.equal(a.k[66000:], b.k) and torch.equal(a.v[66000:], b.v)


# ----------------------------------------------------------------------------- append
def _ref_append(step, bufs, k, v, rope, inter):
    """The definition: new codes' values (float64), scales; requantises pages."""
    kv, vv = ref.e4m3(bufs[0]), ref.e4m3(bufs[1])
    ks, vs = bufs[2].double(), bufs[3].double()
    new = torch.zeros((step.n_pages, PAGE), dtype=torch.bool)
    slack = torch.zeros_like(kv)     # what fp32 may move a key by
    for b, (n, L) in enumerate(zip(step.ql, step.L)):
        r0 = int(step.q_off[b])
        pos = torch.arange(L - n, L)
        kr = k[r0:r0 + n].double()
        mag = torch.zeros_like(kr)
        if rope is not None and n:
            mag = (kr.abs() + kr.abs().amax(-1, keepdim=True)) * 2.0 ** -22 * rope[pos].abs().max()
            kr = ref.rotate(kr, rope[pos], inter)
        i = 0
        while i < n:
            p = L - n + i
            page, o = int(step.pages[b, p // PAGE]), p % PAGE
            m = min(PAGE - o, n - i)
            for src, val, sc in ((kr, kv[page], ks[page]), (v[r0:r0 + n].double(), vv[page].transpose(1, 2), vs[page])):
                x = src[i:i + m].transpose(0, 1)
                want = ref.pow2_scale(x.abs().amax((1, 2)))
                if o:
                    want = torch.maximum(want, sc)
                    val.copy_(ref.to_e4m3(val * (sc / want)[:, None, None]))
                sc.copy_(want)
                val[:, o:o + m] = (x if src is kr else ref.to_e4m3(x / want[:, None, None]) * want[:, None, None]) / want[:, None, None]
                if src is kr:
                    slack[page][:, o:o + m] = mag[i:i + m].transpose(0, 1) / want[:, None, None]
            new[page, o:o + m] = True
            i += m
    return kv, vv, ks, vs, new, slack


APPEND = [
    # ql, L, Hq, Hkv, D, R, interleaved
    ([1], [1], 4, 2, 128, 128, False), ([1, 1, 1], [64, 65, 200], 8, 8, 64, 64, True),
    ([1, 0, 2], [33, 5, 128], 12, 4, 128, 64, False), ([64], [64], 2, 1, 128, 0, False),
    ([100, 3], [100, 66], 8, 2, 128, 128, True), ([130, 1], [333, 1], 6, 2, 64, 6, False),
    ([63, 65, 17], [70, 65, 100], 4, 4, 64, 50, True), ([300], [1000], 2, 1, 128, 2, False),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
@pytest.mark.parametrize("gain", [0.01, 1.0, 300.0])
def test_append_matches_the_definition(case, gain):
    ql, L, Hq, Hkv, D, R, inter = APPEND[case]
    step = Step(ql, L, seed=case)
    bufs = _pool(step, Hkv, D, seed=case, exps=(-8, -6))
    g = torch.Generator().manual_seed(case)
    qkv = (torch.randn((step.N, Hq + 2 * Hkv, D), generator=g) * gain).bfloat16()
    rope = rope_table(max(L), R, device="cpu", magnitude=1.1) if R else None
    cache = _cache(bufs, Hq, Hkv, D, rope=None if rope is None else rope.to(DEV), inter=inter)
    ws = cache.new_workspace()
    q, k, v = qkv.to(DEV).split((Hq, Hkv, Hkv), dim=1)
    q_out = cache.append(k, v, *step.dev(), ws, max_q=step.max_q, q=q)
    assert cache.check(ws) == 0
    kv, vv, ks, vs, new, slack = _ref_append(step, bufs, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], rope, inter)
    assert torch.equal(cache.k_scale.cpu().double(), ks) and torch.equal(cache.v_scale.cpu().double(), vs)
    got_v = ref.e4m3(cache.v.cpu())
    assert torch.equal(got_v, vv)
    got_k = ref.e4m3(cache.k.cpu())
    live = new[:, None, :, None].expand_as(got_k)
    assert torch.equal(got_k[~live], kv[~live])
    tol = ref.half_step(kv) * (1 + 2.0 ** -10) + slack
    assert bool(((got_k - kv).abs() <= tol)[live].all())
    pos = torch.cat([torch.arange(b - n, b) for n, b in zip(ql, L)])
    qr = qkv[:, :Hq].double()
    want = ref.rotate(qr, rope[pos], inter) if R else qr
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -22 * 2.2 * qr.abs().amax(-1, keepdim=True) if R else 0)
    assert bool(((q_out.cpu().double() - want).abs() <= tol).all())
    # appending the same tokens again changes nothing, and keys alone need no queries
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    assert cache.append(k, v, *step.dev(), ws, max_q=1) is None
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)))


def test_append_token_by_token_equals_one_chunk_of_values():
    """Codes shift exactly when the scale grows, so single appends end at the
    chunk's scales, and at its codes wherever E4M3's exponent range is kept."""
    n, Hkv, D = 64, 2, 128
    g = torch.Generator().manual_seed(3)
    kv = torch.randn((n, 2 * Hkv, D), generator=g).bfloat16()
    kv = kv * (2.0 ** (torch.arange(n) // 16))[:, None, None]       # growing: the scale moves three times
    kv = kv.bfloat16().to(DEV)
    chunk, single = KVCache(1, Hkv, Hkv, D), KVCache(1, Hkv, Hkv, D)
    ws = chunk.new_workspace()
    pages = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    chunk.append(kv[:, :Hkv], kv[:, Hkv:], i32(0, n), i32(n), pages, ws, max_q=n)
    for t in range(n):
        x = kv[t:t + 1]
        single.append(x[:, :Hkv], x[:, Hkv:], i32(0, 1), i32(t + 1), pages, ws, max_q=1)
    assert chunk.check(ws) == 0
    for a, b, s in ((chunk.k, single.k, "k_scale"), (chunk.v, single.v, "v_scale")):
        assert torch.equal(getattr(chunk, s), getattr(single, s))
        va, vb = ref.e4m3(a.cpu()), ref.e4m3(b.cpu())
        normal = va.abs() >= 2.0 ** -6
        assert torch.equal(va[normal], vb[normal])
        assert bool(((va - vb).abs() <= 2.0 ** -9)[~normal].all())


@pytest.mark.parametrize("n", [1, 20])
def test_append_nan_and_infinity_poison_only_who_attends_to_them(n):
    """A NaN value and an infinite key: outputs of earlier tokens and of other kv
    heads are untouched, those that see the token are NaN, no v code is NaN."""
    Hkv, D, L = 2, 128, 90
    step = Step([n], [L], seed=1)
    bufs = _pool(step, Hkv, D, seed=1)
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn((n, 3 * Hkv, D), generator=g).bfloat16()
    dirty = qkv.clone()
    at = n // 2
    dirty[at, 2 * Hkv, 5] = float("nan")
    if n > 1:
        dirty[at + 3, Hkv, 7] = float("inf")
    outs = []
    for x in (qkv, dirty):
        cache = _cache(bufs, Hkv, Hkv, D)
        ws = cache.new_workspace()
        q, k, v = x.to(DEV).split((Hkv,) * 3, dim=1)
        cache.append(k, v, *step.dev(), ws, max_q=n)
        outs.append(cache.attend(q, *step.dev(), ws, max_q=n))
        assert cache.check(ws) == 0
        assert bool((cache.v & 127 != 127).all())
    assert bool(outs[1][at:, 0].isnan().all())
    assert torch.equal(outs[0][:, 1], outs[1][:, 1])
    if n > 1:
        # the dirty tokens are left out of the page's scale: compare with its own cache
        k, v, ks, vs = (t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
        sub = Step([at], [L - n + at], seed=1)
        sub.pages = step.pages
        _check_attend(sub, (k, v, ks, vs), dirty[:at, :Hkv], outs[1][:at], 1 / math.sqrt(D))


def test_append_out_of_range_tokens_are_dropped_and_flagged():
    ql, L, Hq, Hkv, D = [2, 2, 3], [70, 130, 66], 4, 2, 128
    step = Step(ql, L, seed=2)
    bufs = _pool(step, Hkv, D, seed=2)
    rope = rope_table(131, 128, device=DEV)
    qkv = torch.randn((step.N, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    q, k, v = qkv.split((Hq, Hkv, Hkv), dim=1)
    q_off, kv_len, pages = step.dev()
    good = _cache(bufs, Hq, Hkv, D, rope=rope)
    ws = good.new_workspace()
    good_q = good.append(k, v, q_off, kv_len, pages, ws, max_q=3, q=q)
    assert good.check(ws) == 0

    def run(kv_len, pages, rope=rope):
        cache = _cache(bufs, Hq, Hkv, D, rope=rope)
        out = cache.append(k, v, q_off, kv_len, pages, ws, max_q=3, q=q)
        assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX
        assert torch.equal(out[:2], good_q[:2]) and torch.equal(out[4:], good_q[4:])
        ids = [int(step.pages[b, p]) for b in (0, 2) for p in range((L[b] + 63) // 64)]
        assert torch.equal(cache.k[ids], good.k[ids]) and torch.equal(cache.v[ids], good.v[ids])
        return cache, out

    for bad in (-1, step.n_pages, 2 ** 31 - 1):
        p = pages.clone()
        p[1, 2] = bad
        cache, out = run(kv_len, p)
        assert bool((out[2:4] == 0).all())
        assert torch.equal(cache.k[step.pages[1, :2].long()].cpu(), bufs[0][step.pages[1, :2].long()])
    for n in (-3, 10 ** 9):
        cache, out = run(torch.tensor([70, n, 66], dtype=torch.int32, device=DEV), pages)
        assert bool((out[2:4] == 0).all())
    cache, out = run(torch.tensor([70, 1, 66], dtype=torch.int32, device=DEV), pages)   # one token has no position
    assert bool((out[2] == 0).all()) and bool((out[3] != 0).any())
    cache, out = run(kv_len, pages, rope=rope[:129])                                    # past the table
    assert bool((out[2:4] == 0).all())


def test_kv_refusals():
    cache = KVCache(4, 4, 2, 64)
    ws = cache.new_workspace()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=DEV)
    pages = torch.zeros((1, 2), dtype=torch.int32, device=DEV)
    ok = (i32(0, 2), i32(2), pages, ws)
    inv, mis, uns = binding.MOE_ERR_INVALID_ARG, binding.MOE_ERR_MISALIGNED, binding.MOE_ERR_UNSUPPORTED_SHAPE
    flat = torch.zeros(4096, dtype=torch.bfloat16, device=DEV)
    bufs = dict(k=cache.k, v=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale)
    rope = torch.zeros((8, 66), dtype=torch.float32, device=DEV)
    cases = [
        (lambda: cache.attend(q[:, :2], *ok, max_q=2), inv), (lambda: cache.attend(q.float(), *ok, max_q=2), inv),
        (lambda: cache.attend(q, *ok, max_q=3), inv), (lambda: cache.attend(q, *ok, max_q=-1), inv),
        (lambda: cache.attend(q, i32(0, 2, 2), i32(2), pages, ws, max_q=2), inv),
        (lambda: cache.attend(q, i32(0, 2).long(), i32(2), pages, ws, max_q=2), inv),
        (lambda: cache.attend(q, i32(0, 2), i32(2), pages[:, :0], ws, max_q=2), inv),
        (lambda: cache.attend(q, i32(0, 2), i32(2), pages, ws[:256], max_q=2), inv),
        (lambda: cache.attend(q, *ok, max_q=2, scale=float("nan")), inv),
        (lambda: cache.attend(q, *ok, max_q=2, out=q[:1]), inv),
        (lambda: cache.attend(flat[4:4 + 512].view(2, 4, 64), *ok, max_q=2), mis),
        (lambda: cache.attend(torch.as_strided(flat, (2, 4, 64), (260, 64, 1)), *ok, max_q=2), mis),
        (lambda: cache.attend(q.transpose(1, 2).contiguous().transpose(1, 2), *ok, max_q=2), inv),
        (lambda: cache.append(k, k[:1], *ok, max_q=2), inv), (lambda: cache.append(k, k.half(), *ok, max_q=2), inv),
        (lambda: cache.append(k, k, *ok, max_q=2, q_out=q), inv),
        (lambda: cache.append(flat[4:4 + 256].view(2, 2, 64), k, *ok, max_q=2), mis),
        (lambda: KVCache(4, 4, 2, 96), uns), (lambda: KVCache(4, 3, 2, 64), uns),
        (lambda: KVCache(4, 4, 2, 64, rope=rope, buffers=bufs), uns),
        (lambda: KVCache(4, 4, 2, 64, rope=rope[:, :3].contiguous(), buffers=bufs), uns),
        (lambda: KVCache(5, 4, 2, 64, buffers=bufs), inv),
    ]
    for i, (call, status) in enumerate(cases):
        with pytest.raises(MoeError) as ei:
            call()
        assert ei.value.status == status, i
    many = torch.zeros(514, dtype=torch.int32, device=DEV)
    with pytest.raises(MoeError):
        cache.attend(q, many, many[:513], torch.zeros((513, 1), dtype=torch.int32, device=DEV), ws, max_q=2)
    # nothing to do is no error
    assert cache.attend(q[:0], i32(0), i32(), pages[:0], ws, max_q=0).shape == (0, 4, 64)
    assert cache.append(k[:0], k[:0], i32(0, 0), i32(0), pages, ws, max_q=0) is None
    assert cache.check(ws) == 0
