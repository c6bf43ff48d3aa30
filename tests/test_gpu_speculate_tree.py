"""Trees of new tokens: moe_kv_append_tree and moe_kv_attend_tree against their 64-bit
definitions, with the tolerances that test_gpu_layer_kv derives for sequences (the same
products, sums and roundings; only what is seen, and what a token turns by, differ)."""
import math

import pytest
import torch

import layer_reference as ref
import speculate_reference as spec
import test_gpu_layer_kv as base
from quantized_moe_routed_gb300 import KVCache, MoeError, binding, rope_table

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 64


def _check(step, bufs, q, out, parents, scale, skip=()):
    Hq, D = q.shape[1:]
    Hkv = bufs[0].shape[1]
    G = Hq // Hkv
    out = out.cpu().double()
    for b, (n, L) in enumerate(zip(step.ql, step.L)):
        if n == 0 or b in skip:
            continue
        r0 = int(step.q_off[b])
        tree = parents[r0:r0 + n].tolist()
        for h in range(Hkv):
            k, v = base._gather(step, bufs, b, h)
            qq = q[r0:r0 + n, h * G:(h + 1) * G]
            want, A, ln, vm = spec.attend_tree(qq, k, v, tree, L, scale)
            ka = k.abs()
            ka = torch.where(ka.isnan(), 0.0, ka).amax(0) if L else torch.zeros(D, dtype=torch.float64)
            mag = (qq.double().abs() * ka).sum(-1)
            ds = abs(scale) * (2.0 ** -20 * mag + 2.0 ** -18 * qq.double().abs().amax(-1) * ka.sum())
            seen = torch.clamp(L - n + torch.arange(n).double() + 1, 0, L)[:, None]
            tol = (2.0 ** -8 * want.abs() + (2.0 ** -9 + 2 * ds)[..., None] * A +
                   (2.0 ** -18 * seen * vm / ln)[..., None] + 1e-37)
            err = (out[r0:r0 + n, h * G:(h + 1) * G] - want).abs()
            assert bool((err <= tol).all()), (b, h, float((err / tol).max()))


ATTEND = [
    # ql, L, Hq, Hkv, D: single tokens, few rows, many; trees across one page and more; nothing before the tree
    ([1], [1], 1, 1, 64), ([4], [4], 4, 2, 128), ([2, 1, 2], [66, 700, 2], 8, 2, 128), ([8], [70], 8, 8, 64),
    ([16], [80], 4, 4, 128), ([5, 3], [64, 67], 24, 8, 64), ([7], [300], 33, 1, 128), ([16, 9], [16, 4000], 16, 2, 64),
    ([63, 0, 65], [100, 5, 65], 8, 2, 128), ([64], [128], 6, 2, 64), ([130], [140], 4, 1, 128), ([256], [256], 2, 1, 64),
    ([256, 1], [319, 64], 8, 2, 128), ([200, 40], [1000, 40], 1, 1, 128), ([37] * 9, [130, 37, 64, 65, 200, 39, 127, 511, 90], 16, 2, 128),
]


@pytest.mark.parametrize("deep", [False, True])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend_matches_the_definition(case, deep):
    ql, L, Hq, Hkv, D = ATTEND[case]
    step = base.Step(ql, L, seed=case)
    bufs = base._pool(step, Hkv, D, seed=case)
    base._stale(step, bufs[0])
    parents = spec.random_trees(ql, case, deep)
    q = torch.randn((step.N, Hq, D), generator=torch.Generator().manual_seed(case)).bfloat16()
    cache = base._cache(bufs, Hq, Hkv, D)
    ws = cache.new_workspace()
    args = (q.to(DEV), *step.dev(), ws)
    out = cache.attend(*args, max_q=step.max_q, parents=parents.to(DEV))
    assert cache.check(ws) == 0
    _check(step, bufs, q, out, parents, 1 / math.sqrt(D))
    assert torch.equal(out, cache.attend(*args, max_q=step.max_q, parents=parents.to(DEV)))


@pytest.mark.parametrize("max_q", [1, 4, 8, 60, 256])
def test_attend_tiles_do_not_change_the_answer(max_q):
    ql, L, Hq, Hkv, D = [60, 1, 9, 196], [200, 333, 9, 300], 8, 2, 128
    step = base.Step(ql, L, seed=1)
    bufs = base._pool(step, Hkv, D, seed=1)
    parents = spec.random_trees(ql, 5)
    q = torch.randn((step.N, Hq, D), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache = base._cache(bufs, Hq, Hkv, D)
    ws = cache.new_workspace()
    out = cache.attend(q.to(DEV), *step.dev(), ws, max_q=max_q, parents=parents.to(DEV))
    assert cache.check(ws) == 0
    _check(step, bufs, q, out, parents, 1 / math.sqrt(D))


@pytest.mark.parametrize("ql,L", [([1], [500]), ([4, 2], [64, 500]), ([40, 70], [100, 70])])
def test_a_chain_is_a_sequence(ql, L):
    """Parents i - 1: the bits of the append and the attention of a sequence."""
    Hq, Hkv, D = 8, 2, 128
    step = base.Step(ql, L, seed=3)
    bufs = base._pool(step, Hkv, D, seed=3, exps=(-8, -6))
    rope = rope_table(max(L), D, device=DEV)
    qkv = torch.randn((step.N, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    q, k, v = qkv.split((Hq, Hkv, Hkv), dim=1)
    parents = torch.cat([torch.arange(n, dtype=torch.int32) - 1 for n in ql]).to(DEV)
    got = []
    for p in (None, parents):
        cache = base._cache(bufs, Hq, Hkv, D, rope=rope)
        ws = cache.new_workspace()
        qr = cache.append(k, v, *step.dev(), ws, max_q=step.max_q, q=q, parents=p)
        got.append((qr, cache.attend(qr, *step.dev(), ws, max_q=step.max_q, parents=p), cache.k, cache.v, cache.k_scale,
                    cache.v_scale))
        assert cache.check(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("n", [3, 12, 40])
def test_attend_sees_no_sibling(n):
    """NaN keys of tokens in other branches, and scores that would take every weight,
    reach nobody but those that follow them; a row sees itself alone where nothing is
    before the tree."""
    Hq, Hkv, D, L = 4, 1, 128, n
    step = base.Step([n], [L], seed=4)
    bufs = base._pool(step, Hkv, D, seed=4)
    parents = torch.full((n,), -1, dtype=torch.int32)
    parents[n - 1] = 0
    page = step.pages[0]
    bufs[0][page[0], :, 1] = 0x7F                     # token 1's key is NaN
    q = torch.randn((n, Hq, D), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache = base._cache(bufs, Hq, Hkv, D)
    ws = cache.new_workspace()
    out = cache.attend(q.to(DEV), *step.dev(), ws, max_q=n, parents=parents.to(DEV)).cpu()
    assert bool(out[1].isnan().all())
    v = ref.e4m3(bufs[1][page[0], 0].transpose(0, 1)) * float(bufs[3][page[0], 0])
    for i in range(n - 1):
        if i != 1:  # (one token alone: its value, rounded to bf16, from a weight of 1 rounded to fp16's 2^-11)
            assert bool(((out[i].double() - v[i]).abs() <= (2.0 ** -8 + 2.0 ** -11) * v[i].abs()).all()), i
    assert bool(out[n - 1].isfinite().all())


@pytest.mark.parametrize("n,Hq", [(9, 2), (40, 8)])
def test_attend_tokens_without_a_position_give_zeros(n, Hq):
    """A length of zero, and one smaller than the new tokens."""
    step = base.Step([n, n, n], [0, n - 3, 64], seed=2)
    bufs = base._pool(step, 2, 128, seed=2)
    parents = spec.random_trees(step.ql, 2)
    q = torch.randn((step.N, Hq, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache = base._cache(bufs, Hq, 2, 128)
    ws = cache.new_workspace()
    out = torch.full((step.N + 2, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    qd = torch.cat((q, q[:2])).to(DEV)
    cache.attend(qd, *step.dev(), ws, max_q=n, out=out, parents=torch.cat((parents, parents[:2])).to(DEV))
    assert bool((out[:n + 3] == 0).all()) and bool((out[step.N:] == 7).all())   # rows behind the last sequence: as they were
    _check(step, bufs, q, out[:step.N], parents, 1 / math.sqrt(128))


def test_bad_parents_and_long_trees_are_flagged():
    ql, L, Hq, Hkv, D = [6, 5, 300], [70, 130, 400], 4, 2, 128
    step = base.Step(ql, L, seed=6)
    bufs = base._pool(step, Hkv, D, seed=6, exps=(-8, -6))
    rope = rope_table(400, D, device=DEV)
    parents = spec.random_trees(ql, 3)
    qkv = torch.randn((step.N, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(1)).bfloat16()
    q, k, v = qkv.to(DEV).split((Hq, Hkv, Hkv), dim=1)
    cache = base._cache(bufs, Hq, Hkv, D, rope=rope)
    ws = cache.new_workspace()
    # the third sequence is no tree: nothing of it is appended, its rows are zeros
    before = cache.k[step.pages[2, :7].long()].clone()
    qr = cache.append(k, v, *step.dev(), ws, max_q=256, q=q, parents=parents.to(DEV))
    assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX and cache.check(ws) == 0
    assert bool((qr[11:] == 0).all()) and bool((qr[:11] != 0).any()) and torch.equal(before, cache.k[step.pages[2, :7].long()])
    out = cache.attend(q, *step.dev(), ws, max_q=256, parents=parents.to(DEV))
    assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX
    now = tuple(t.cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
    _check(step, now, qkv[:, :Hq], out, parents, 1 / math.sqrt(D), skip=(2,))
    assert bool((out[11:] == 0).all())
    # a parent that is no earlier token counts as none
    small = base.Step(ql[:2], L[:2], seed=6)
    small.pages = step.pages[:2]
    want = parents[:11].clone()
    want[8] = -1
    for bad in (-2, 2, 3, 5, 11, 2 ** 31 - 1, -2 ** 31):
        p = want.clone()
        p[8] = bad
        got = cache.attend(q[:11], *small.dev(), ws, max_q=6, parents=p.to(DEV))
        assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX, bad
        assert torch.equal(got, cache.attend(q[:11], *small.dev(), ws, max_q=6, parents=want.to(DEV)))
        one = cache.append(k[:11], v[:11], *small.dev(), ws, max_q=6, q=q[:11], parents=p.to(DEV))
        assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX, bad
        assert torch.equal(one, cache.append(k[:11], v[:11], *small.dev(), ws, max_q=6, q=q[:11], parents=want.to(DEV)))
        assert cache.check(ws) == 0


APPEND = [
    # ql, L, Hq, Hkv, D, R, interleaved
    ([1], [1], 4, 2, 128, 128, False), ([9, 1, 4], [64, 65, 200], 8, 8, 64, 64, True),
    ([12, 0, 20], [33, 5, 128], 12, 4, 128, 64, False), ([64], [64], 2, 1, 128, 0, False),
    ([100, 3], [100, 66], 8, 2, 128, 128, True), ([256, 1], [333, 1], 6, 2, 64, 6, False), ([60, 17], [70, 100], 4, 4, 64, 50, True),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_matches_the_definition(case):
    """What a sequence's append stores, with each token turned by its depth."""
    ql, L, Hq, Hkv, D, R, inter = APPEND[case]
    step = base.Step(ql, L, seed=case)
    bufs = base._pool(step, Hkv, D, seed=case, exps=(-8, -6))
    parents = spec.random_trees(ql, case)
    g = torch.Generator().manual_seed(case)
    qkv = torch.randn((step.N, Hq + 2 * Hkv, D), generator=g).bfloat16()
    rope = rope_table(max(L), R, device="cpu", magnitude=1.1) if R else None
    cache = base._cache(bufs, Hq, Hkv, D, rope=None if rope is None else rope.to(DEV), inter=inter)
    ws = cache.new_workspace()
    q, k, v = qkv.to(DEV).split((Hq, Hkv, Hkv), dim=1)
    q_out = cache.append(k, v, *step.dev(), ws, max_q=step.max_q, q=q, parents=parents.to(DEV))
    assert cache.check(ws) == 0
    pos = torch.tensor([b - n + len(spec.path(parents[r0:r0 + n].tolist(), i)) - 1
                        for r0, n, b in zip(step.q_off.tolist(), ql, L) for i in range(n)])
    turned = qkv[:, :Hq + Hkv].double()
    slack = 0.0
    if R:
        slack = (turned.abs() + turned.abs().amax(-1, keepdim=True)) * 2.0 ** -22 * 1.1
        turned = ref.rotate(turned, rope[pos], inter)
    # keys that are turned already, stored without a rotation
    kv, vv, ks, vs, new, _ = base._ref_append(step, bufs, turned[:, Hq:], qkv[:, Hq + Hkv:], None, inter)
    assert torch.equal(cache.k_scale.cpu().double(), ks) and torch.equal(cache.v_scale.cpu().double(), vs)
    assert torch.equal(ref.e4m3(cache.v.cpu()), vv)
    got = ref.e4m3(cache.k.cpu())
    live = new[:, None, :, None].expand_as(got)
    assert torch.equal(got[~live], kv[~live])
    # half an E4M3 step, and what fp32 may move a key by (2^-22 of the pair, in units of the scale)
    tol = ref.half_step(kv) * (1 + 2.0 ** -10)
    if R:
        top = turned[:, Hq:].abs().max() * 2 * 2.0 ** -22 * 1.1
        tol = tol + top / ks[:, :, None, None].clamp(min=1e-30)
    assert bool(((got - kv).abs() <= tol)[live].all())
    tol = 2.0 ** -8 * turned[:, :Hq].abs() + (slack[:, :Hq] if R else 0)
    assert bool(((q_out.cpu().double() - turned[:, :Hq]).abs() <= tol).all())
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    assert cache.append(k, v, *step.dev(), ws, max_q=1, parents=parents.to(DEV)) is None
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)))


def test_append_in_place_and_short_tables():
    """Queries turned in place; tokens stored past the table are dropped and flagged."""
    ql, L, Hq, Hkv, D, R = [20], [90], 4, 2, 64, 42
    step = base.Step(ql, L, seed=1)
    bufs = base._pool(step, Hkv, D, seed=1)
    parents = spec.random_trees(ql, 7).to(DEV)
    rope = rope_table(90, R, device=DEV)
    q, k, v = (torch.randn((20, h, D), generator=torch.Generator().manual_seed(h)).bfloat16().to(DEV) for h in (Hq, Hkv, Hkv))
    cache = base._cache(bufs, Hq, Hkv, D, rope=rope)
    ws = cache.new_workspace()
    want = cache.append(k, v, *step.dev(), ws, max_q=20, q=q, parents=parents)
    mine = q.clone()
    cache.append(k, v, *step.dev(), ws, max_q=20, q=mine, q_out=mine, parents=parents)
    assert torch.equal(want, mine) and cache.check(ws) == 0
    short = base._cache(bufs, Hq, Hkv, D, rope=rope[:89].contiguous())
    out = short.append(k, v, *step.dev(), ws, max_q=20, q=q, parents=parents)
    assert short.check(ws) == binding.MOE_ERR_BAD_INDEX and bool((out == 0).all())


def test_streams_graphs_and_strides():
    ql, L, Hq, Hkv, D = [13, 4], [500, 60], 8, 2, 128
    step = base.Step(ql, L, seed=7)
    bufs = base._pool(step, Hkv, D, seed=7, exps=(-8, -6))
    parents = spec.random_trees(ql, 1)
    qkv = torch.randn((step.N, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache = base._cache(bufs, Hq, Hkv, D)
    ws = cache.new_workspace()
    args, qd, pd = step.dev(), qkv.to(DEV), parents.to(DEV)
    torch.cuda.synchronize()
    first = cache.attend(qd[:, :Hq], *args, ws, max_q=13, parents=pd)
    _check(step, bufs, qkv[:, :Hq], first, parents, 1 / math.sqrt(D))
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [cache.attend(qd[:, :Hq], *args, ws, max_q=13, parents=pd, stream=streams[i % 3]) for i in range(9)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    out = torch.empty_like(first)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]   # two graphs that share the workspace
    for g in graphs:
        with torch.cuda.graph(g):
            cache.attend(qd[:, :Hq], *args, ws, max_q=13, parents=pd, out=out)
    for g in graphs * 2:
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)


def test_refusals():
    cache = KVCache(4, 4, 2, 64)
    ws = cache.new_workspace()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=DEV)
    ok = (i32(0, 2), i32(2), torch.zeros((1, 2), dtype=torch.int32, device=DEV), ws)
    p = i32(-1, 0)
    for bad in (p.long(), p[:1], p.cpu(), i32(-1, -1, 0, 0)[::2], p.view(1, 2), [0, 1]):
        for call in (lambda: cache.attend(q, *ok, max_q=2, parents=bad), lambda: cache.append(k, k, *ok, max_q=2, parents=bad)):
            with pytest.raises(MoeError) as ei:
                call()
            assert ei.value.status == binding.MOE_ERR_INVALID_ARG
    many = torch.zeros((300, 4, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(MoeError) as ei:
        cache.attend(many, *ok, max_q=257, parents=torch.zeros(300, dtype=torch.int32, device=DEV))
    assert ei.value.status == binding.MOE_ERR_UNSUPPORTED_SHAPE
    assert cache.attend(q[:0], i32(0), i32(), ok[2][:0], ws, max_q=0, parents=p[:0]).shape == (0, 4, 64)
    assert cache.check(ws) == 0
