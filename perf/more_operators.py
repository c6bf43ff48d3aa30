"""Speculative decoding and parallel sampling over the paged 8-bit cache, as measured cases.

Five operators: the append of a tree of drafted tokens (`append_tree`), the attention
of its tokens (`attend_tree`), the compaction of the cache to the tokens that were
accepted (`compact`), the fork of sequences (`fork`), and the sampling of tokens from
logits with given random numbers (`sample`).  `run` computes them in plain torch
operations, or with the package's kernels when `own` is true.
"""
import math

import torch

own = False

DEV = "cuda"
PAGE = 64          # tokens of a cache page: one scale for each page and kv head
LO_EXP = -64       # smallest exponent of a cache scale
GREEDY = 1e-6      # largest temperature that means: the most likely token


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence, a small tree: the smallest call, latency counts
        dict(name="append_tree_one", op="append_tree", B=1, n=8, kv=4001, Hq=32, Hkv=8, D=128, R=128, inter=False, ragged=False),
        # a verification batch: trees of up to 60 tokens, part of the head rotated, interleaved pairs
        dict(name="append_tree_batch", op="append_tree", B=32, n=60, kv=8192, Hq=32, Hkv=8, D=128, R=64, inter=True, ragged=True),
        # one sequence, a small tree after a short cache: latency
        dict(name="attend_tree_one", op="attend_tree", B=1, n=16, kv=4001, Hq=32, Hkv=8, D=128, ragged=False),
        # trees of different sizes over short caches, small heads, an odd group
        dict(name="attend_tree_ragged", op="attend_tree", B=7, n=37, kv=3000, Hq=24, Hkv=8, D=64, ragged=True),
        # a verification batch far into long sequences: cache bandwidth and arithmetic
        dict(name="attend_tree_batch", op="attend_tree", B=16, n=60, kv=16384, Hq=64, Hkv=8, D=128, ragged=True),
        # one sequence keeps the accepted path of a small tree
        dict(name="compact_one", op="compact", B=1, n=16, kv=4001, Hq=32, Hkv=8, D=128),
        # a large verification batch keeps its paths
        dict(name="compact_batch", op="compact", B=128, n=60, kv=2048, Hq=32, Hkv=8, D=128),
        # eight samples of one prompt, the first in the prompt's own pages
        dict(name="fork_samples", op="fork", B=1, C=8, kv=4001, Hq=32, Hkv=8, D=128),
        # a step of a search with many beams: most move to another sequence's pages
        dict(name="fork_beams", op="fork", B=384, C=384, kv=1000, Hq=32, Hkv=8, D=128),
        # one decoded token: latency
        dict(name="sample_one", op="sample", T=1, V=65543, half=False, masked=False, plain=False),
        # a decode batch, every row with settings of its own
        dict(name="sample_batch", op="sample", T=24, V=65543, half=False, masked=False, plain=False),
        # the rows of a verification batch over a larger vocabulary, logits in 16 bits, whole distributions
        dict(name="sample_many", op="sample", T=256, V=131075, half=True, masked=False, plain=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append_tree", "attend_tree", "attend_tree", "compact", "fork", "sample", "sample"])
    if op == "sample":
        return dict(op=op, T=_log_int(rng, 1, 256), V=_log_int(rng, 32, 131075), half=rng.random() < 0.5,
                    masked=rng.random() < 0.25, plain=rng.random() < 0.25)
    Hq, Hkv, D = rng.choice([(32, 8, 128), (64, 8, 128), (16, 1, 128), (8, 8, 128), (24, 8, 64), (8, 8, 64), (20, 4, 64)])
    if op == "fork":
        B = _log_int(rng, 1, 384)
        return dict(op=op, B=B, C=_log_int(rng, 1, 384), kv=_log_int(rng, 1, 1000), Hq=Hq, Hkv=Hkv, D=D)
    n = _log_int(rng, 1, 60)
    if op == "compact":
        return dict(op=op, B=_log_int(rng, 1, 128), n=n, kv=_log_int(rng, 1, 2048), Hq=Hq, Hkv=Hkv, D=D)
    if op == "append_tree":
        return dict(op=op, B=_log_int(rng, 1, 32), n=n, kv=_log_int(rng, 1, 8192), Hq=min(Hq, 32), Hkv=Hkv, D=D,
                    R=2 * rng.randint(0, D // 2), inter=rng.random() < 0.5, ragged=rng.random() < 0.5)
    return dict(op=op, B=_log_int(rng, 1, 16), n=n, kv=_log_int(rng, 1, 16384), Hq=Hq, Hkv=Hkv, D=D,
                ragged=rng.random() < 0.5)


# ----------------------------------------------------------------------------- inputs
def _lengths(case):
    """Tree tokens and total length of each sequence: plain values that depend on the
    case alone.  kv is the largest length before this step."""
    B, n, kv = case["B"], case.get("n", 0), case["kv"]
    ql = [(n, n // 2 + 1, 1, n, n // 3)[b % 5] if case.get("ragged") else n for b in range(B)]
    past = [kv if b == 0 else 1 + (kv * (16 + (b * 37) % 48)) // 64 for b in range(B)]
    return ql, [min(p, kv) + m for p, m in zip(past, ql)]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _cache(g, case, spare):
    """A paged cache with its tokens in it, pages in random order, `spare` of them free."""
    ql, kl = _lengths(case)
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    need = torch.tensor([(m + PAGE - 1) // PAGE for m in kl], device=DEV)
    used, width = int(need.sum()), int(need.max()) + 1
    n_pages = used + spare
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    live = torch.arange(width, device=DEV) < need[:, None]
    pages = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    pages[live] = perm[:used]
    k = torch.empty((n_pages, Hkv, PAGE, D), dtype=torch.uint8, device=DEV)
    v = torch.empty((n_pages, Hkv, D, PAGE), dtype=torch.uint8, device=DEV)
    for c in (k, v):
        for p0 in range(0, n_pages, 1024):
            part = c[p0:p0 + 1024]
            part.copy_((torch.randn(part.shape, generator=g, device=DEV) * 80).clamp_(-448, 448)
                       .to(torch.float8_e4m3fn).view(torch.uint8))
    ks, vs = torch.exp2(torch.randint(-8, -5, (2, n_pages, Hkv), generator=g, device=DEV).float())
    off = [0]
    for m in ql:
        off.append(off[-1] + m)
    return dict(k=k, v=v, ks=ks.contiguous(), vs=vs.contiguous(), pages=pages, free=perm[used:],
                q_off=torch.tensor(off, dtype=torch.int32, device=DEV),
                kv_len=torch.tensor(kl, dtype=torch.int32, device=DEV), ql=ql, kl=kl, N=off[-1])


def _trees(g, ql):
    """The token before each of a tree's (counted inside its sequence), -1 at the root:
    every token after the first follows a random earlier one."""
    at = torch.cat([torch.arange(m, device=DEV) for m in ql])
    return ((torch.rand(len(at), generator=g, device=DEV) * at).floor().to(torch.int32) - (at == 0).int()).to(torch.int32)


def _logits(g, case):
    """Normal logits of a spread of their own for each row, a few dozen far above."""
    T, V = case["T"], case["V"]
    x = torch.randn((T, V), generator=g, device=DEV) * (0.7 + 2 * torch.rand((T, 1), generator=g, device=DEV))
    m = min(V, 40)
    at = (torch.randint(0, V, (T, 1), generator=g, device=DEV) + torch.arange(m, device=DEV) * (V // m)) % V  # apart
    top = 12 * torch.exp(-torch.arange(m, device=DEV) / 8.0) * torch.rand((T, m), generator=g, device=DEV)
    x.scatter_(1, at, 4 + top)
    if case["masked"]:  # a grammar leaves a tenth of the tokens, one at least
        gone = torch.rand((T, V), generator=g, device=DEV) < 0.9
        x.masked_fill_(gone.scatter_(1, at[:, :1], False), float("-inf"))
    return x.bfloat16() if case["half"] else x


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=case, op=op)
    if op == "sample":
        T = case["T"]

        def pick(values, dtype):
            return torch.tensor(values, dtype=dtype, device=DEV)[torch.randint(0, len(values), (T,), generator=g, device=DEV)]

        st["logits"] = _logits(g, case)
        st["u"] = torch.rand(T, generator=g, device=DEV)
        st["temperature"] = pick([0.6, 0.8, 1.0, 1.3] if case["plain"] else [0.0, 0.3, 0.6, 0.8, 1.0, 1.0, 1.3], torch.float32)
        st["top_k"] = pick([0] if case["plain"] else [0, 0, 1, 20, 50, 50, 1000], torch.int32)
        st["top_p"] = pick([1.0] if case["plain"] else [1.0, 1.0, 0.5, 0.9, 0.95], torch.float32)
        st["min_p"] = pick([0.0] if case["plain"] else [0.0, 0.0, 0.0, 0.02, 0.1], torch.float32)
        return st
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    st.update(_cache(g, case, case["C"] if op == "fork" else 5))
    rope = None
    if op in ("append_tree", "attend_tree"):
        st["parents"] = _trees(g, st["ql"])
    if op == "append_tree":
        # queries, keys and values are slices of one projection's output, as they come from it
        st["qkv"] = torch.randn((st["N"], Hq + 2 * Hkv, D), generator=g, device=DEV).bfloat16()
        R = case["R"]
        pos = torch.arange(max(st["kl"]), dtype=torch.float64, device=DEV)
        inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / max(R, 1))
        ang = pos[:, None] * inv[None, :]
        rope = torch.stack((ang.cos(), ang.sin()), -1).reshape(len(pos), R).float()
        st["rope"] = rope
    elif op == "attend_tree":
        st["qr"] = torch.randn((st["N"], Hq, D), generator=g, device=DEV).bfloat16()
    elif op == "compact":
        # the accepted path: of each tree's tokens, the first and some later ones in order
        n = case["n"]
        K = min(n, 8)
        st["n_keep"] = torch.randint(1, K + 1, (case["B"],), generator=g, device=DEV).to(torch.int32)
        order = torch.rand((case["B"], n), generator=g, device=DEV)
        order[:, 0] = -1
        first = torch.arange(K, device=DEV) < st["n_keep"][:, None]
        chosen = order.argsort(-1)[:, :K]
        st["keep"] = torch.where(first, chosen, n).sort(-1).values.to(torch.int32).contiguous()
    else:
        # most children follow a sequence that has children already; the first of each stays in its pages
        B, C = case["B"], case["C"]
        src = (torch.rand(C, generator=g, device=DEV).square() * B).long().clamp_(max=B - 1)
        if C <= B:
            src[0] = 0
        later = torch.tril((src[:, None] == src[None, :]), -1).any(1)
        st["src"] = src.to(torch.int32)
        st["fresh"] = torch.where(later, st["free"], -1).to(torch.int32).contiguous()
    if own:
        from quantized_moe_routed_gb300 import KVCache
        st["cache"] = KVCache(st["k"].shape[0], Hq, Hkv, D, rope=rope if rope is not None and rope.shape[1] else None,
                              interleaved=bool(case.get("inter")),
                              buffers=dict(k=st["k"], v=st["v"], k_scale=st["ks"], v_scale=st["vs"]))
        st["ws"] = st["cache"].new_workspace()
    return st


# ----------------------------------------------------------------------------- plain forms
def _e4m3(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _codes(values):
    return values.to(torch.float8_e4m3fn).view(torch.uint8)


def _pow2_scale(a):
    """Smallest power of two s with a <= 448 s (at least 2^LO_EXP)."""
    m, e = torch.frexp(a / 448)
    return torch.exp2(torch.where(m > 0.5, e, e - 1).clamp(min=LO_EXP).to(a.dtype)).where(a > 0, 2.0 ** LO_EXP)


def _rows(st):
    """Each sequence's rows of the step, padded to the longest: [B, n] and which are there."""
    n = max(st["ql"])
    at = torch.arange(n, device=DEV)
    there = at < (st["q_off"][1:] - st["q_off"][:-1])[:, None]
    return (st["q_off"][:-1, None] + at).long().clamp(max=st["N"] - 1), there


def _ancestors(st):
    """[B, n, n]: whether token j is token i or one before it (parents doubled)."""
    rows, there = _rows(st)
    n = rows.shape[1]
    parent = st["parents"][rows]
    up = ((parent[..., None] == torch.arange(n, device=DEV)) & there[..., None]).float()
    see = torch.eye(n, device=DEV) + up
    for _ in range(n.bit_length()):
        up = up @ up
        see = see + see @ up
    return see > 0


def _rotate(x, rope, inter):
    """x [..., heads, D] float, rope [..., R]: (cos, sin) pairs."""
    R = rope.shape[-1]
    if R == 0:
        return x
    cos, sin = rope[..., None, 0::2], rope[..., None, 1::2]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    rot = torch.stack((ra, rb), -1).flatten(-2) if inter else torch.cat((ra, rb), -1)
    return torch.cat((rot, x[..., R:]), -1)


def _append_tree(st):
    case = st["case"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    rows, there = _rows(st)
    n = rows.shape[1]
    past = st["kv_len"] - (st["q_off"][1:] - st["q_off"][:-1])
    depth = _ancestors(st).sum(-1) - 1
    x = st["qkv"][rows].float()
    rope = st["rope"][(past[:, None] + depth).clamp(max=len(st["rope"]) - 1)]
    q_out = torch.empty((st["N"], Hq, D), dtype=torch.bfloat16, device=DEV)
    q_out[rows[there]] = _rotate(x[:, :, :Hq], rope, case["inter"])[there].bfloat16()
    first, fill = past // PAGE, past % PAGE
    NP = (n + 62) // PAGE + 1
    slot = (fill[:, None] + torch.arange(n, device=DEV)).long()            # of the pages from the first one on
    which = torch.arange(B, device=DEV)[:, None].expand(B, n)
    live = torch.zeros((B, NP * PAGE), dtype=torch.bool, device=DEV)
    live[which[there], slot[there]] = True
    live = live.view(B, NP, PAGE)
    at = (first[:, None] + torch.arange(NP, device=DEV)).long()
    ids = torch.gather(st["pages"], 1, at.clamp(max=st["pages"].shape[1] - 1)).long()
    got = live.any(-1)
    kept = torch.zeros((B, NP), dtype=torch.bool, device=DEV)
    kept[:, 0] = fill > 0
    ids = ids[got]
    for new, codes, scales, turn in ((_rotate(x[:, :, Hq:Hq + Hkv], rope, case["inter"]), st["k"], st["ks"], False),
                                     (x[:, :, Hq + Hkv:], st["v"], st["vs"], True)):
        t = torch.zeros((B, NP * PAGE, Hkv, D), device=DEV)
        t[which[there], slot[there]] = new[there]
        t = t.view(B, NP, PAGE, Hkv, D).transpose(2, 3)[got]                # [pages, Hkv, PAGE, D]
        old, was = _e4m3(codes[ids]), scales[ids]
        old = old.transpose(2, 3) if turn else old
        sc = _pow2_scale(t.abs().amax((2, 3)))
        sc = torch.where(kept[got][:, None], torch.maximum(sc, was), sc)
        grew = kept[got][:, None] & (was < sc)
        old = old * torch.where(grew, was / sc, 1.0)[:, :, None, None]
        val = torch.where(live[got][:, None, :, None], t / sc[:, :, None, None], old)
        codes[ids] = _codes((val.transpose(2, 3) if turn else val).contiguous())
        scales[ids] = sc
    return q_out


def _attend_tree(st):
    case = st["case"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    rows, there = _rows(st)
    n, P = rows.shape[1], (max(st["kl"]) + PAGE - 1) // PAGE
    ids = st["pages"][:, :P].long().clamp(min=0)
    k = (_e4m3(st["k"][ids]) * st["ks"][ids][..., None, None]).transpose(1, 2).reshape(B, Hkv, P * PAGE, D)
    v = (_e4m3(st["v"][ids]) * st["vs"][ids][..., None, None]).permute(0, 2, 1, 4, 3).reshape(B, Hkv, P * PAGE, D)
    q = st["qr"][rows].float().view(B, n, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, n * G, D)
    s = (q @ k.transpose(-1, -2)).view(B, Hkv, n, G, P * PAGE) / math.sqrt(D)
    past = (st["kv_len"] - (st["q_off"][1:] - st["q_off"][:-1]))[:, None]
    t = torch.arange(P * PAGE, device=DEV)
    node = (t - past).long()
    vis = torch.gather(_ancestors(st), 2, node.clamp(0, n - 1)[:, None, :].expand(B, n, P * PAGE))
    vis = (vis & (node < n)[:, None]) | (node < 0)[:, None]
    s = s.masked_fill(~vis[:, None, :, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, n * G, P * PAGE) @ v).view(B, Hkv, n, G, D).transpose(1, 2).reshape(B, n, Hq, D)
    out = torch.zeros((st["N"], Hq, D), dtype=torch.bfloat16, device=DEV)
    out[rows[there]] = o[there].bfloat16()
    return out


def _compact(st):
    case = st["case"]
    n, pages = case["n"], st["pages"]
    keep = st["keep"].long().clamp(max=n - 1)
    K = keep.shape[1]
    past = st["kv_len"].long() - n
    j = torch.arange(K, device=DEV)
    there = j < st["n_keep"][:, None]
    to, frm = past[:, None] + j, past[:, None] + keep
    page_of = lambda t: torch.gather(pages, 1, (t // PAGE).clamp(max=pages.shape[1] - 1)).long()  # noqa: E731
    sp, dp = page_of(frm), page_of(to)
    first = past // PAGE
    at = first[:, None] + torch.arange(2, device=DEV)                       # a path of 8 ends in the next page at the latest
    ids = page_of(at * PAGE)
    comes = there[:, None] & ((to // PAGE)[:, None] == at[..., None])       # [B, 2, K]
    kept = torch.zeros_like(at, dtype=torch.bool)
    kept[:, 0] = past % PAGE > 0
    changes = comes.any(-1)
    rows = torch.arange(len(past), device=DEV)[:, None].expand_as(there)
    t = (to // PAGE - first[:, None])[there]
    for codes, scales, turn in ((st["k"], st["ks"], False), (st["v"], st["vs"], True)):
        own_scale, src_scale = scales[ids], scales[sp]                      # [B, 2, H], [B, K, H]
        new = torch.where(comes[..., None], src_scale[:, None], 0.0).amax(2)
        new = torch.maximum(new, torch.where(kept[..., None], own_scale, 0.0))
        moved = _e4m3(codes[sp[there], :, :, frm[there] % PAGE] if turn else codes[sp[there], :, frm[there] % PAGE])
        moved = moved * (src_scale[there] / new[rows[there], t])[..., None]
        fall = torch.where(own_scale < new, own_scale / new, 1.0)[changes][..., None, None]
        codes[ids[changes]] = _codes(_e4m3(codes[ids[changes]]) * fall)
        if turn:
            codes[dp[there], :, :, to[there] % PAGE] = _codes(moved)
        else:
            codes[dp[there], :, to[there] % PAGE] = _codes(moved)
        scales[ids[changes]] = new[changes]
    return (past + st["n_keep"]).to(torch.int32)


def _fork(st):
    src, fresh = st["src"].long(), st["fresh"]
    kv_len = st["kv_len"][src]
    pages = st["pages"][src]
    at = (kv_len // PAGE).long()
    mine = fresh >= 0
    tail = torch.gather(pages, 1, at[:, None])[:, 0]
    pages[mine, at[mine]] = fresh[mine]
    copies = mine & (kv_len % PAGE > 0)
    to, frm = fresh[copies].long(), tail[copies].long()
    for buf in (st["k"], st["v"], st["ks"], st["vs"]):
        buf[to] = buf[frm]
    return pages, kv_len


def _sample(st):
    # in 64 bits: the borders lie between sums over the whole vocabulary
    d = torch.float64
    s, order = torch.sort(st["logits"].float(), dim=-1, descending=True, stable=True)
    rank = torch.arange(s.shape[1], device=DEV)
    t, u = st["temperature"].to(d)[:, None], st["u"].to(d)[:, None]
    k, p, mp = st["top_k"][:, None], st["top_p"].to(d)[:, None], st["min_p"].to(d)[:, None]
    w = torch.exp((s.to(d) - s[:, :1].to(d)) / t.clamp(min=GREEDY))
    w = torch.where((t <= GREEDY) & (rank > 0), 0.0, w)
    w = torch.where(((k > 0) & (rank >= k)) | (w < mp), 0.0, w)
    w = torch.where((p < 1) & (rank > 0) & (w.cumsum(-1) - w >= p * w.sum(-1, keepdim=True)), 0.0, w)
    cum = w.cumsum(-1)
    at = (cum <= u * cum[:, -1:]).sum(-1, keepdim=True)
    return order.gather(1, at)[:, 0].to(torch.int32), (w.gather(1, at) / cum[:, -1:])[:, 0].float()


# ----------------------------------------------------------------------------- one pass
def _cache_out(st, **more):
    return dict(k=st["k"].view(torch.float8_e4m3fn), v=st["v"].view(torch.float8_e4m3fn), k_scale=st["ks"],
                v_scale=st["vs"], **more)


def run(st):
    op, case = st["op"], st["case"]
    if not own:
        if op == "append_tree":
            return _cache_out(st, q=_append_tree(st))
        if op == "attend_tree":
            return _attend_tree(st)
        if op == "compact":
            return _cache_out(st, kv_len=_compact(st))
        if op == "fork":
            pages, kv_len = _fork(st)
            return _cache_out(st, pages=pages, kv_len=kv_len)
        token, prob = _sample(st)
        return dict(token=token, prob=prob)
    if op == "sample":
        from quantized_moe_routed_gb300 import sample
        token, prob = sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                             min_p=st["min_p"], return_prob=True)
        return dict(token=token, prob=prob)
    cache, ws = st["cache"], st["ws"]
    if op == "fork":
        pages, kv_len = cache.fork(st["src"], st["fresh"], st["kv_len"], st["pages"], ws)
        return _cache_out(st, pages=pages, kv_len=kv_len)
    step = (st["q_off"], st["kv_len"], st["pages"], ws, max(st["ql"]))
    if op == "append_tree":
        Hq, Hkv = case["Hq"], case["Hkv"]
        q, k, v = st["qkv"].split((Hq, Hkv, Hkv), dim=1)
        return _cache_out(st, q=cache.append(k, v, *step, q=q, parents=st["parents"]))
    if op == "attend_tree":
        return cache.attend(st["qr"], *step, parents=st["parents"])
    return _cache_out(st, kv_len=cache.compact(st["keep"], st["n_keep"], *step))


# ----------------------------------------------------------------------------- least work
def work(case):
    op = case["op"]
    if op == "sample":
        n = case["T"] * case["V"]
        return dict(bytes=n * (2 if case["half"] else 4) + 28 * case["T"], flops=4 * n)
    ql, kl = _lengths(case)
    Hq, Hkv, D, N = case["Hq"], case["Hkv"], case["D"], sum(ql)
    if op == "append_tree":
        return dict(bytes=N * D * (4 * Hq + 4 * Hkv + 2 * Hkv) + 4 * N * (case["R"] + 1), flops=N * D * (3 * Hq + 5 * Hkv))
    if op == "attend_tree":
        # of its own tree a token sees its path: about the logarithm of the tree's size
        pairs = sum(m * (L - m + 1 + math.log(m)) for m, L in zip(ql, kl) if m)
        read = sum(L for m, L in zip(ql, kl) if m)
        return dict(bytes=read * Hkv * 2 * D + 4 * N * Hq * D + 4 * N, flops=4 * pairs * Hq * D)
    if op == "compact":  # half of up to eight tokens move
        moved = case["B"] * (min(case["n"], 8) + 1) / 2
        return dict(bytes=moved * Hkv * D * 4 + 8 * case["B"] * (2 * Hkv + 4), flops=0)
    # every second child copies its page, roughly
    width = (max(kl) + PAGE - 1) // PAGE + 1
    return dict(bytes=case["C"] * (0.5 * Hkv * D * PAGE * 4 + 8 * width + 16), flops=0)


# ----------------------------------------------------------------------------- the definitions in 64 bits
def _scale64(a):
    """Smallest power of two s with a <= 448 s, from exact comparisons."""
    e = torch.floor(torch.log2(a.clamp(min=1e-300) / 448)) - 1
    for _ in range(3):
        e = torch.where(a > 448 * torch.exp2(e), e + 1, e)
    return torch.exp2(e.clamp(min=LO_EXP))


def _code64(v):
    """Nearest E4M3 value (ties to even), |v| <= 448, in 64-bit arithmetic."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _values64():
    c = torch.arange(256, device=DEV)
    e, m, sign = (c >> 3) & 15, (c & 7).double(), 1 - 2 * (c >> 7).double()
    return sign * torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))


def _paths(parents, ql):
    """For each token the list of those it sees of its tree, itself last."""
    out, at, p = [], 0, parents.tolist()
    for m in ql:
        mine = []
        for i in range(m):
            mine.append((mine[p[at + i]] if p[at + i] >= 0 else []) + [i])
        out.append(mine)
        at += m
    return out


def _exact_sample(st):
    token, prob = [], []
    for i in range(st["case"]["T"]):
        l = st["logits"][i].double()
        t, k, p, mp = (float(st[name][i]) for name in ("temperature", "top_k", "top_p", "min_p"))
        if t <= GREEDY:
            best = int((l == l.max()).nonzero()[0])
            token.append(best)
            prob.append(1.0)
            continue
        ids = torch.argsort(-l, stable=True)
        q = torch.softmax(l[ids] / t, 0)
        q = q[:int(k)] if k > 0 else q
        q = q[q >= mp * q[0]]
        q = q / q.sum()
        if p < 1:
            q = q[:max(1, int((q.cumsum(0) - q < p).sum()))]
            q = q / q.sum()
        at = min(int((q.cumsum(0) <= float(st["u"][i])).sum()), len(q) - 1)
        token.append(int(ids[at]))
        prob.append(float(q[at]))
    return dict(token=torch.tensor(token, dtype=torch.int32, device=DEV), prob=torch.tensor(prob, dtype=torch.float64, device=DEV))


def _exact_append(st):
    case, d = st["case"], torch.float64
    Hq, Hkv = case["Hq"], case["Hkv"]
    val = _values64()
    kv, vv, ks, vs = val[st["k"].long()], val[st["v"].long()], st["ks"].to(d), st["vs"].to(d)
    x = st["qkv"].to(d)
    paths = _paths(st["parents"], st["ql"])
    pos = torch.tensor([L - n + len(path) - 1 for n, L, mine in zip(st["ql"], st["kl"], paths) for path in mine], device=DEV)
    half, tab = case["R"] // 2, st["rope"].to(d)[pos]
    for j in range(half):
        i0, i1 = (2 * j, 2 * j + 1) if case["inter"] else (j, j + half)
        c, s = tab[:, 2 * j, None], tab[:, 2 * j + 1, None]
        a, b = x[:, :Hq + Hkv, i0].clone(), x[:, :Hq + Hkv, i1].clone()
        x[:, :Hq + Hkv, i0], x[:, :Hq + Hkv, i1] = a * c - b * s, a * s + b * c
    at = 0
    for b, (n, L) in enumerate(zip(st["ql"], st["kl"])):
        p = L - n
        while p < L:
            m = min(PAGE - p % PAGE, L - p)          # new tokens of this page
            page, o = int(st["pages"][b, p // PAGE]), p % PAGE
            i = at + p - (L - n)
            for new, old, sc in ((x[i:i + m, Hq:Hq + Hkv].permute(1, 0, 2), kv[page], ks[page]),
                                 (x[i:i + m, Hq + Hkv:].permute(1, 0, 2), vv[page].transpose(1, 2), vs[page])):
                want = _scale64(new.abs().amax((1, 2)))
                if o:
                    want = torch.maximum(want, sc)
                    old.copy_(_code64(old * (sc / want)[:, None, None]))
                old[:, o:o + m] = _code64(new / want[:, None, None])
                sc.copy_(want)
            p += m
        at += n
    return dict(q=x[:, :Hq], k=kv, v=vv, k_scale=ks, v_scale=vs)


def _exact_attend(st):
    case, d = st["case"], torch.float64
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    val = _values64()
    out = torch.zeros((st["N"], Hq, D), dtype=d, device=DEV)
    at = 0
    for b, (n, L) in enumerate(zip(st["ql"], st["kl"])):
        ids = st["pages"][b, :(L + PAGE - 1) // PAGE].long()
        hide = torch.zeros((n, L), dtype=d, device=DEV)
        hide[:, L - n:] = float("-inf")
        for i, path in enumerate(_paths(st["parents"][at:at + n], [n])[0]):
            hide[i, [L - n + a for a in path]] = 0
        for h in range(Hkv if n else 0):
            k = (val[st["k"][ids, h].long()] * st["ks"][ids, h].to(d)[:, None, None]).reshape(-1, D)[:L]
            v = (val[st["v"][ids, h].long()] * st["vs"][ids, h].to(d)[:, None, None]).transpose(1, 2).reshape(-1, D)[:L]
            q = st["qr"][at:at + n, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].to(d)
            s = torch.einsum("igd,jd->gij", q, k) * D ** -0.5 + hide
            out[at:at + n, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = torch.einsum("gij,jd->igd", torch.softmax(s, -1), v)
        at += n
    return out


def _exact_compact(st):
    d, val = torch.float64, _values64()
    kv, vv, ks, vs = val[st["k"].long()], val[st["v"].long()], st["ks"].to(d), st["vs"].to(d)
    n, pages, keep, n_keep = st["case"]["n"], st["pages"].tolist(), st["keep"].tolist(), st["n_keep"].tolist()
    kv_len = []
    for b, L in enumerate(st["kl"]):
        past, m = L - n, n_keep[b]
        kv_len.append(past + m)
        place = [(pages[b][(past + i) // PAGE], (past + i) % PAGE) for i in keep[b][:m]]
        for val_, sc, turn in ((kv, ks, False), (vv, vs, True)):
            col = [(val_[p, :, :, o] if turn else val_[p, :, o]).clone() for p, o in place]
            was = [sc[p].clone() for p, _ in place]
            for t in range(past // PAGE, (past + m - 1) // PAGE + 1):
                page = pages[b][t]
                here = [j for j in range(m) if (past + j) // PAGE == t]
                want = torch.stack([was[j] for j in here] + ([sc[page]] if past > t * PAGE else [])).amax(0)
                f = torch.where(sc[page] < want, sc[page] / want, torch.ones_like(want))
                val_[page] = _code64(val_[page] * f[:, None, None])
                for j in here:
                    new = _code64(col[j] * (was[j] / want)[:, None])
                    if turn:
                        val_[page, :, :, (past + j) % PAGE] = new
                    else:
                        val_[page, :, (past + j) % PAGE] = new
                sc[page] = want
    return dict(k=kv, v=vv, k_scale=ks, v_scale=vs, kv_len=torch.tensor(kv_len, dtype=torch.int32, device=DEV))


def _exact_fork(st):
    val = _values64()
    k, v, ks, vs = val[st["k"].long()], val[st["v"].long()], st["ks"].double(), st["vs"].double()
    pages, lens = [], []
    for s, f in zip(st["src"].tolist(), st["fresh"].tolist()):
        L, row = st["kl"][s], st["pages"][s].tolist()
        if f >= 0:
            if L % PAGE:
                for buf in (k, v, ks, vs):
                    buf[f] = buf[row[L // PAGE]]
            row[L // PAGE] = f
        pages.append(row)
        lens.append(L)
    return dict(k=k, v=v, k_scale=ks, v_scale=vs, pages=torch.tensor(pages, dtype=torch.int32, device=DEV),
                kv_len=torch.tensor(lens, dtype=torch.int32, device=DEV))


def exact(case, seed):
    form = dict(append_tree=_exact_append, attend_tree=_exact_attend, compact=_exact_compact, fork=_exact_fork, sample=_exact_sample)
    return form[case["op"]](prepare(case, seed))
