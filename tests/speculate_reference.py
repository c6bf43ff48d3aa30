"""Plain 64-bit definitions, on the CPU, of what the tests of trees of tokens, of
the cache's moves and of the sampling compare with."""
import math

import torch

import layer_reference as ref

PAGE = ref.PAGE


def random_trees(ql, seed, deep=False):
    """Parents of the tokens of each sequence: a random earlier one (deep: a near one),
    now and then a second root."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in ql:
        for i in range(n):
            r = float(torch.rand((), generator=g))
            lo = max(0, i - 3) if deep else 0
            out.append(-1 if i == 0 or r > 0.97 else min(i - 1, lo + int(r / 0.97 * (i - lo))))
    return torch.tensor(out, dtype=torch.int32)


def path(parents, i):
    """Token i and those before it, from i to its root."""
    out = [i]
    while parents[out[-1]] >= 0:
        out.append(int(parents[out[-1]]))
    return out


def attend_tree(q, k, v, parents, L, scale):
    """One sequence, one kv head, as layer_reference.attend: q [n, G, D], k and v [L, D]."""
    n, G, D = q.shape
    past = L - n
    o, A = torch.zeros((n, G, D), dtype=torch.float64), torch.zeros((n, G, D), dtype=torch.float64)
    ln, vm = torch.ones((n, G), dtype=torch.float64), torch.zeros((n, G), dtype=torch.float64)
    for i in range(n):
        see = list(range(max(past, 0))) + [past + a for a in path(parents, i) if past + a >= 0]
        if not see:
            continue
        s = (q[i].double() @ k[see].T) * scale
        p = torch.exp(s - s.amax(-1, keepdim=True))
        ln[i] = p.sum(-1)
        p = p / p.sum(-1, keepdim=True)
        o[i], A[i], vm[i] = p @ v[see], p @ v[see].abs(), v[see].abs().max()
    return o, A, ln, vm


def compact(bufs, pages, q_off, kv_len, keep, n_keep):
    """Values (float64) of k and v, their scales, the new lengths."""
    k, v = ref.e4m3(bufs[0]), ref.e4m3(bufs[1])
    ks, vs = bufs[2].double().clone(), bufs[3].double().clone()
    out = []
    for b, L in enumerate(kv_len):
        n, m = q_off[b + 1] - q_off[b], n_keep[b]
        past = L - n
        out.append(past + m)
        place = [(int(pages[b, (past + i) // PAGE]), (past + i) % PAGE) for i in keep[b][:m]]
        for val, sc, turn in ((k, ks, False), (v, vs, True)):
            col = [(val[p, :, :, o] if turn else val[p, :, o]).clone() for p, o in place]
            was = [sc[p].clone() for p, _ in place]
            for t in range(past // PAGE, (past + m - 1) // PAGE + 1 if m else 0):
                page = int(pages[b, t])
                here = [j for j in range(m) if (past + j) // PAGE == t]
                want = torch.stack([was[j] for j in here] + ([sc[page]] if past > t * PAGE else [])).amax(0)
                f = torch.where(sc[page] < want, sc[page] / want, torch.ones_like(want))[:, None, None]
                val[page] = torch.where(f == 1, val[page], ref.to_e4m3(val[page] * f))
                for j in here:
                    fj = (was[j] / want)[:, None]
                    new = torch.where(fj == 1, col[j], ref.to_e4m3(col[j] * fj))
                    if turn:
                        val[page, :, :, (past + j) % PAGE] = new
                    else:
                        val[page, :, (past + j) % PAGE] = new
                sc[page] = want
    return k, v, ks, vs, out


def sample(row, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability, how near the decision is to another, relative to the sums) of one row."""
    l = row.double()
    l = torch.where(l.isnan(), -math.inf, l)
    if bool((l == -math.inf).all()):
        return -1, 0.0, 1.0
    order = torch.argsort(-l, stable=True)
    top = l[order[0]]
    if not temperature > 1e-6:
        return int(order[0]), 1.0, 1.0
    if top == math.inf:
        w = (l[order] == math.inf).double()
    else:
        w = torch.exp((l[order] - top) / temperature)
    near = 1.0
    if top_k > 0:
        w = w[:top_k]
    if min_p > 0:
        left = w >= min(min_p, 1.0)
        if min_p < 1:
            near = min(near, float((w / min_p - 1).abs().min()))
        w = w[left]
    if top_p < 1:
        before = w.cumsum(0) - w
        target = top_p * w.sum()
        near = min(near, float((before[1:] / target - 1).abs().min()) if len(w) > 1 and top_p > 0 else 1.0)
        left = before < target
        left[0] = True
        w = w[left]
    w = w[w > 0]
    cum, z = w.cumsum(0), w.sum()
    u = 0.0 if not u > 0 else u
    if u > 0:
        near = min(near, float((cum[:-1] / (u * z) - 1).abs().min()) if len(w) > 1 else 1.0)
    at = min(int((cum <= u * z).sum()), len(w) - 1)
    return int(order[at]), float(w[at] / z), near
