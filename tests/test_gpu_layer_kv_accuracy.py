"""moe_kv_attend as accurate as its operands' formats are: against the definition in
64 bits, for each kernel with the bound that its own roundings give.

With w a row's weights, s its scores, v = code * scale of the page, A = sum w |v| / sum w, M =
the row's largest w * scale, C = sum |code| over the visible tokens, qm the row's largest
|q|, mag = sum |q k| of a score:

  output    rounded to bf16: 2^-8 |o|
  weights   (weight x scale) rounded to fp16: 2^-11 of each, or half of fp16's smallest step:
            up to 16 rows 256 of them at the reference, which is at most 2 M: 2^-25 / 256 * 2 M
            = 2^-32 M; more rows 64 of them: 2^-30 M
  scores    eight tensor-core additions of fp32 sums: 2^-20 mag, half as much again for the
            scaling; and what q's format leaves out: 2^-38 qm an element (fp16), 2^-17 qm
            (two E4M3 digits: half of E4M3's smallest step where qm is in [128, 256));
            2^-20 for the exponential and its argument
  sums      each addition on the tensor cores cuts less than 2^-23 of the sum: one for 128
            tokens and warp (up to 16 rows), one for 16 tokens of a run of 128 x 128 (more); 40
            for joining
    |error| <= 2^-8 |o| + (2^-11 + 2 ds + cut) A + {2^-32, 2^-30} M C / sum w

And in the norm, where roundings of either sign do not add up: with R = sqrt(sum (w v)^2) /
sum w, a sum of such errors, each at most u of its w v, is off by u R / sqrt(3) in the mean, and
partial sums of values of either sign stay within 4 R.  So
    ||error|| <= 2^-8 ||o|| + ||(2^-11 + 2 left + 4 cut) R + (2^-19 mag + 2^-19) A + third||
(left: what q's format leaves out of a score), 0.4 to 0.9% of ||o|| in most cases here: a sum
that is wrong by one per cent, for instance by a rescaling that is, fails them.
"""
import math

import pytest
import torch

from quantized_moe_routed_gb300 import KVCache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4 = torch.float8_e4m3fn


class Pool:
    """Sequences of lengths L over pages in random order; exps: powers of two of the
    scales, frac: scales that are no powers of two."""

    def __init__(self, L, Hkv, D, seed, exps=(-8, -4), frac=False):
        self.L, self.D = L, D
        g = self.g = torch.Generator(device=DEV).manual_seed(seed)
        need = [(n + 63) // 64 for n in L]
        N = sum(need) + 3
        self.k, self.v = ((torch.randn(s, generator=g, device=DEV) * 60).clamp(-448, 448).to(E4)
                          for s in ((N, Hkv, 64, D), (N, Hkv, D, 64)))
        e = torch.randint(exps[0], exps[1], (2, N, Hkv), generator=g, device=DEV).float()
        if frac:
            e = e + torch.rand(e.shape, generator=g, device=DEV)
        self.ks, self.vs = torch.exp2(e)
        perm = torch.randperm(N, generator=g, device=DEV).int()
        self.pages = torch.full((len(L), max(need)), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b, m in enumerate(need):
            self.pages[b, :m] = perm[at:at + m]
            at += m

    def run(self, n, Hq, q, scale):
        cache = KVCache(self.k.shape[0], Hq, self.k.shape[1], self.D,
                        buffers=dict(k=self.k.view(torch.uint8), v=self.v.view(torch.uint8), k_scale=self.ks.contiguous(),
                                     v_scale=self.vs.contiguous()))
        ws, B = cache.new_workspace(), len(self.L)
        out = cache.attend(q, (torch.arange(B + 1, device=DEV) * n).int(), torch.tensor(self.L, dtype=torch.int32, device=DEV),
                           self.pages, ws, n, scale=scale)
        assert cache.check(ws) == 0
        return out


def check(p, n, Hq, q, scale):
    out, D, Hkv = p.run(n, Hq, q, scale).double(), p.D, p.k.shape[1]
    G = Hq // Hkv
    few = n * G <= 16
    for b, L in enumerate(p.L):
        ids = p.pages[b, :(L + 63) // 64].long()
        for h in range(Hkv):
            k = (p.k[ids, h].double() * p.ks[ids, h].double()[:, None, None]).reshape(-1, D)[:L]
            code = p.v[ids, h].double().transpose(1, 2).reshape(-1, D)[:L]
            vs = p.vs[ids, h].double().repeat_interleave(64)[:L]
            x = q[b * n:(b + 1) * n, h * G:(h + 1) * G].double().reshape(n * G, D)
            got = out[b * n:(b + 1) * n, h * G:(h + 1) * G].reshape(n * G, D)
            seen = (L - n + 1 + torch.arange(n * G, device=DEV) // G)[:, None] > torch.arange(L, device=DEV)
            s = (x @ k.T * scale).masked_fill(~seen, -math.inf)
            w = torch.exp(s - s.amax(-1, keepdim=True))
            tot = w.sum(-1, keepdim=True)
            v = code * vs[:, None]
            o, A = w @ v / tot, w @ v.abs() / tot
            M = (w * vs).amax(-1, keepdim=True)
            C = seen.double() @ code.abs()
            ka = k.abs()
            mag, qm = (x.abs() @ ka.T).masked_fill(~seen, 0).amax(-1, keepdim=True), x.abs().amax(-1, keepdim=True)
            left = abs(scale) * 2.0 ** (-38 if few else -17) * qm * ka.sum(-1).max()
            add = abs(scale) * 1.5 * 2.0 ** -20 * mag + 2.0 ** -20
            cut = ((L / 128 if few else min(L / 16, 1024)) + 40) * 2.0 ** -23
            third = 2.0 ** (-32 if few else -30) * M * C / tot
            tol = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * (add + left) + cut) * A + third
            err = (got - o).abs()
            assert bool((err <= tol * (1 + 2.0 ** -7)).all()), (b, h, float((err / tol).max()))
            R = ((w * w) @ (v * v)).sqrt() / tot
            bound = 2.0 ** -8 * o.norm() + ((2.0 ** -11 + 2 * left + 4 * cut) * R + 2 * add * A + third).norm()
            assert float(err.norm()) <= float(bound), (b, h, float(err.norm() / bound))


# new tokens, query heads, kv heads: tiles of 8, 16 and 128 rows
FEW = [(1, 8, 2), (1, 8, 1), (2, 32, 4), (1, 16, 1), (4, 16, 4), (5, 2, 1)]
MANY = [(5, 16, 4), (16, 64, 8), (33, 4, 4), (200, 16, 4), (1, 40, 2)]


@pytest.mark.parametrize("n,Hq,Hkv", FEW + MANY)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("frac", [False, True])
def test_random(n, Hq, Hkv, D, frac):
    p = Pool([n + 2500, n + 37, max(n, 64), 5000], Hkv, D, seed=n + Hq, frac=frac)
    q = torch.randn((4 * n, Hq, D), generator=p.g, device=DEV).bfloat16()
    check(p, n, Hq, q, D ** -0.5)


@pytest.mark.parametrize("n,Hq,Hkv", FEW + MANY)
@pytest.mark.parametrize("D", [64, 128])
def test_scales_far_apart(n, Hq, Hkv, D):
    """Values of pages that differ by up to 2^40: small weights of large pages count,
    large weights of small ones hardly."""
    p = Pool([n + 2000, n + 700], Hkv, D, seed=n + Hq, exps=(-25, 15))
    p.ks.fill_(2.0 ** -6)
    q = (torch.randn((2 * n, Hq, D), generator=p.g, device=DEV) * 3).bfloat16()
    check(p, n, Hq, q, D ** -0.5)


@pytest.mark.parametrize("n,Hq,Hkv,up", [(1, 8, 2, 18), (4, 16, 4, 18), (5, 16, 4, 7), (16, 64, 8, 9), (200, 16, 4, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_with_an_element_far_larger_than_the_rest(n, Hq, Hkv, up, D):
    """Where keys have nothing at that element the others keep the bits that their format
    promises: all of them with up to 16 rows, those above 2^-10 of the largest with more."""
    p = Pool([n + 900, n + 60], Hkv, D, seed=n + Hq)
    p.k.view(torch.uint8)[..., 7] = 0
    q = torch.randn((2 * n, Hq, D), generator=p.g, device=DEV)
    q[..., 7] *= 2.0 ** up
    check(p, n, Hq, q.bfloat16(), D ** -0.5)


@pytest.mark.parametrize("gain", [1, 3, 5])
@pytest.mark.parametrize("n,Hq,Hkv,D", [(16, 64, 8, 128), (16, 64, 8, 64), (200, 16, 4, 128), (1, 64, 8, 128), (1, 64, 8, 64)])
def test_maxima_that_move(n, Hq, Hkv, D, gain):
    """Long sequences, scores of several units: every sequence and head."""
    L = [16400, 9488, 2576, 12048, 5136, 14608, 7696, 784]
    for seed in range(2):
        p = Pool(L, Hkv, D, seed=seed, exps=(-6, -5))
        q = (torch.randn((len(L) * n, Hq, D), generator=p.g, device=DEV) * gain).bfloat16()
        check(p, n, Hq, q, D ** -0.5)


@pytest.mark.parametrize("n,Hq,Hkv", [(1, 8, 1), (2, 8, 1), (40, 8, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_maximum_at_every_place(n, Hq, Hkv, D):
    """One token far above the others, wherever it stands: rescaling by next to nothing,
    and sums that end with next to one weight."""
    L = [40, 64, 65, 130, 200, 300, 511, 700]
    p = Pool(L, Hkv, D, seed=n, exps=(-6, -5))
    q = torch.randn((len(L) * n, Hq, D), generator=p.g, device=DEV).bfloat16()
    for b, length in enumerate(L):
        at = (length - n) * (b + 1) // (len(L) + 1)
        key = (q[b * n, 0].float() * 100).clamp(-448, 448).to(E4)
        p.k.view(torch.uint8)[p.pages[b, at // 64].long(), 0, at % 64] = key.view(torch.uint8)
    check(p, n, Hq, q, D ** -0.5)
