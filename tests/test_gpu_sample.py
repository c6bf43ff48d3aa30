"""moe_sample against its definition in 64 bits.

Weights are off by at most 2^-36 of themselves and 2^-46 of the largest, so sums of up to
2^18 of them by 2^-36 and 2^-28 of the largest's weight, at the worst; a decision
nearer to a border than that may go either way.  Errors of both signs add up far slower:
the tokens have to be equal wherever the definition is 2^-34 away from another one.
A probability is a quotient of a weight and such a sum, rounded to fp32: 2^-24 and 2^-33
of it, and the 2^-45 that a weight's unit may be in sums of 1 and more."""
import math

import pytest
import torch

import speculate_reference as spec
from quantized_moe_routed_gb300 import MoeError, binding, sample

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NEAR = 2.0 ** -34


def _logits(T, V, seed, spread=2.0, half=False, peaks=20):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, V), generator=g) * spread
    for t in range(T):
        at = torch.randperm(V, generator=g)[:peaks]
        x[t, at] += 8 * torch.rand(len(at), generator=g)
    return x.bfloat16() if half else x


def _compare(x, u, t=None, k=None, p=None, mp=None):
    """Sample with the settings (lists of a value a row, or one value) and compare every row."""
    T = x.shape[0]
    row = lambda v, one, i: one if v is None else (v[i] if isinstance(v, list) else v)  # noqa: E731
    arg = lambda v, dt: torch.tensor(v, dtype=dt, device=DEV) if isinstance(v, list) else v  # noqa: E731
    f = torch.float32
    kw = {n: arg(v, d) for n, v, d in (("temperature", t, f), ("top_k", k, torch.int32), ("top_p", p, f), ("min_p", mp, f))
          if v is not None}
    ud = torch.tensor(u, dtype=f)
    tok, prob = sample(x.to(DEV), ud.to(DEV), return_prob=True, **kw)
    alone = sample(x.to(DEV), ud.to(DEV), **kw)
    assert torch.equal(tok, alone)
    f32 = lambda v: float(torch.tensor(v, dtype=f))  # noqa: E731
    skipped = 0
    for i in range(T):
        want, wp, near = spec.sample(x[i].float(), float(ud[i]), f32(row(t, 1.0, i)), row(k, 0, i), f32(row(p, 1.0, i)),
                                     f32(row(mp, 0.0, i)))
        if near < NEAR:
            skipped += 1
            continue
        assert int(tok[i]) == want, (i, int(tok[i]), want, near)
        assert abs(float(prob[i]) - wp) <= (2.0 ** -24 + 2.0 ** -33) * wp + 2.0 ** -45, (i, float(prob[i]), wp)
    assert skipped <= T // 50 + 1


def _u(T, seed):
    return torch.rand(T, generator=torch.Generator().manual_seed(seed)).tolist()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 511, 2049, 4096, 4097, 8193, 16385, 65543, 131075, 262144])
def test_every_vocabulary_and_filter(V, half):
    T = 24 if V < 100000 else 12
    x = _logits(T, V, V, half=half)
    u = _u(T, V + 1)
    _compare(x, u)
    _compare(x, u, t=0.7, k=50, p=0.95, mp=0.02)
    g = torch.Generator().manual_seed(V)
    pick = lambda *v: [v[int(i)] for i in torch.randint(0, len(v), (T,), generator=g)]  # noqa: E731
    _compare(x, u, t=pick(0.0, 0.3, 0.8, 1.0, 2.5), k=pick(0, 1, 2, 40, 3000, 2 ** 31 - 1), p=pick(1.0, 0.5, 0.9, 0.99),
             mp=pick(0.0, 0.0, 0.05, 0.3))


@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.05, 6.0, 40.0])
@pytest.mark.parametrize("V", [300, 9000, 70001])
def test_flat_and_steep_rows(V, spread):
    """Rows that are nearly or quite flat (thousands of tokens in a bin), and rows where few tokens count."""
    x = _logits(8, V, 3, spread=spread, peaks=0)
    for half in (False, True):
        y = x.bfloat16() if half else x
        _compare(y, _u(8, 4))
        _compare(y, _u(8, 5), p=0.7)
        _compare(y, _u(8, 6), k=V // 2, p=0.99)


@pytest.mark.parametrize("T,V", [(3, 9001), (6, 131075), (24, 65543), (60, 131075), (20, 262144), (100, 20000), (170, 33000)])
def test_the_same_however_rows_are_split(T, V):
    """A row in a call of many, whose blocks have more of it and may count it by value, gets what it gets alone,
    bit for bit; masked rows, rows of one value, of two, with infinities and of nothing among them."""
    for half in (False, True):
        x = _logits(T, V, T, half=half)
        x[0] = 1.5
        x[1, ::3] = -math.inf
        x[2] = -2.0
        x[2, V // 2:] = 1.0
        if T > 5:
            x[3] = -math.inf
            x[4, V // 3], x[4, V - 1] = math.inf, math.inf
            x[5, :V - 2] = math.nan
        x = x.to(DEV)
        u = torch.tensor(_u(T, V), device=DEV)
        for t, k, p in ((1.0, 0, 1.0), (0.7, 0, 0.9), (1.2, 700, 0.95)):
            tok, prob = sample(x, u, temperature=t, top_k=k, top_p=p, return_prob=True)
            for i in list(range(min(T, 8))) + [T - 1]:
                one, its = sample(x[i:i + 1], u[i:i + 1], temperature=t, top_k=k, top_p=p, return_prob=True)
                assert int(one) == int(tok[i]) and float(its) == float(prob[i]), (i, half)


def test_many_rows_of_16_bits():
    """Logits that are counted by value: whole rows of one value (more than a counter holds; twice 2^16), two
    values, infinite and masked and NaN ones beside ordinary rows."""
    T, V = 80, 131072
    x = _logits(T, V, 21, half=True)
    x[0] = 0.0
    x[1] = -3.0
    x[1, 70000:] = 2.0
    x[2, ::2] = -math.inf
    x[3] = -math.inf
    x[4] = math.nan
    x[5, 100], x[5, 99999] = math.inf, math.inf
    x[6] = 1.0
    x[6, ::2] = -1.0
    x[7, :65536] = 5.0
    x[8] = -0.0
    x[8, 1::2] = 0.0
    x[9] = -math.inf
    x[9, 131071] = -7.0
    u = _u(T, 22)
    _compare(x, u)
    _compare(x, u, t=0.8, k=70000, p=0.97)
    _compare(x[:, 1:], u, t=[0.0, 1.0] * (T // 2), mp=0.05)
    tok = sample(x[:1].repeat(T, 1).to(DEV), (torch.arange(T) / T).to(DEV))
    assert tok.tolist() == [int(math.floor(float(torch.tensor(i / T)) * V)) for i in range(T)]


def test_ties_go_to_the_lowest_index():
    """All logits equal, and two values: ranks are indices, exactly, at every u."""
    V, T = 10007, 64
    x = torch.zeros((T, V))
    u = [i / T for i in range(T)]
    tok = sample(x.to(DEV), torch.tensor(u, device=DEV))
    assert tok.tolist() == [int(math.floor(a * V)) for a in u]          # cum > u V: V units, exact
    tok = sample(x.to(DEV), torch.tensor(u, device=DEV), top_k=100)
    assert tok.tolist() == [int(math.floor(a * 100)) for a in u]
    tok = sample(x.to(DEV), torch.tensor(u, device=DEV), top_p=0.5)     # 5004 tokens: 5003 are less than half
    assert tok.tolist() == [int(math.floor(a * 5004)) for a in u]
    x[:, 1::2] = -0.0                                                   # no other value than 0
    assert torch.equal(tok, sample(x.to(DEV), torch.tensor(u, device=DEV), top_p=0.5))
    x[:] = -5.0
    x[:, 4000:4010] = 3.0
    assert sample(x.to(DEV), torch.tensor(u, device=DEV), temperature=0).tolist() == [4000] * T
    assert sample(x.to(DEV), torch.tensor(u, device=DEV), top_k=10).tolist() == [4000 + int(math.floor(a * 10)) for a in u]
    assert sample(x.to(DEV), torch.tensor(u, device=DEV), min_p=1.0).tolist() == [4000 + int(math.floor(a * 10)) for a in u]


@pytest.mark.parametrize("V", [50, 5000, 70000])
def test_infinite_and_nan_logits(V):
    inf, nan = math.inf, math.nan
    x = _logits(7, V, 9)
    x[0] = -inf
    x[1] = nan
    x[2, ::2], x[2, 1::2] = nan, -inf
    x[2, 17] = -3.0                                 # one token is left
    x[3, 5], x[3, 40] = inf, inf                    # two infinite ones share it
    x[4, ::3] = -inf
    x[5] = -inf
    x[5, 20:30] = torch.arange(10.0)
    x[6, 3] = nan
    for u in (0.0, 0.4999, 0.5, 0.9999):
        _compare(x, [u] * 7)
        _compare(x, [u] * 7, k=3, p=0.9)
    tok, prob = sample(x.to(DEV), torch.zeros(7, device=DEV), temperature=0.0, return_prob=True)
    assert tok[:4].tolist() == [-1, -1, 17, 5] and prob.tolist() == [0, 0, 1, 1, 1, 1, 1]
    huge = torch.tensor([[3e38, -3e38, 2.9e38, 0.0] * (V // 4)])
    _compare(huge, [0.999])


def test_settings_at_their_limits():
    x = _logits(1, 3000, 11)
    order = torch.argsort(-x[0].double(), stable=True)
    ask = lambda u=0.5, **kw: int(sample(x.to(DEV), torch.tensor([u], device=DEV), **kw))  # noqa: E731
    top = int(order[0])
    for kw in (dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=1e-6), dict(temperature=math.nan), dict(top_k=1),
               dict(top_p=0.0), dict(top_p=-1.0), dict(min_p=1.0), dict(min_p=5.0), dict(top_p=1e-30), dict(temperature=1e-5)):
        assert ask(u=0.999, **kw) == top, kw
    plain = ask()
    for kw in (dict(top_k=0), dict(top_k=-3), dict(top_k=3000), dict(top_k=2 ** 31 - 1), dict(top_p=1.0), dict(top_p=7.0),
               dict(top_p=math.nan), dict(min_p=0.0), dict(min_p=-1.0), dict(min_p=math.nan)):
        assert ask(**kw) == plain, kw
    assert ask(u=0.0) == top and ask(u=-1.0) == top and ask(u=math.nan) == top and ask(u=1e-45) == top
    last = ask(u=1.0, top_k=7)
    assert last == int(order[6]) and ask(u=3.0, top_k=7) == last and ask(u=math.inf, top_k=7) == last
    assert ask(u=1 - 2.0 ** -24, top_k=2) == int(order[1])
    # an infinite temperature weighs all tokens the same: order stays that of the logits
    assert ask(u=0.5, temperature=math.inf) == int(order[1500])


def test_the_order_of_filters():
    """top-p counts what top-k and min-p leave."""
    x = torch.log(torch.tensor([[0.4, 0.3, 0.2, 0.1]]))
    _compare(x, [0.999], k=2, p=0.5)     # of .4 / .7: token 0 is enough
    _compare(x, [0.999], p=0.5)          # .4 is less: two tokens
    _compare(x, [0.999], mp=0.6, p=0.6)  # .4, .3 are left; .4 / .7 is less: both
    tok = sample(x.to(DEV), torch.tensor([0.999], device=DEV), top_k=2, top_p=0.5)
    assert int(tok) == 0


def test_frequencies():
    """Even random numbers draw each token as often as its probability says: the counts differ by
    one at most, as each token has an interval of its own."""
    n = 4096
    x = torch.log(torch.tensor([0.5, 0.125, 0.25, 0.125])).repeat(n, 1)
    u = (torch.arange(n) + 0.5) / n
    count = torch.bincount(sample(x.to(DEV), u.to(DEV)).cpu(), minlength=4)
    assert bool(((count - n * torch.tensor([0.5, 0.125, 0.25, 0.125])).abs() <= 1).all())


def test_strides_streams_and_graphs():
    T, V = 5, 9001
    wide = _logits(T, V + 23, 13)
    u = torch.tensor(_u(T, 3))
    for view in (wide[:, 3:3 + V], wide[:, :V], wide.bfloat16()[:, 1:V + 1]):
        x = wide.to(DEV).bfloat16()[:, 1:V + 1] if view.dtype == torch.bfloat16 else wide.to(DEV)[:, view.storage_offset():view.storage_offset() + V]
        tok = sample(x, u.to(DEV), temperature=0.9, top_p=0.95)
        want = [spec.sample(view[i].float(), float(u[i]), float(torch.tensor(0.9)), 0, float(torch.tensor(0.95)))[0] for i in range(T)]
        assert tok.tolist() == want
    xd, ud = wide.to(DEV), u.to(DEV)
    torch.cuda.synchronize()
    first = sample(xd, ud)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [sample(xd, ud, stream=streams[i % 3]) for i in range(9)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    out = torch.zeros(T, dtype=torch.int32, device=DEV)
    prob = torch.zeros(T, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert sample(xd, ud, out=out, prob=prob)[0] is out
    for i in range(3):
        ud.copy_(torch.tensor(_u(T, 20 + i)))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sample(xd, ud))


def test_refusals():
    x, u = torch.zeros((2, 64), device=DEV), torch.zeros(2, device=DEV)
    inv = binding.MOE_ERR_INVALID_ARG
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    cases = [lambda: sample(x.half(), u), lambda: sample(x[0], u), lambda: sample(x.t(), u), lambda: sample(x, u[:1]),
             lambda: sample(x, u.double()), lambda: sample(x, u.cpu()), lambda: sample(x, u, temperature=u[:1]),
             lambda: sample(x, u, top_k=u), lambda: sample(x, u, top_p=i32(1, 1)), lambda: sample(x, u, min_p=u.cpu()),
             lambda: sample(x, u, out=u), lambda: sample(x, u, out=i32(1)), lambda: sample(x, u, prob=i32(1, 1)),
             lambda: sample(x.cpu(), u)]
    for i, call in enumerate(cases):
        with pytest.raises(MoeError) as ei:
            call()
        assert ei.value.status == inv, i
    with pytest.raises(MoeError) as ei:
        sample(torch.zeros((1, 262145), device=DEV), u[:1])
    assert ei.value.status == binding.MOE_ERR_UNSUPPORTED_SHAPE
    assert sample(x[:0], u[:0]).shape == (0,)
