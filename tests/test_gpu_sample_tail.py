"""moe_sample on rows with a long tail of tokens that weigh less than half a unit of 2^-45
each: they are given to nobody, but count in the sums that borders are made of.

A weight w = 2^-x of the tail counts in units of 2^-63 where x < 63.5, rounded, so a sum of
2^18 of them is off by 2^-46 and what the 30 bits of a weight leave, 2^-29 of itself.  A
border that equal logits meet exactly (m tokens of weight 1, top_p = j / m) is decided by
whether anything counts behind them."""
import math

import pytest
import torch

import speculate_reference as spec
from quantized_moe_routed_gb300 import sample

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# rows and vocabulary: one row over a cluster, many rows of a block each, in fp32 and bf16 (weighed one
# by one, and counted by value)
SHAPES = [(1, 262144, False), (1, 262144, True), (1, 9001, False), (1, 9001, True), (200, 33000, False), (200, 33000, True)]


def _row(T, V, half, tops, tail, peak=0.0):
    """Rows of `tail` with `tops` places of the largest logit, apart and in no special place."""
    x = torch.full((T, V), tail)
    at = [(V * (2 * i + 1)) // (2 * tops) for i in range(tops)]
    x[:, at] = peak
    return (x.bfloat16() if half else x), at


def _ask(x, u, **kw):
    T = x.shape[0]
    tok, prob = sample(x.to(DEV), torch.full((T,), u, device=DEV), return_prob=True, **kw)
    assert bool((tok == tok[0]).all()) and bool((prob == prob[0]).all())
    return int(tok[0]), float(prob[0])


@pytest.mark.parametrize("T,V,half", SHAPES)
@pytest.mark.parametrize("tail", [-24.0, -31.0, -32.5, -38.0, -43.5])
def test_the_tail_moves_a_border_that_is_met_exactly(T, V, half, tail):
    """m tokens of weight 1 and a tail of weight 2^-34.6 to 2^-62.8 each: j / m of the sum is more than j tokens."""
    assert tail == float(torch.tensor(tail).bfloat16())
    for m, j in ((2, 1), (4, 1), (4, 3), (8, 5)):
        x, at = _row(T, V, half, m, tail)
        want, prob = at[j], 1 / (j + 1)
        if V * math.exp(tail) > 2.0 ** -45:                     # (where 64 bits hold the sum, the definition says so)
            assert spec.sample(x[0].float(), 0.999, top_p=j / m)[0] == want
        tok, p = _ask(x, 0.999, top_p=j / m)
        assert tok == want and abs(p - prob) <= 2.0 ** -24, (m, j)
        assert _ask(x, 0.0, top_p=j / m)[0] == at[0]


@pytest.mark.parametrize("T,V,half", SHAPES)
@pytest.mark.parametrize("tail", [-60.0, -1e4, float(torch.finfo(torch.bfloat16).min), -math.inf])
def test_a_tail_that_counts_nothing_moves_no_border(T, V, half, tail):
    """Masked tokens, by -inf or by a low value: from 2^-63.5 down a weight is none."""
    for m, j in ((2, 1), (4, 3)):
        x, at = _row(T, V, half, m, tail)
        tok, p = _ask(x, 0.999, top_p=j / m)
        assert tok == at[j - 1] and abs(p - 1 / j) <= 2.0 ** -24, (m, j)


@pytest.mark.parametrize("T,V,half", SHAPES)
def test_filters_take_the_tail_away(T, V, half):
    """The tail (2^-46.9 each) is behind top-k's tokens, below min-p's weight, or neither."""
    x, at = _row(T, V, half, 2, -32.5)
    for kw, first in ((dict(top_k=2), True), (dict(top_k=3), False), (dict(top_k=V), False), (dict(min_p=2.0 ** -40), True),
                      (dict(min_p=2.0 ** -46), True), (dict(min_p=2.0 ** -46.5), True), (dict(min_p=2.0 ** -47), False),
                      (dict(min_p=2.0 ** -60), False), (dict(min_p=1e-30), False), (dict(top_k=2, min_p=2.0 ** -60), True)):
        tok, _ = _ask(x, 0.999, top_p=0.5, **kw)
        assert tok == at[0 if first else 1], kw
    # at another temperature: the same row, scaled (bf16 holds both)
    y, at = _row(T, V, half, 2, -8.125)
    assert _ask(y, 0.999, top_p=0.5, temperature=0.25)[0] == at[1]
    assert _ask(y, 0.999, top_p=0.5, temperature=0.125)[0] == at[0]


@pytest.mark.parametrize("V", [262144, 131075])
@pytest.mark.parametrize("T", [1, 160])
def test_the_tail_counts_with_its_weight(T, V):
    """A second token of weight 1 - x beside a tail of sum s: half of 2 - x + s is met by the first token alone where
    x > s.  x is a 32nd of s off: more than 2^-34, where a weight is exact to 2^-36 and the tail to 2^-29 of itself."""
    tail = -32.5
    s = (V - 2) * math.exp(tail)
    x, at = _row(T, V, False, 1, tail)
    second = V // 2 + V // 4
    for f, want in ((1 - 2.0 ** -5, second), (1 + 2.0 ** -5, at[0])):
        x[:, second] = -s * f
        assert s * 2.0 ** -5 > 2.0 ** -34.9
        assert spec.sample(x[0], 0.999, top_p=0.5)[0] == want
        assert _ask(x, 0.999, top_p=0.5)[0] == want


@pytest.mark.parametrize("T,V,half", SHAPES)
def test_the_tail_is_given_to_nobody(T, V, half):
    """u of 1 and above gives the last token whose weight does not round to nothing."""
    x, at = _row(T, V, half, 3, -33.0)
    x[:, at[1]] = -2.0
    assert _ask(x, 1.0)[0] == at[1] and _ask(x, math.inf)[0] == at[1] and _ask(x, 1 - 2.0 ** -24)[0] == at[1]
    x[:, 1:V // 2:2] = -math.inf
    x[:, 0] = math.nan
    assert _ask(x, 1.0)[0] == at[1]
    assert _ask(x, 0.999, top_p=0.5)[0] == at[2]                # (.5 of 2 + e^-2 is more than one token)
