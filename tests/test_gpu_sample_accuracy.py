"""How far moe_sample's sums may be off: by a unit of 2^-45 a token and 2^-36 of themselves.

A row of one logit of 0, one of weight 1 - x, and a tail of equal ones whose sum is s: half of
the sum is met by the first token alone where 1 - x + s <= 1.  All errors of such a tail have one
sign, so this is the worst row there is."""
import math

import pytest
import torch

from quantized_moe_routed_gb300 import sample

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _second(s, by, up):
    """The fp32 logit of the second token nearest to where w + s - 1 is `by` (up) or -by, not nearer to 0; and that."""
    x = s - by if up else s + by
    f = torch.tensor(math.log1p(-x), dtype=torch.float32)
    while True:
        margin = math.expm1(float(f)) + s
        if (margin >= by) if up else (margin <= -by):
            return float(f), margin
        f = torch.nextafter(f, torch.tensor(math.inf if up else -math.inf))


# weights of 2^-19 to half a unit; of 5.5, 2.5, 1.5 and 0.51 units, whose roundings are the largest
TAILS = [-13.2, -17.0, -20.3, -24.0, -28.0] + [math.log(u * 2.0 ** -45) for u in (5.5, 2.5, 1.5, 0.51)]


@pytest.mark.parametrize("T,V", [(1, 262144), (160, 262144), (1, 131075), (160, 50001)])
@pytest.mark.parametrize("tail", TAILS)
def test_a_tail_of_equal_logits(T, V, tail):
    l = float(torch.tensor(tail, dtype=torch.float32))
    s = (V - 2) * math.exp(l)
    by = V * 2.0 ** -45 + (2 + s) * 2.0 ** -36
    x = torch.full((T, V), l, device=DEV)
    first, second = V // 3, V // 2
    x[:, first] = 0
    for up, want in ((True, second), (False, first)):
        if up and s <= by:              # (the second would be the largest)
            continue
        x[:, second], margin = _second(s, by, up)
        assert by <= abs(margin) < 2 * by + 2.0 ** -24          # (near the border, and past what the sums are off by)
        tok = sample(x, torch.full((T,), 0.999, device=DEV), top_p=0.5)
        assert tok.tolist() == [want] * T, (up, margin, by)


def test_u_past_the_end_gives_the_last_token_of_a_unit():
    V = 5000
    x = torch.full((1, V), math.log(0.4 * 2.0 ** -45), device=DEV)
    x[:, 100] = 0
    x[:, 40] = math.log(0.6 * 2.0 ** -45)
    for u in (1.0, 2.0, math.inf):
        assert int(sample(x, torch.tensor([u], device=DEV))) == 40
