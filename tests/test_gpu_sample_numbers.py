"""Settings of `sample` that are Python numbers of any size."""
import pytest
import torch

from quantized_moe_routed_gb300 import sample

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_top_k_past_32_bits_is_no_limit():
    x = torch.zeros((1, 2000), device=DEV)
    u = torch.full((1,), 0.75, device=DEV)
    assert int(sample(x, u)) == 1500
    for k in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 32 + 8, 2 ** 63 - 1, 10 ** 30, 0, -1, -2 ** 31, -2 ** 32 + 1):
        assert int(sample(x, u, top_k=k)) == 1500, k
    assert int(sample(x, u, top_k=8)) == 6


@pytest.mark.parametrize("temperature", [1.0, 1e30, 1e38, float("inf")])
def test_a_distance_past_fp32_weighs_nothing(temperature):
    """Two tokens within fp32's range of the largest share what is left of one that is not."""
    x = torch.tensor([[-3e38, 3e38, 3e38, -3.4e38] + [float("-inf")] * 60], device=DEV)
    for u, want in ((0.0, 1), (0.49, 1), (0.51, 2), (0.9999, 2)):
        assert int(sample(x, torch.tensor([u], device=DEV), temperature=temperature)) == want
