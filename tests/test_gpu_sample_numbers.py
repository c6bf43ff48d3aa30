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
