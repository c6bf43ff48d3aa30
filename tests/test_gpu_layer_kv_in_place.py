"""moe_kv_append with q_out = q: the bits of a separate output, for every way of
pairing elements (halves whose partners one thread holds, halves whose partners
are other threads' elements, neighbours, none), and the cache's as well."""
import pytest
import torch

from quantized_moe_routed_gb300 import rope_table
from test_gpu_layer_kv import Step, _cache, _pool

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("D,R", [(64, 0), (64, 64), (64, 6), (64, 50), (128, 128), (128, 32), (128, 2), (128, 104), (128, 126)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("ql,L", [([1, 1, 1], [1, 64, 65]), ([7, 0, 130], [9, 3, 333]), ([64], [64])])
def test_queries_in_place(D, R, inter, ql, L):
    Hq, Hkv = 12, 4
    step = Step(ql, L, seed=R)
    bufs = _pool(step, Hkv, D, seed=R)
    g = torch.Generator().manual_seed(R)
    q = torch.randn((step.N, Hq, D), generator=g).bfloat16().to(DEV)
    k, v = torch.randn((2, step.N, Hkv, D), generator=g).bfloat16().to(DEV)
    rope = rope_table(max(L), R, device=DEV) if R else None
    a, b = (_cache(bufs, Hq, Hkv, D, rope=rope, inter=inter) for _ in range(2))
    ws = a.new_workspace()
    want = a.append(k, v, *step.dev(), ws, step.max_q, q=q)
    for _ in range(10):
        mine = q.clone()
        assert b.append(k, v, *step.dev(), ws, step.max_q, q=mine, q_out=mine) is mine
        assert torch.equal(mine, want)
    assert a.check(ws) == 0
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(a, name), getattr(b, name))
