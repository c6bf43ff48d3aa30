"""Trees of more than 32 tokens in the attention of few rows (a max_q that is too small), whose last tile has rows
past the sequence's: those see nothing, and are written by nobody."""
import math

import pytest
import torch

import speculate_reference as spec
import test_gpu_layer_kv as base
import test_gpu_speculate_tree as tree

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("max_q", [1, 5])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 128), (9, 3, 64), (3, 1, 128)])
def test_rows_past_the_last_token(Hq, Hkv, D, max_q):
    ql, L = [33, 45, 91], [400, 45, 100]
    step = base.Step(ql, L, seed=1)
    bufs = base._pool(step, Hkv, D, seed=1)
    parents = spec.random_trees(ql, 5)
    G = Hq // Hkv
    rows = 8 if max_q * G <= 8 else 16
    assert max_q * G <= 16 and any(n * G % rows for n in ql)
    q = torch.randn((step.N, Hq, D), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache = base._cache(bufs, Hq, Hkv, D)
    ws = cache.new_workspace()
    out = torch.full((step.N + 16, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    wide = torch.full((step.N + 16, Hq, D), math.inf, dtype=torch.bfloat16, device=DEV)   # behind the sequences: not read
    wide[:step.N] = q.to(DEV)
    more = torch.cat((parents, torch.full((16,), 2 ** 30, dtype=torch.int32))).to(DEV)
    runs = []
    for _ in range(2):
        cache.attend(wide, *step.dev(), ws, max_q=max_q, out=out, parents=more)
        runs.append(out.clone())
    assert cache.check(ws) == 0 and torch.equal(*runs) and bool((out[step.N:] == 7).all())
    tree._check(step, bufs, q, out[:step.N], parents, 1 / math.sqrt(D))
