"""The cache's moves where their answers were once others: what the tests of the cache do not call."""
import pytest
import torch

import speculate_reference as spec
import test_gpu_layer_kv as base
import test_gpu_speculate_cache as moves
from quantized_moe_routed_gb300 import binding

pytestmark = pytest.mark.gpu
PAGE, i32 = moves.PAGE, moves.i32


# ----------------------------------------------------------------------------- pages between kept tokens
@pytest.mark.parametrize("past,keep", [(0, [0, 200]), (60, [1, 2, 255]), (0, [130, 255]), (63, [0, 1, 200])])
def test_compact_needs_only_the_pages_that_it_reads_and_writes(past, keep):
    """A page between them, whose tokens are all dropped, may have any id."""
    Hkv, D, n = 2, 64, 256
    step = base.Step([n], [past + n], seed=len(keep))
    bufs = base._pool(step, Hkv, D, seed=3)
    kept, n_keep = moves._table([keep])
    q_off, kv_len, pages = step.dev()
    *want, lens = spec.compact(bufs, step.pages, [0, n], [past + n], [keep], [len(keep)])
    need = {(past + i) // PAGE for i in keep} | {(past + j) // PAGE for j in range(len(keep))}
    gaps = [t for t in range(past // PAGE, (past + n - 1) // PAGE + 1) if t not in need]
    assert gaps
    for bad in (-1, step.n_pages, 2 ** 31 - 1):
        p = pages.clone()
        p[0, gaps] = bad
        cache = base._cache(bufs, Hkv, Hkv, D)
        ws = cache.new_workspace()
        out = cache.compact(kept, n_keep, q_off, kv_len, p, ws, max_q=n)
        assert cache.check(ws) == 0 and out.tolist() == lens
        assert moves._same(moves._values(cache), want)
    for t in sorted(need):          # one that is needed: left as it is, flagged
        p = pages.clone()
        p[0, t] = -1
        cache = base._cache(bufs, Hkv, Hkv, D)
        ws = cache.new_workspace()
        out = cache.compact(kept, n_keep, q_off, kv_len, p, ws, max_q=n)
        assert cache.check(ws) == binding.MOE_ERR_BAD_INDEX and out.tolist() == [past + n]
        assert torch.equal(cache.k.cpu(), bufs[0]) and torch.equal(cache.v.cpu(), bufs[1])


# ----------------------------------------------------------------------------- arguments
def test_compact_asks_for_no_max_q():
    """Nothing depends on it: left out, or any number."""
    step = base.Step([12, 3], [100, 67], seed=5)
    bufs = base._pool(step, 2, 128, seed=5)
    keep, n_keep = moves._table([[0, 4, 11], [1]])
    *want, lens = spec.compact(bufs, step.pages, step.q_off.tolist(), step.L, [[0, 4, 11], [1]], [3, 1])
    for more in ({}, dict(max_q=12), dict(max_q=1), dict(max_q=10 ** 6)):
        cache = base._cache(bufs, 2, 2, 128)
        ws = cache.new_workspace()
        assert cache.compact(keep, n_keep, *step.dev(), ws, **more).tolist() == lens and cache.check(ws) == 0
        assert moves._same(moves._values(cache), want)
