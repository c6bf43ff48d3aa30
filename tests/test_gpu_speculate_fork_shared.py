"""moe_kv_fork where several children are left the page that a sequence's next token goes to.

Two that are left a partly filled one would write its tokens and its one scale both."""
import pytest
import torch

import test_gpu_layer_kv as base
import test_gpu_speculate_cache as moves
from quantized_moe_routed_gb300 import binding

pytestmark = pytest.mark.gpu
PAGE, i32 = moves.PAGE, moves.i32


def _fork(L, src, own, change=lambda table, spare: table):
    step, bufs, free = moves._pool_of(L, 2, 64, len(src), 5)
    cache = base._cache(bufs, 2, 2, 64)
    ws = cache.new_workspace()
    _, lens, table = step.dev()
    table = change(table, free[len(src)])
    fresh = [free[c] if o else -1 for c, o in enumerate(own)]
    p, n = cache.fork(i32(*src), i32(*fresh), lens, table, ws)
    assert torch.equal(cache.k.cpu()[free[len(src)]], bufs[0][free[len(src)]])
    return table.cpu(), fresh, p.cpu(), n.tolist(), cache.check(ws)


@pytest.mark.parametrize("L", [100, 1, 63, 65, 127])
def test_a_second_child_in_a_partly_filled_page_is_flagged(L):
    src, own = [0, 1, 0, 1, 0, 0], [False, False, True, True, False, False]
    table, fresh, p, n, status = _fork([L, 30], src, own)
    assert status == binding.MOE_ERR_BAD_INDEX
    for c, s in enumerate(src):
        if c in (4, 5):
            assert bool((p[c] == -1).all()) and n[c] == 0
        else:
            want = table[s].clone()
            if fresh[c] >= 0:
                want[[L, 30][s] // PAGE] = fresh[c]
            assert torch.equal(p[c], want) and n[c] == [L, 30][s]


def test_children_that_share_no_partly_filled_page_are_not():
    """A table that is full has no place for a next token; a next page is still to be given, whatever stands there."""
    table, _, p, n, status = _fork([128, 128], [0, 0, 1], [False] * 3, lambda t, _: t[:, :2].contiguous())
    assert status == 0 and n == [128] * 3 and torch.equal(p, table[[0, 0, 1]])
    for page in (-1, 0, 10 ** 6):
        def change(t, _):
            t[:, 2] = page
            return t
        table, _, p, n, status = _fork([128, 128], [1, 1, 1], [False] * 3, change)
        assert status == 0 and n == [128] * 3 and torch.equal(p, table[[1, 1, 1]])
    table, _, p, n, status = _fork([0, 5], [0, 0, 1], [False] * 3)     # nothing in it yet
    assert status == 0 and n == [0, 0, 5] and torch.equal(p, table[[0, 0, 1]])


def test_a_child_that_is_none_leaves_the_page_to_the_next():
    """An earlier child counts only if it goes on from the same sequence."""
    table, _, p, n, status = _fork([100, 30], [5, 0, 1], [False] * 3)
    assert status == binding.MOE_ERR_BAD_INDEX and n == [0, 100, 30]
    assert torch.equal(p[1:], table[[0, 1]])
