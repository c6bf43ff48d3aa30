"""moe_sample refuses outputs that share memory with its inputs or each other (no GPU needed: arguments are
refused before anything is queued)."""
import ctypes as C

import pytest

import test_speculate_host as host
from quantized_moe_routed_gb300 import layer
from test_speculate_host import lib  # noqa: F401  (a fixture)

OK, INVALID = host.OK, host.INVALID
L, U, S, O = 1 << 20, 1 << 24, 1 << 25, 1 << 26   # logits; u; settings; outputs: far apart


def _ask(lib, T=3, V=100, stride=128, bf16=0, u=U, t=None, k=None, p=None, mp=None, token=O, prob=O + 4096):  # noqa: F811
    lib.fake_device(0)
    lib.fake_clear()
    d = layer.moe_sample_desc(L, stride, bf16, T, V, u, t, 1.0, k, 0, p, 1.0, mp, 0.0, token, prob)
    st = lib.moe_sample(C.byref(d), None)
    assert lib.fake_queued() == (b"launch_sample " if st == OK else b"")
    return st


@pytest.mark.parametrize("name", ["token", "prob"])
@pytest.mark.parametrize("other", ["u", "t", "k", "p", "mp"])
def test_settings(lib, name, other):  # noqa: F811
    for off, st in ((0, INVALID), (8, INVALID), (-8, INVALID), (12, OK), (-12, OK)):
        assert _ask(lib, **{other: S, name: S + off}) == st, off


@pytest.mark.parametrize("name", ["token", "prob"])
@pytest.mark.parametrize("bf16", [0, 1])
def test_logits(lib, name, bf16):  # noqa: F811
    size = 2 if bf16 else 4
    row, step = size * 100, size * 128
    end = 2 * step + row
    for off, st in ((0, INVALID), (-12, OK), (-8, INVALID), (row - 4, INVALID), (row, OK), (step - 12, OK), (step - 8, INVALID),
                    (step + row, OK), (step + row - 4, INVALID), (2 * step - 12, OK), (2 * step - 8, INVALID), (2 * step, INVALID),
                    (end - 4, INVALID), (end, OK), (end + 4096, OK)):
        assert _ask(lib, bf16=bf16, **{name: L + off}) == st, off
    # outputs longer than the room between rows reach the next one
    assert _ask(lib, bf16=bf16, stride=102, **{name: L + row}) == INVALID


@pytest.mark.parametrize("stride", [1 << 40, 1 << 61, 1 << 62, (1 << 63) - 1])
def test_one_row_of_any_stride(lib, stride):  # noqa: F811
    assert _ask(lib, T=1, stride=stride) == OK
    assert _ask(lib, T=1, stride=stride, token=L + 396) == INVALID
    assert _ask(lib, T=1, stride=stride, token=L + 400) == OK


def test_outputs(lib):  # noqa: F811
    for off, st in ((0, INVALID), (8, INVALID), (-8, INVALID), (12, OK), (-12, OK)):
        assert _ask(lib, prob=O + off) == st, off
    assert _ask(lib, prob=None) == OK
    # no row: nothing is written
    assert _ask_empty(lib) == OK


def _ask_empty(lib):  # noqa: F811
    d = layer.moe_sample_desc(L, 128, 0, 0, 100, U, None, 1.0, None, 0, None, 1.0, None, 0.0, U, U)
    return lib.moe_sample(C.byref(d), None)
