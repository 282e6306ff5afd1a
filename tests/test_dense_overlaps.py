"""Cross entropy of dense rows: what it writes shares no byte with what it reads, since both are
in use until the last piece of the rows is done. Without a GPU: every call here is refused."""
import ctypes

import pytest

from test_dense_abi import INV, P, WS, ce, lib, view  # noqa: F401

# 8 queries and 8 items of 100 float32 values; targets, bias and weights 32 bytes each
SMALL = dict(targets=4 * P, bias=9 * P, weights=10 * P)
GRAD = 8 * 100 * 4


@pytest.mark.parametrize("side", ["gq", "gi"])
@pytest.mark.parametrize("what", SMALL)
def test_gradients_in_what_is_read(lib, side, what):  # noqa: F811
    at = SMALL[what]
    for off in (0, 28, -4, 4 - GRAD):
        assert ce(lib, **SMALL, **{side: at + off}) == INV
        assert b"gradient" in lib.sps_last_error_message()
    for off in (32, -GRAD):  # beside it: only the size is wrong
        assert ce(lib, **SMALL, **{side: at + off}, size=100) == WS
    # a wider gradient, whose rows lie on both sides of it
    ld = "ldq" if side == "gq" else "ldi"
    assert ce(lib, **SMALL, **{side: at - 400, ld: 112}, size=100) == WS
    assert ce(lib, **SMALL, **{side: at - 396, ld: 112}) == INV


def need(lib, **kw):  # noqa: F811
    n = ctypes.c_size_t()
    assert lib.sps_dense_ce_workspace_size(view(), view(data=2 * P), 1, 1, ctypes.byref(n)) == 0
    return n.value


def test_a_workspace_in_any_argument(lib):  # noqa: F811
    size = need(lib)
    assert size % 256 == 0
    args = dict(SMALL, loss=5 * P, gq=6 * P, gi=7 * P)
    for at, many in ((P, GRAD), (2 * P, GRAD), (4 * P, 32), (9 * P, 32), (10 * P, 32), (5 * P, 32),
                     (6 * P, GRAD), (7 * P, GRAD)):
        last = (at + many - 1) // 256 * 256
        for ws in (at, last, at - size + 256):
            assert ce(lib, **args, ws=ws, size=size) == INV
            assert b"workspace" in lib.sps_last_error_message()
            assert ce(lib, **args, ws=ws, size=size - 1) == WS


def test_no_gradients_no_overlap(lib):  # noqa: F811
    assert ce(lib, **SMALL, gq=None, gi=None, size=100) == WS
    assert ce(lib, targets=4 * P, gq=9 * P, gi=10 * P, size=100) == WS
