"""The refusals of the entry points on dense rows, without a GPU: every call here returns its
documented status before any device work."""
import ctypes

import pytest
import torch

import sparse_embedding_exact_amd as sps
from test_rows_devices import calls, i32, on, Reached  # noqa: F401

INV, DIM, WS, OVF, UNS = -1, -3, -4, -6, -8
P = 1 << 40  # stands for a device address: never read


@pytest.fixture(scope="module")
def lib():
    return sps.load_library()


def view(data=P, dtype=0, rows=8, cols=100, ld=100, begin=0):
    return ctypes.byref(sps._Scores(data, dtype, rows, cols, ld, begin))


def rows8(values=2 * P, scales=3 * P, rows=8, dim=100, ld=112):
    return ctypes.byref(sps._Int8Rows(values, scales, rows, dim, ld))


BAD_VIEWS = [
    (dict(data=None), INV), (dict(dtype=3), INV), (dict(dtype=-1), INV), (dict(rows=-1), INV),
    (dict(cols=-1), INV), (dict(ld=99), INV), (dict(data=P + 2), INV), (dict(data=P + 1, dtype=1), INV),
    (dict(rows=2**31), OVF), (dict(cols=2**31, ld=2**31), OVF), (dict(ld=2**62), OVF),
]
BAD_ROWS8 = [
    (dict(values=None), INV), (dict(scales=None), INV), (dict(rows=-1), INV), (dict(dim=0), INV),
    (dict(dim=-5), INV), (dict(ld=96), INV), (dict(ld=104), INV), (dict(values=P + 8), INV),
    (dict(scales=P + 2), INV), (dict(rows=2**31), OVF), (dict(dim=131073, ld=131088), UNS),
    (dict(ld=2**23), OVF),
]


@pytest.mark.parametrize("kw,want", BAD_VIEWS)
def test_bad_views(lib, kw, want):
    n = ctypes.c_size_t()
    assert lib.sps_quantize_rows(view(**kw), 2 * P, 112, 3 * P, None) == want
    assert lib.sps_dense_ce_workspace_size(view(**kw), view(), 1, 1, ctypes.byref(n)) == want
    assert lib.sps_dense_ce_workspace_size(view(), view(**kw), 1, 1, ctypes.byref(n)) == want
    assert lib.sps_dense_ce(view(**kw), view(data=2 * P), P, None, 1.0, None, P, None, 0, None, 0, 0, P,
                            1 << 40, None) == want
    assert lib.sps_last_error_message()


@pytest.mark.parametrize("kw,want", BAD_ROWS8)
def test_bad_rows8(lib, kw, want):
    assert lib.sps_dequantize_rows(rows8(**kw), P, 0, 131088, None) == want
    assert lib.sps_int8_scores(rows8(**kw), rows8(), P, 0, 100, None) == want
    assert lib.sps_int8_scores(rows8(), rows8(**kw), P, 0, 100, None) == want


def test_int8_refusals(lib):
    assert lib.sps_quantize_rows(None, P, 112, P, None) == INV
    assert lib.sps_quantize_rows(view(), 2 * P, 96, 3 * P, None) == INV
    assert lib.sps_quantize_rows(view(), 2 * P, 120, 3 * P, None) == INV
    assert lib.sps_quantize_rows(view(), None, 112, 3 * P, None) == INV
    assert lib.sps_quantize_rows(view(), 2 * P, 112, None, None) == INV
    assert lib.sps_quantize_rows(view(cols=0, ld=0), 2 * P, 112, 3 * P, None) == INV
    assert lib.sps_quantize_rows(view(cols=131073, ld=131073), 2 * P, 131088, 3 * P, None) == UNS
    # integers in the rows themselves
    assert lib.sps_quantize_rows(view(), P + 16, 112, 3 * P, None) == INV
    assert b"overlap" in lib.sps_last_error_message()
    # scales in the rows, or in the integers
    assert lib.sps_quantize_rows(view(), 2 * P, 112, P + 16, None) == INV
    assert lib.sps_quantize_rows(view(), 2 * P, 112, 2 * P + 16, None) == INV
    assert b"overlap" in lib.sps_last_error_message()
    assert lib.sps_quantize_rows(view(rows=2**30, ld=100), 2**50, 112, 3 * P, None) == OVF
    assert lib.sps_dequantize_rows(None, P, 0, 100, None) == INV
    assert lib.sps_dequantize_rows(rows8(), P, 3, 100, None) == INV
    assert lib.sps_dequantize_rows(rows8(), P, 0, 99, None) == INV
    assert lib.sps_dequantize_rows(rows8(), None, 0, 100, None) == INV
    assert lib.sps_dequantize_rows(rows8(), 2 * P + 16, 0, 100, None) == INV
    assert lib.sps_dequantize_rows(rows8(), 3 * P, 0, 100, None) == INV
    assert lib.sps_int8_scores(None, rows8(), P, 0, 8, None) == INV
    assert lib.sps_int8_scores(rows8(), None, P, 0, 8, None) == INV
    assert lib.sps_int8_scores(rows8(), rows8(dim=99), P, 0, 8, None) == DIM
    assert lib.sps_int8_scores(rows8(), rows8(), P, 0, 7, None) == INV
    assert lib.sps_int8_scores(rows8(), rows8(), None, 0, 8, None) == INV
    assert lib.sps_int8_scores(rows8(), rows8(), P, 5, 8, None) == INV
    for at in (2 * P, 2 * P + 96, 3 * P + 28):  # scores in the integers or the scales
        assert lib.sps_int8_scores(rows8(), rows8(values=9 * P, scales=8 * P), at, 0, 8, None) == INV
        assert lib.sps_int8_scores(rows8(values=9 * P, scales=8 * P), rows8(), at, 0, 8, None) == INV
    assert lib.sps_int8_scores(rows8(rows=2**30), rows8(rows=2**30), 2**55, 0, 2**30, None) == OVF
    # nothing to do: no launch
    assert lib.sps_quantize_rows(view(rows=0), None, 112, None, None) == 0
    assert lib.sps_dequantize_rows(rows8(rows=0), None, 0, 100, None) == 0
    assert lib.sps_int8_scores(rows8(rows=0), rows8(), P, 0, 8, None) == 0
    assert lib.sps_int8_scores(rows8(), rows8(rows=0), P, 0, 8, None) == 0


def ce(lib, q=None, i=None, targets=4 * P, bias=None, tau=1.0, weights=None, loss=5 * P, gq=6 * P,
       ldq=100, gi=7 * P, ldi=100, dtype=0, ws=8 * P, size=1 << 40):
    return lib.sps_dense_ce(view() if q is None else q, view(data=2 * P) if i is None else i, targets,
                            bias, tau, weights, loss, gq, ldq, gi, ldi, dtype, ws, size, None)


def test_cross_entropy_refusals(lib):
    assert ce(lib, targets=None) == INV
    assert ce(lib, loss=None) == INV
    assert ce(lib, ws=None) == INV
    assert ce(lib, ws=8 * P + 128) == INV
    assert ce(lib, size=100) == WS
    for tau in (0.0, -1.0, 1e-7, 2e6, float("nan"), float("inf")):
        assert ce(lib, tau=tau) == INV
    assert ce(lib, q=view(dtype=1)) == INV
    assert ce(lib, q=view(dtype=1), i=view(dtype=2)) == INV
    assert ce(lib, q=view(cols=99)) == DIM
    assert ce(lib, q=view(cols=0), i=view(cols=0)) == INV
    assert ce(lib, ldq=99) == INV and ce(lib, ldi=99) == INV
    assert ce(lib, gq=6 * P + 2) == INV
    assert ce(lib, dtype=1) == INV  # float32 rows have float32 gradients
    assert ce(lib, q=view(dtype=1), i=view(dtype=1, data=2 * P), dtype=2) == INV
    for at in (P, P + 8 * 400 - 4, 2 * P + 4):  # gradients in the rows
        assert ce(lib, gq=at) == INV and ce(lib, gi=at) == INV
    assert ce(lib, gq=7 * P + 8) == INV  # and in each other
    for at in (P + 4, 2 * P + 4, 4 * P, 6 * P + 8, 7 * P + 8, 9 * P + 28, 10 * P):  # losses in anything
        assert ce(lib, loss=at, bias=9 * P, weights=10 * P) == INV
        assert b"losses" in lib.sps_last_error_message()
    assert ce(lib, q=view(cols=70000, ld=70000), i=view(cols=70000, ld=70000), gq=None, gi=None) == UNS
    assert ce(lib, i=view(rows=4000001), gq=None, gi=None) == UNS
    assert ce(lib, q=view(rows=4000001), gq=None, gi=None) == UNS
    assert ce(lib, q=view(rows=4000000, cols=65536, ld=65536), i=view(rows=4000000, cols=65536, ld=65536),
              gq=None, gi=None) == OVF  # more tiles than a launch has
    assert ce(lib, i=view(ld=2**22), gq=None, gi=None) == OVF


def test_cross_entropy_sizing(lib):
    n = ctypes.c_size_t()
    size = lambda **kw: (lib.sps_dense_ce_workspace_size(  # noqa: E731
        view(dtype=kw.get("dtype", 2), rows=kw["n"], cols=kw["d"], ld=kw["d"]),
        view(dtype=kw.get("dtype", 2), rows=kw["m"], cols=kw["d"], ld=kw["d"]), kw.get("gq", 1),
        kw.get("gi", 1), ctypes.byref(n)), n.value)[1]
    assert lib.sps_dense_ce_workspace_size(view(), view(), 1, 1, None) == INV
    assert size(n=0, m=10, d=8) == 0 and size(n=10, m=0, d=8) == 0
    # the logits never stand whole: rows that grow 16 times add their own size and statistics only
    small, large = size(n=8192, m=131072, d=64), size(n=131072, m=131072, d=64)
    assert large < 1.5 * small + 131072 * 64 * 8
    assert large < 0.1 * 131072 * 131072 * 2
    alone = size(n=131072, m=131072, d=64, gq=0, gi=0)
    assert alone < 2 ** 30
    assert size(n=100, m=1000, d=72, gi=0) < size(n=100, m=1000, d=72)
    for dt in (0, 1, 2):
        assert size(n=1, m=1, d=1, dtype=dt) > 0


@pytest.mark.parametrize("which", [None, 0, 1, 2, 3, 4])
def test_tensors_on_another_device(calls, monkeypatch, which):  # noqa: F811
    g = [1 if k == which else 0 for k in range(5)]
    want = Reached if which is None else AssertionError
    with pytest.raises(want):
        sps.dense_cross_entropy(on(g[0], 3, 8), on(g[1], 5, 8), i32(g[2], 3), 1.0, on(g[3], 5),
                                on(g[4], 3))
    rows = lambda a, b: sps.Int8Rows(on(a, 3, 16, dtype=torch.int8), on(b, 3), 9)  # noqa: E731
    with pytest.raises(want):
        sps.int8_scores(rows(g[0], g[1]), rows(g[2], g[3]), on(g[4], 3, 3))
    if which is not None:  # its buffers are real, on no GPU here
        with pytest.raises(want):
            sps.int8_select(rows(g[0], g[1]), rows(g[2], g[3] or g[4]), 2)
    with pytest.raises(want):
        sps.dequantize_rows(rows(g[0] or g[1], g[2] or g[3]), out=on(g[4], 3, 9))
    with pytest.raises(want):
        sps.quantize_rows(on(max(g), 3, 9))


def test_binding_refusals(calls):  # noqa: F811
    x, w, t = on(0, 3, 8), on(0, 5, 8), i32(0, 3)
    for bad in (lambda: sps.dense_cross_entropy(x, w.half(), t),
                lambda: sps.dense_cross_entropy(x, w, t.long()),
                lambda: sps.dense_cross_entropy(x, w, t[:2]),
                lambda: sps.dense_cross_entropy(x, w, t, bias=on(0, 4)),
                lambda: sps.dense_cross_entropy(x, w, t, row_weights=on(0, 3).double()),
                lambda: sps.dense_cross_entropy(x, w, t, need_grad="both"),
                lambda: sps.dense_cross_entropy(x, w, t, grad_dtype=torch.float16),
                lambda: sps.dense_cross_entropy(x.double(), w.double(), t),
                lambda: sps.quantize_rows(x.t()),
                lambda: sps.Int8Rows(on(0, 3, 8, dtype=torch.int8), on(0, 3), 8)._c(),
                lambda: sps.Int8Rows(on(0, 3, 16), on(0, 3), 8)._c(),
                lambda: sps.Int8Rows(on(0, 3, 16, dtype=torch.int8), on(0, 4), 8)._c()):
        with pytest.raises(AssertionError):
            bad()
