"""The refusals of the entry points on rows of scores, without a GPU: every
call here returns its documented status before any device work."""
import ctypes
import random

import pytest
import torch

import sparse_embedding_exact_amd as sps

INV, WS, OVF = -1, -4, -6
P = 0x10000  # stands for a device address: never read


@pytest.fixture(scope="module")
def lib():
    return sps.load_library()


def view(data=P, dtype=0, rows=8, cols=100, ld=100, begin=0):
    return ctypes.byref(sps._Scores(data, dtype, rows, cols, ld, begin))


BAD_VIEWS = [
    (dict(data=None), INV), (dict(dtype=3), INV), (dict(dtype=-1), INV), (dict(rows=-1), INV),
    (dict(cols=-1), INV), (dict(begin=-1), INV), (dict(ld=99), INV), (dict(data=P + 2), INV),
    (dict(data=P + 1, dtype=1), INV), (dict(rows=2**31), OVF), (dict(cols=2**31, ld=2**31), OVF),
    (dict(begin=2**31 - 50), OVF), (dict(ld=2**62), OVF),
]


@pytest.mark.parametrize("kw,want", BAD_VIEWS)
def test_bad_views(lib, kw, want):
    assert lib.sps_select_chunk(view(**kw), None, 4, 1, P, P, P, 1 << 30, None) == want
    assert lib.sps_beam_select(view(**kw), None, 1, 4, P, P, P, P, 1 << 30, None) == want
    assert lib.sps_last_error_message()


@pytest.mark.parametrize("k", [0, -1, 257])
def test_bad_k(lib, k):
    n = ctypes.c_size_t()
    assert lib.sps_select_workspace_size(8, 100, k, ctypes.byref(n)) == INV
    assert lib.sps_beam_workspace_size(8, 100, 1, k, ctypes.byref(n)) == INV
    assert lib.sps_select_chunk(view(), None, k, 1, P, P, P, 1 << 30, None) == INV
    assert lib.sps_beam_select(view(), None, 1, k, P, P, P, P, 1 << 30, None) == INV
    assert lib.sps_beam_join(P, P, 8, k, 1, 4, P, P, P, None) == INV
    assert lib.sps_beam_join(P, P, 8, 4, 1, k, P, P, P, None) == INV


def test_select_refusals(lib):
    n = ctypes.c_size_t()
    assert lib.sps_select_workspace_size(8, 100, 4, None) == INV
    assert lib.sps_beam_workspace_size(8, 100, 1, 4, None) == INV
    assert lib.sps_select_workspace_size(-1, 100, 4, ctypes.byref(n)) == INV
    assert lib.sps_select_workspace_size(2**31, 100, 4, ctypes.byref(n)) == OVF
    assert lib.sps_select_chunk(None, None, 4, 1, P, P, None, 0, None) == INV
    assert lib.sps_select_chunk(view(), None, 4, 1, None, P, None, 0, None) == INV
    assert lib.sps_select_chunk(view(), None, 4, 1, P, None, None, 0, None) == INV
    # few long rows need a workspace
    wide = dict(rows=2, cols=100000, ld=100000)
    assert lib.sps_select_workspace_size(2, 100000, 4, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.sps_select_chunk(view(**wide), None, 4, 1, P, P, None, 0, None) == INV
    assert lib.sps_select_chunk(view(**wide), None, 4, 1, P, P, P, n.value - 1, None) == WS
    assert lib.sps_select_chunk(view(**wide), None, 4, 1, P, P, P + 8, n.value, None) == INV


def test_beam_refusals(lib):
    n = ctypes.c_size_t()
    assert lib.sps_beam_workspace_size(8, 100, 2, 4, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.sps_beam_workspace_size(8, 8192, 4, 4, ctypes.byref(n)) == 0 and n.value == 8 * 4 * 8
    for beams in (0, -1, 3):
        assert lib.sps_beam_workspace_size(8, 100, beams, 4, ctypes.byref(n)) == INV
        assert lib.sps_beam_select(view(), None, beams, 4, P, P, P, P, n.value, None) == INV
        assert lib.sps_beam_join(P, P, 8, 4, beams, 4, P, P, P, None) == INV
    assert lib.sps_beam_select(view(), None, 2, 4, None, P, P, P, n.value, None) == INV
    assert lib.sps_beam_select(view(), None, 2, 4, P, None, P, P, 0, None) == INV
    assert lib.sps_beam_select(view(), None, 2, 4, P, P, None, P, 0, None) == INV
    big = dict(cols=8192, ld=8192)
    assert lib.sps_beam_select(view(**big), None, 4, 4, P, P, P, P, 8 * 4 * 8 - 1, None) == WS
    assert lib.sps_beam_select(view(**big), None, 4, 4, P, P, P, None, 8 * 4 * 8, None) == INV
    assert lib.sps_beam_join(None, P, 8, 4, 2, 4, P, P, P, None) == INV
    assert lib.sps_beam_join(P, P, -8, 4, 2, 4, P, P, P, None) == INV
    assert lib.sps_beam_join(P, P, 2**31, 4, 2, 4, P, P, P, None) == OVF
    # more candidates in a group than a place can number
    assert lib.sps_beam_join(P, P, 2**30, 256, 2**30, 4, P, P, P, None) == OVF


def state(src=P, dst=2 * P, row=64, ss=64, ds=64):
    return (ctypes.c_int64 * 5)(src or 0, dst or 0, row, ss, ds)


@pytest.mark.parametrize("st,want", [
    (state(src=None), INV), (state(dst=None), INV), (state(row=-1), INV), (state(ss=63), INV),
    (state(ds=63), INV), (state(ss=2**62), OVF), (state(ds=2**62), OVF),
    (state(dst=P), INV), (state(dst=P + 7 * 64 + 63), INV), (state(dst=P - 7 * 64 - 63), INV),
])
def test_reorder_refusals(lib, st, want):
    assert lib.sps_reorder_states(ctypes.byref(st), 1, P, 8, 8, None) == want


def test_reorder_counts(lib):
    st = state()
    assert lib.sps_reorder_states(None, 1, P, 8, 8, None) == INV
    assert lib.sps_reorder_states(ctypes.byref(st), 1, None, 8, 8, None) == INV
    assert lib.sps_reorder_states(ctypes.byref(st), -1, P, 8, 8, None) == INV
    assert lib.sps_reorder_states(ctypes.byref(st), 1, P, -8, 8, None) == INV
    assert lib.sps_reorder_states(ctypes.byref(st), 1, P, 2**31, 8, None) == OVF
    # nothing to do: no launch
    assert lib.sps_reorder_states(ctypes.byref(st), 0, P, 8, 8, None) == 0
    assert lib.sps_reorder_states(ctypes.byref(st), 1, P, 0, 8, None) == 0
    # an output that overlaps another state's source
    two = (ctypes.c_int64 * 10)(*state(), *state(src=8 * P, dst=P + 64))
    assert lib.sps_reorder_states(two, 2, P, 8, 8, None) == INV


def test_reorder_outputs_that_overlap(lib):
    """Two outputs that share bytes would be written in no order."""
    for off, ds in ((0, 64), (8, 64), (-63, 64), (7 * 64 + 63, 64), (100, 128), (1, 65)):
        two = (ctypes.c_int64 * 10)(*state(src=0x100000, dst=0x900000, ds=ds),
                                    *state(src=0x200000, dst=0x900000 + off, ds=ds))
        assert lib.sps_reorder_states(two, 2, P, 8, 8, None) == INV, (off, ds)
    # nor may the parents be written over while they are read
    for at in (0x900000, 0x900000 - 28, 0x900000 + 7 * 64 + 60):
        one = state(src=0x100000, dst=0x900000)
        assert lib.sps_reorder_states(ctypes.byref(one), 1, at, 8, 8, None) == INV


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are accepted would launch")
def test_rows_that_share_bytes(lib):
    """Refused if and only if two rows share a byte; calls that are not refused end at the launch,
    for want of a GPU."""
    r = random.Random(0)
    counts = {}
    for i in range(30000):
        n_src, n_out, row = r.randint(0, 5), r.randint(1, 5), r.randint(0, 9)
        ss = r.randint(row, 15)
        ds = ss if r.random() < 0.5 else r.randint(row, 15)
        src, dst = P + r.randint(0, 120), P + 60
        shared = meet(src, n_src, row, ss, dst, n_out, row, ds)
        st = state(src=src, dst=dst, row=row, ss=ss, ds=ds)
        got = lib.sps_reorder_states(ctypes.byref(st), 1, P, n_out, n_src, None)
        assert (got == INV) == shared, (src - P, row, ss, ds, n_src, n_out)
        counts[ss == ds, shared] = counts.get((ss == ds, shared), 0) + 1
    assert min(counts.values()) > 2000 and len(counts) == 4


def meet(a, na, la, sa, b, nb, lb, sb):
    one = {a + i * sa + x for i in range(na) for x in range(la)}
    return any(b + j * sb + x in one for j in range(nb) for x in range(lb))


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are accepted would launch")
def test_gradient_beside_the_scores(lib):
    """A gradient may stand in other columns of the wide matrix that holds the scores."""
    both = set()
    for dtype, gtype in ((0, 0), (1, 1), (1, 0), (2, 2)):
        size, gsize = 2 if dtype else 4, 2 if gtype else 4
        for rows in (1, 2, 8):
            for ld in (100, 200, 201, 300, 400):
                for gld in (100, 150, ld, ld // 2, ld + 1):
                    for at in (-gld, -101, -100, -99, -50, 0, 50, 99, 100, 101, 200, 300, 301, 9 * ld):
                        g = P + at * gsize
                        same = at == 0 and dtype == gtype and (ld == gld or rows == 1)
                        want = gld < 100 or not same and meet(P, rows, 100 * size, ld * size, g, rows,
                                                              100 * gsize, gld * gsize)
                        got = rows_call(lib, view(rows=rows, ld=ld, dtype=dtype), grad=g, gtype=gtype, ld=gld)
                        assert (got == INV) == want, (dtype, gtype, rows, ld, gld, at)
                        both.add((want, ld * size == gld * gsize))
    assert len(both) == 4


def test_nothing_to_do(lib):
    assert lib.sps_select_chunk(view(rows=0, data=None), None, 4, 1, None, None, None, 0,
                                None) == 0
    assert lib.sps_beam_select(view(rows=0, data=None), None, 2, 4, None, None, None, None, 0,
                               None) == 0
    assert lib.sps_beam_join(None, None, 0, 4, 2, 4, None, None, None, None) == 0


def size(lib, n, k):
    b = ctypes.c_size_t()
    assert lib.sps_distill_workspace_size(n, k, ctypes.byref(b)) == 0
    return b.value


def test_distill_sizes(lib):
    b = ctypes.c_size_t()
    assert size(lib, 8, 16) >= 8 * 16 * 12
    for k in (0, -1, 1025):
        assert lib.sps_distill_workspace_size(8, k, ctypes.byref(b)) == INV
    assert lib.sps_distill_workspace_size(8, 16, None) == INV
    assert lib.sps_distill_workspace_size(-1, 16, ctypes.byref(b)) == INV
    assert lib.sps_distill_workspace_size(2**31, 16, ctypes.byref(b)) == OVF


def prepare(lib, ids=P, logits=P, lse=None, n=8, k=16, cols=100, tau=1.0, ws=P, bytes_=None):
    out = ctypes.c_void_p()
    bytes_ = 1 << 30 if bytes_ is None else bytes_
    st = lib.sps_distill_prepare(ids, logits, lse, n, k, cols, tau, ws, bytes_, None,
                                 ctypes.byref(out))
    assert out.value is None or st == 0
    if out.value is not None:
        lib.sps_distill_destroy(out)
    return st


BAD_LISTS = [
    (dict(ids=None), INV), (dict(logits=None), INV), (dict(n=-1), INV), (dict(k=0), INV),
    (dict(k=1025), INV), (dict(tau=0.0), INV), (dict(tau=-1.0), INV), (dict(tau=float("nan")), INV),
    (dict(tau=float("inf")), INV), (dict(tau=9e-7), INV), (dict(ws=None), INV),
    (dict(ws=P + 16), INV), (dict(bytes_=100), WS), (dict(n=2**31), OVF),
]


@pytest.mark.parametrize("kw,want", BAD_LISTS + [(dict(cols=-1), INV), (dict(cols=2**31), OVF)])
def test_distill_prepare_refusals(lib, kw, want):
    assert prepare(lib, **kw) == want


@pytest.mark.parametrize("kw,want", BAD_LISTS)
def test_distill_rows_refusals(lib, kw, want):
    a = dict(ids=P, logits=P, lse=None, n=8, k=16, tau=1.0, ws=P, bytes_=1 << 30)
    a.update(kw)
    assert lib.sps_distill_rows(view(rows=a["n"]), a["ids"], a["logits"], a["lse"], a["k"], a["tau"],
                                None, P, None, 0, 0, a["ws"], a["bytes_"], None) == want


def rows_size(lib, n, cols, k):
    b = ctypes.c_size_t()
    assert lib.sps_distill_rows_workspace_size(n, cols, k, ctypes.byref(b)) == 0
    return b.value


def test_distill_rows_sizes(lib):
    """Rows that one launch takes keep nothing in the workspace."""
    b = ctypes.c_size_t()
    for n, cols, k in ((8, 100, 16), (10000, 8192, 1024), (4, 32768, 1024), (128, 10**6, 64)):
        assert rows_size(lib, n, cols, k) == 256
        if not torch.cuda.is_available():  # accepted: ends at the launch, for want of a GPU
            st = lib.sps_distill_rows(view(rows=n, cols=cols, ld=cols), P, P, None, k, 1.0, None, P, None,
                                      0, 0, P, 256, None)
            assert st not in (0, INV, WS, OVF)
    for n, cols, k in ((4, 32769, 16), (127, 10**6, 1024)):
        assert rows_size(lib, n, cols, k) == size(lib, n, k)
        assert lib.sps_distill_rows(view(rows=n, cols=cols, ld=cols), P, P, None, k, 1.0, None, P, None, 0,
                                    0, P, size(lib, n, k) - 1, None) == WS
    assert rows_size(lib, 0, 100, 16) == 0
    assert lib.sps_distill_rows(view(rows=0, data=None), None, None, None, 16, 1.0, None, None, None, 0, 0,
                                None, 0, None) == 0
    for n, cols, k, want in ((-1, 9, 4, INV), (9, -1, 4, INV), (9, 9, 0, INV), (9, 9, 1025, INV),
                             (2**31, 9, 4, OVF), (9, 2**31, 4, OVF), (2**23, 9, 4, OVF)):
        assert lib.sps_distill_rows_workspace_size(n, cols, k, ctypes.byref(b)) == want
    assert lib.sps_distill_rows_workspace_size(9, 9, 4, None) == INV


def rows_call(lib, v, loss=P, grad=None, gtype=0, ld=100):
    return lib.sps_distill_rows(v, P, P, None, 16, 1.0, None, loss, grad, gtype, ld, P, 1 << 30, None)


def test_distill_rows_outputs(lib):
    for kw, want in BAD_VIEWS:
        if kw not in (dict(begin=2**31 - 50),):
            assert rows_call(lib, view(**kw)) == want, kw
    assert rows_call(lib, view(begin=1)) == INV
    assert rows_call(lib, view(), loss=None) == INV
    g = 64 * P
    assert rows_call(lib, view(), grad=g, gtype=1) == INV            # fp16 about fp32 scores
    assert rows_call(lib, view(dtype=1), grad=g, gtype=2) == INV
    assert rows_call(lib, view(), grad=g, ld=99) == INV
    assert rows_call(lib, view(), grad=g + 2) == INV
    assert rows_call(lib, view(), grad=P + 4) == INV                 # overlaps the scores
    assert rows_call(lib, view(), grad=P, ld=101) == INV
    assert rows_call(lib, view(dtype=1), grad=P, gtype=0) == INV     # in place, wider type
    assert rows_call(lib, view(), grad=g, ld=2**62) == OVF


def test_distill_null_handles(lib):
    assert lib.sps_distill_chunk(None, view(), 1, None) == INV
    assert lib.sps_distill_loss(None, P, None, None) == INV
    assert lib.sps_distill_chunk_grad(None, view(), None, P, 0, 100, None) == INV
    lib.sps_distill_destroy(None)


def csr(n=4, cols=50, nnz=9, indptr=P, indices=P, values=P):
    return ctypes.byref(sps._Csr(n, cols, nnz, indptr, indices, values))


BAD_CSR = [(dict(n=-1), INV), (dict(cols=0), INV), (dict(nnz=-1), INV), (dict(indptr=None), INV),
           (dict(indices=None), INV), (dict(values=None), INV), (dict(n=2**31), OVF),
           (dict(nnz=2**31), OVF), (dict(cols=2**31), OVF)]


@pytest.mark.parametrize("kw,want", BAD_CSR)
def test_grad_bad_csr(lib, kw, want):
    # the CSR is looked at before the other side's handle
    assert lib.sps_cosine_grad(csr(**kw), None, 0, view(), 0, 1, P, None, 0, None) == want
    assert lib.sps_cosine_grad_values(csr(**kw), P, P, None) == want


def test_grad_refusals(lib):
    n = ctypes.c_size_t()
    assert lib.sps_cosine_grad_workspace_size(5, None, ctypes.byref(n)) == INV
    assert lib.sps_cosine_grad_workspace_size(5, None, None) == INV
    assert lib.sps_cosine_grad(None, None, 0, view(), 0, 1, P, None, 0, None) == INV
    assert lib.sps_cosine_grad(csr(), None, 0, view(), 0, 1, P, None, 0, None) == INV
    assert lib.sps_cosine_grad_values(None, P, P, None) == INV
    assert lib.sps_cosine_grad_values(csr(), None, P, None) == INV
    assert lib.sps_cosine_grad_values(csr(), P, None, None) == INV
    assert lib.sps_cosine_grad_values(csr(n=0, nnz=0, indices=None, values=None), None, None,
                                      None) == 0


@pytest.mark.parametrize("kw,want", BAD_CSR)
def test_both_bad_csr(lib, kw, want):
    both = lib.sps_cosine_grad_both
    assert both(csr(**kw), csr(), view(rows=4, cols=4), P, P, P, 1 << 30, None) == want
    assert both(csr(), csr(**kw), view(rows=4, cols=4), P, P, P, 1 << 30, None) == want


def test_both_refusals(lib):
    n = ctypes.c_size_t()
    sizes = lib.sps_cosine_grad_both_workspace_size
    assert sizes(5, 5, None) == INV and sizes(-1, 5, ctypes.byref(n)) == INV
    assert sizes(2**31 - 70000, 9000, ctypes.byref(n)) == OVF and sizes(2**31, 9, ctypes.byref(n)) == OVF
    assert sizes(9, 9, ctypes.byref(n)) == 0
    v = view(rows=4, cols=4)
    both = lib.sps_cosine_grad_both
    assert both(None, csr(), v, P, P, P, n.value, None) == INV
    assert both(csr(), csr(), None, P, P, P, n.value, None) == INV
    assert both(csr(), csr(cols=51), v, P, P, P, n.value, None) == -3
    assert both(csr(), csr(n=5), v, P, P, P, n.value, None) == INV
    assert both(csr(), csr(), v, None, P, P, n.value, None) == INV
    assert both(csr(), csr(), v, P, None, P, n.value, None) == INV
    assert both(csr(), csr(), v, P, P, None, n.value, None) == INV
    assert both(csr(), csr(), v, P, P, P, n.value - 1, None) == WS
    assert both(csr(), csr(), v, P, P, P + 16, n.value, None) == INV
    empty = dict(nnz=0, indices=None, values=None)
    assert both(csr(**empty), csr(**empty), v, None, None, None, 0, None) == 0


def test_launch_limits(lib):
    """Sizes within 31 bits whose launches would count their threads past 32: refused."""
    n = ctypes.c_size_t()
    many = dict(rows=2**25, cols=1, ld=1)
    assert lib.sps_select_chunk(view(**many), None, 1, 1, P, P, None, 0, None) == OVF
    assert lib.sps_beam_select(view(**many), None, 1, 1, P, P, P, None, 0, None) == OVF
    assert lib.sps_beam_join(P, P, 2**25, 1, 1, 1, P, P, P, None) == OVF
    assert lib.sps_distill_workspace_size(2**23, 1, ctypes.byref(n)) == OVF
    st = state(row=1, ss=1, ds=1, src=P, dst=2**40)
    assert lib.sps_reorder_states(ctypes.byref(st), 1, P, 2**30, 8, None) == OVF
    assert lib.sps_cosine_grad_values(csr(n=2**27), P, P, None) == OVF
    wide = view(rows=4, cols=2**29, ld=2**29)
    assert lib.sps_cosine_grad_both(csr(), csr(n=2**29), wide, P, P, P, 1 << 40, None) == OVF
