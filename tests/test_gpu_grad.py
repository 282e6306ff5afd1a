"""The gradient of the cosines about the stored values, against dense float64 products and
against differences of float64 losses. Bound of a unit value's gradient: float32 sums of at
most L products in a fixed tree whose longest path is L / 64 steps, 6 of the wave and one a
slice, each product of two values rounded once."""
import numpy as np
import pytest

import distill_oracle as do
import synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_embedding_exact_amd as sps
    sps.load_library()
    return torch, sps, torch.device("cuda:0")


def corpus(r, n, dim, per_row, zeros=True):
    """Host CSR with empty rows, a row of stored zeros and signed values."""
    indptr, ix, v = [0], [], []
    for i in range(n):
        k = min(dim, per_row(i))
        d = np.sort(r.choice(dim, k, replace=False))
        w = r.randn(k) + 0.1
        if zeros and i == n - 1:
            w[:] = 0
        elif k > 2:
            w[0] = 0.0  # a stored zero
        ix.append(d)
        v.append(w)
        indptr.append(indptr[-1] + k)
    cat = np.concatenate
    return synth.HostCSR(np.array(indptr, np.int32), cat(ix).astype(np.int32) if indptr[-1] else
                         np.zeros(0, np.int32), cat(v).astype(np.float32) if indptr[-1] else
                         np.zeros(0, np.float32), n, dim)


def dense(m):
    d = np.zeros((m.n_rows, m.n_cols))
    rows = np.repeat(np.arange(m.n_rows), np.diff(m.indptr))
    d[rows, m.indices] = m.values
    n = np.sqrt((d * d).sum(1))
    inv = np.divide(1.0, n, out=np.zeros_like(n), where=n > 0)
    return rows, d * inv[:, None], inv


def oracle(a, b, g, slices):
    """(dv, bound) of a's entries for G (a's rows, b's rows) float64."""
    rows, u, inv = dense(a)
    _, w, _ = dense(b)
    cols = a.indices
    du = (g @ w)[rows, cols]
    mag = (np.abs(g) @ np.abs(w))[rows, cols]
    count = (w != 0).sum(0)[cols]
    bar = mag * U * (count / 64 + 8 + 8 + slices + 2)
    uu = u[rows, cols]
    dot = np.bincount(rows, uu * du, a.n_rows)
    dot_bar = np.bincount(rows, np.abs(uu) * bar, a.n_rows)
    dv = (du - uu * dot[rows]) * inv[rows]
    return dv, (bar + np.abs(uu) * dot_bar[rows]) * inv[rows] + np.abs(dv) * U + 1e-38


def close(got, want, bar):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > bar
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], bar[bad][:5])


def by_chunks(env, rows, other, g, transposed, chunk_size):
    torch, sps, dev = env
    h = sps.prepare(other, min(chunk_size, max(other.n_rows, 1)))
    # a corpus without chunks starts no sums
    du = torch.full((rows.nnz,), float("nan") if h.num_chunks else 0.0, device=dev)
    for c in range(h.num_chunks):
        b = c * h.chunk_size
        part = g[b:b + h.chunk_size] if transposed else g[:, b:b + h.chunk_size]
        sps.cosine_chunk_grad(rows, h, c, part, du, transposed=transposed, first=c == 0)
    return sps.cosine_grad_values(rows, du)


SHAPES = [(1, 1, 5), (3, 7, 40), (17, 1023, 60), (8, 1025, 3000), (40, 3000, 20), (1030, 33, 90),
          (2100, 1100, 400), (3, 17000, 50), (9000, 5, 30), (0, 4, 9), (4, 0, 9)]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("nq,ni,dim", SHAPES)
def test_both_sides(env, dtype, nq, ni, dim):
    torch, sps, dev = env
    r = np.random.RandomState(nq + ni)
    q = corpus(r, nq, dim, lambda i: [5, 0, 12, 90, 1][i % 5])
    it = corpus(r, ni, dim, lambda i: [7, 20, 0, 3][i % 4])
    g = torch.from_numpy(r.randn(nq, ni).astype(np.float32)).to(getattr(torch, dtype)).to(dev)
    g64 = g.double().cpu().numpy()
    qc, ic = sps.CSR.from_host(q, dev), sps.CSR.from_host(it, dev)
    want_q, want_i = oracle(q, it, g64, ni // 256 + 4), oracle(it, q, g64.T, nq // 256 + 4)
    gq, gi = sps.cosine_grad(qc, ic, g)
    close(gq, *want_q)
    close(gi, *want_i)
    for cs in (4096, 1500, 700):  # by chunks of a prepared corpus
        close(by_chunks(env, qc, ic, g, False, cs), *want_q)
        close(by_chunks(env, ic, qc, g, True, cs), *want_i)


def test_shared_dims_and_long_rows(env):
    """Every row holds the same 100 dims (lists as long as a slice) and more than a wave's
    entries."""
    torch, sps, dev = env
    r = np.random.RandomState(0)
    q, it = corpus(r, 30, 150, lambda i: 150), corpus(r, 2500, 150, lambda i: 100 + i % 51)
    g = torch.randn(30, 2500, device=dev)
    qc, ic = sps.CSR.from_host(q, dev), sps.CSR.from_host(it, dev)
    gq, gi = sps.cosine_grad(qc, ic, g)
    g64 = g.double().cpu().numpy()
    want_q, want_i = oracle(q, it, g64, 3), oracle(it, q, g64.T, 3)
    close(gq, *want_q)
    close(gi, *want_i)
    close(by_chunks(env, qc, ic, g, False, 2500), *want_q)
    close(by_chunks(env, ic, qc, g, True, 30), *want_i)


@pytest.mark.parametrize("nq,ni", [(1030, 9000), (2050, 4100), (5000, 300)])
def test_lists_over_several_tiles(env, nq, ni):
    """Rows of a workgroup that share some long lists, not others, over several tiles of
    columns; a dim held only by items of the first columns."""
    torch, sps, dev = env
    r = np.random.RandomState(nq)

    def some(n, first):
        rows = []
        for i in range(n):
            d = np.nonzero(r.rand(40) < np.linspace(0.95, 0.02, 40))[0]
            if i % 7 == 3:
                d = d[d > 4]
            rows.append(np.concatenate([d, [40] if i < first else [], [41 + i % 50]]).astype(np.int32))
        ptr = np.concatenate([[0], np.cumsum([len(x) for x in rows])]).astype(np.int32)
        ix = np.concatenate(rows)
        return synth.HostCSR(ptr, ix, r.randn(len(ix)).astype(np.float32), n, 91)
    q, it = some(nq, nq), some(ni, 200)
    g = torch.from_numpy(r.randn(nq, ni).astype(np.float32)).to(dev)
    gq, gi = sps.cosine_grad(sps.CSR.from_host(q, dev), sps.CSR.from_host(it, dev), g)
    g64 = g.double().cpu().numpy()
    close(gq, *oracle(q, it, g64, ni // 256 + 4))
    close(gi, *oracle(it, q, g64.T, nq // 256 + 4))


def rests(n, this):
    """(this side, other side of n rows): dims whose lists of more than 128 entries leave 0, 1, 4
    or 5 behind the first tile of 4096 columns, in the next tile, in the last one or over both, or
    lie across the tiles' ends; each held by one row of this side and by five."""
    r = np.random.RandomState(n)
    lists = []
    for many in (129, 400):
        for k in (0, 1, 4, 5):
            for late in (np.arange(k) + 4097, n - 1 - np.arange(k),
                         np.where(np.arange(k) % 2, 5000 + np.arange(k), n - 1 - np.arange(k))):
                lists.append(np.unique(np.concatenate([r.choice(4096, many, replace=False), late])))
    lists += [np.arange(4090, 4290), np.arange(4096 - 130, 4097), np.r_[0:127, 4095, 4096, 8191],
              np.arange(8192 - 131, n), np.r_[4096:4224, n - 1], np.arange(0, n, 61)]
    dim = 2 * len(lists)
    rows = [[] for _ in range(n)]
    for d, x in enumerate(lists):
        for i in x:
            rows[i] += [2 * d, 2 * d + 1]
    other = from_rows(r, rows, dim)
    mine = from_rows(r, [[d for d in range(dim) if d % 2 or i == d // 2 % 6] if i < 6 else
                         [7 * i % dim] for i in range(this)], dim)
    return mine, other


def from_rows(r, rows, dim):
    ptr = np.concatenate([[0], np.cumsum([len(x) for x in rows])]).astype(np.int32)
    ix = np.concatenate([np.sort(np.array(x, np.int32)) for x in rows]).astype(np.int32)
    return synth.HostCSR(ptr, ix, r.randn(len(ix)).astype(np.float32), len(rows), dim)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("n,this", [(8193, 6), (9000, 9), (12289, 6), (16400, 7)])
def test_rests_of_lists_behind_a_tile(env, dtype, n, this):
    """A long list's last few entries lie tiles behind the others: each counts once, with its own
    column."""
    torch, sps, dev = env
    mine, other = rests(n, this)
    g = torch.from_numpy(np.random.RandomState(n).randn(this, n).astype(np.float32))
    g = g.to(getattr(torch, dtype)).to(dev)
    g64 = g.double().cpu().numpy()
    mc, oc = sps.CSR.from_host(mine, dev), sps.CSR.from_host(other, dev)
    want_m, want_o = oracle(mine, other, g64, n // 256 + 4), oracle(other, mine, g64.T, 4)
    for got_m, got_o in (sps.cosine_grad(mc, oc, g),                       # the queries' side
                         sps.cosine_grad(oc, mc, g.t().contiguous())[::-1]):  # the items'
        close(got_m, *want_m)
        close(got_o, *want_o)


def test_rows_of_many_entries(env):
    """Rows of more entries than are walked at a time, over more columns than a tile, dims up
    to the largest key."""
    torch, sps, dev = env
    r = np.random.RandomState(8)
    q, it = corpus(r, 4, 2000, lambda i: [1200, 0, 700, 3][i]), corpus(r, 9000, 2000, lambda i: i % 9)
    g = torch.randn(4, 9000, device=dev)
    g64 = g.double().cpu().numpy()
    want_q, want_i = oracle(q, it, g64, 40), oracle(it, q, g64.T, 40)
    for shift in (0, 2**31 - 2 - 2000):  # the same rows at the upper end of the dims
        for m in (q, it):
            m.indices += np.int32(shift)
            m.n_cols = 2000 + shift
        gq, gi = sps.cosine_grad(sps.CSR.from_host(q, dev), sps.CSR.from_host(it, dev), g)
        close(gq, *want_q)
        close(gi, *want_i)


def test_workload(env):
    """The skewed corpus of the page's shape, a part of it: sampled entries."""
    torch, sps, dev = env
    q, it, _ = synth.make_workload("mid", n_item=9000, n_query=300)
    g = torch.randn(300, 9000, device=dev) / 300
    gq, gi = sps.cosine_grad(sps.CSR.from_host(q, dev), sps.CSR.from_host(it, dev), g)
    import scipy.sparse as sp
    g64 = g.double().cpu().numpy()

    def check(a, b, g64, got):
        m = []
        for x in (a, b):
            rows = np.repeat(np.arange(x.n_rows), np.diff(x.indptr))
            v = x.values.astype(np.float64)
            inv = 1 / np.sqrt(np.bincount(rows, v * v, x.n_rows))
            m.append((sp.csr_matrix((v * inv[rows], x.indices, x.indptr), (x.n_rows, x.n_cols)), inv))
        (u, inv), (w, _) = m
        w = w.tocsc()
        got = got.double().cpu().numpy()
        for row in range(0, a.n_rows, max(1, a.n_rows // 25)):
            b0, e0 = a.indptr[row], a.indptr[row + 1]
            cols = w[:, a.indices[b0:e0]]
            du = cols.T @ g64[row]
            mag = abs(cols).T @ np.abs(g64[row])
            bar = mag * U * (cols.getnnz(0) / 64 + 40)
            uu = u.data[b0:e0]
            dv = (du - uu * (uu @ du)) * inv[row]
            lim = (bar + np.abs(uu) * (np.abs(uu) @ bar)) * inv[row] + np.abs(dv) * U
            assert (np.abs(got[b0:e0] - dv) <= lim).all()
    check(q, it, g64, gq)
    check(it, q, g64.T, gi)


def test_views_and_chunk_order(env):
    torch, sps, dev = env
    r = np.random.RandomState(2)
    q, it = corpus(r, 21, 100, lambda i: 20), corpus(r, 2100, 100, lambda i: 10)
    qc = sps.CSR.from_host(q, dev)
    h = sps.prepare(sps.CSR.from_host(it, dev), 1000)
    wide = torch.randn(21, 2200, device=dev)
    g = wide[:, 37:37 + 2100]
    want = oracle(q, it, g.double().cpu().numpy(), 4)
    for order in ([0, 1, 2], [2, 0, 1]):
        du = torch.full((q.nnz,), float("nan"), device=dev)
        for j, c in enumerate(order):
            sps.cosine_chunk_grad(qc, h, c, g[:, c * 1000:c * 1000 + h.chunk_len(c)], du, first=j == 0)
        out = sps.cosine_grad_values(qc, du)
        close(out, *want)
        close(sps.cosine_grad_values(qc, du, du), *want)


def test_reproducible_streams_and_graphs(env):
    torch, sps, dev = env
    r = np.random.RandomState(3)
    q, it = corpus(r, 50, 200, lambda i: 30), corpus(r, 3000, 200, lambda i: 25)
    qc = sps.CSR.from_host(q, dev)
    h = sps.prepare(sps.CSR.from_host(it, dev), 3000)
    g = torch.randn(50, 3000, device=dev)
    torch.cuda.synchronize()

    def step(out, stream=None):
        sps.cosine_chunk_grad(qc, h, 0, g, out, first=True, stream=stream)
        return sps.cosine_grad_values(qc, out, out, stream=stream)
    a = step(torch.empty(q.nnz, device=dev))
    for s in [torch.cuda.Stream() for _ in range(2)]:
        b = torch.empty(q.nnz, device=dev)
        torch.cuda.synchronize()
        step(b, s)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    ic = sps.CSR.from_host(it, dev)
    both = sps.cosine_grad(qc, ic, g)
    for s in [torch.cuda.Stream() for _ in range(2)]:
        again = sps.cosine_grad(qc, ic, g, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(both[0], again[0]) and torch.equal(both[1], again[1])
    out = torch.empty(q.nnz, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step(out)
        both = sps.cosine_grad(qc, ic, g)
    for i in range(4):
        g.copy_(torch.randn(50, 3000, device=dev))
        graph.replay()
        e = step(torch.empty(q.nnz, device=dev))
        fresh = sps.cosine_grad(qc, ic, g)
        torch.cuda.synchronize()
        assert torch.equal(out, e)
        assert torch.equal(both[0], fresh[0]) and torch.equal(both[1], fresh[1])


def test_faulty_other_side_scores_nothing(env):
    """A corpus whose structure is refused on the device holds no lists: gradient 0."""
    torch, sps, dev = env
    r = np.random.RandomState(4)
    q, it = corpus(r, 5, 50, lambda i: 9), corpus(r, 60, 50, lambda i: 9)
    it.indices[3] = 50  # outside the dims
    h = sps.prepare(sps.CSR.from_host(it, dev), 60)
    du = torch.ones(q.nnz, device=dev)
    sps.cosine_chunk_grad(sps.CSR.from_host(q, dev), h, 0, torch.ones(5, 60, device=dev), du, first=True)
    assert (du == 0).all()


def test_refusals(env):
    torch, sps, dev = env
    r = np.random.RandomState(5)
    q, it = corpus(r, 5, 50, lambda i: 9), corpus(r, 2060, 50, lambda i: 9)
    qc = sps.CSR.from_host(q, dev)
    h = sps.prepare(sps.CSR.from_host(it, dev), 2000)
    du = torch.zeros(q.nnz, device=dev)
    g = torch.ones(5, 2000, device=dev)
    other = sps.CSR.from_host(corpus(r, 5, 51, lambda i: 9), dev)
    for bad, status in ((lambda: sps.cosine_chunk_grad(qc, h, 2, g, du), -5),
                        (lambda: sps.cosine_chunk_grad(qc, h, -1, g, du), -5),
                        (lambda: sps.cosine_chunk_grad(qc, h, 1, g, du), -1),
                        (lambda: sps.cosine_chunk_grad(qc, h, 0, g, du, transposed=True), -1),
                        (lambda: sps.cosine_chunk_grad(qc, h, 0, g[:4], du), -1),
                        (lambda: sps.cosine_grad(qc, qc, g), -1), (lambda: sps.cosine_grad(qc, other, g[:, :5]), -3),
                        (lambda: sps.cosine_chunk_grad(other, h, 0, g, torch.zeros(other.nnz, device=dev)), -3)):
        with pytest.raises(sps.SpsError) as e:
            bad()
        assert e.value.status == status
    for bad in (lambda: sps.cosine_chunk_grad(qc, h, 0, g, du[1:]),
                lambda: sps.cosine_chunk_grad(qc, h, 0, g, du.double()),
                lambda: sps.cosine_grad(qc, qc, g.double()), lambda: sps.cosine_grad_values(qc, du, du[1:])):
        with pytest.raises(AssertionError):
            bad()


def test_distillation_of_a_corpus(env):
    """A whole step: teacher's lists, losses over all chunks, both gradients; against float64
    throughout, and against differences of float64 losses along random directions."""
    torch, sps, dev = env
    r = np.random.RandomState(6)
    q, it = corpus(r, 13, 300, lambda i: 20, False), corpus(r, 2500, 300, lambda i: [25, 0, 14][i % 3], False)
    qc, ic = sps.CSR.from_host(q, dev), sps.CSR.from_host(it, dev)
    tau, k = 0.1, 12
    ids = np.stack([r.choice(2500, k, replace=False) for _ in range(13)]).astype(np.int32)
    ids[3, 6:] = -1
    t = r.randn(13, k).astype(np.float32) * 0.2
    w = (r.rand(13) / 13).astype(np.float32)
    loss, gq, gi = sps.bulk_distill(qc, ic, torch.from_numpy(ids).to(dev), torch.from_numpy(t).to(dev),
                                    tau, row_weights=torch.from_numpy(w).to(dev), chunk_size=1100)

    def total(qv, iv):
        a = synth.HostCSR(q.indptr, q.indices, qv, 13, 300)
        b = synth.HostCSR(it.indptr, it.indices, iv, 2500, 300)
        s = dense(a)[1] @ dense(b)[1].T
        v = do.batch(s, ids, t, tau)
        return v[0], v[1] * w[:, None].astype(np.float64)
    qv, iv = q.values.astype(np.float64), it.values.astype(np.float64)
    l, g = total(qv, iv)
    # scores are within 2^-22 (two roundings of unit values, fixed point): z within 2^-22 / tau
    dz = 2.0 ** -22 / tau
    assert (np.abs(loss.double().cpu().numpy() - l) <= 2 * dz + 100 * U * (1 + np.abs(l))).all()
    # and the gradient about the scores within a factor 1 + 2 dz, listed columns by p as well
    for got, a, b, gg in ((gq, q, it, g), (gi, it, q, g.T)):
        rows, u, inv = dense(a)
        _, wn, _ = dense(b)
        want, bar = oracle(a, b, gg, 4)
        mag = (np.abs(gg) @ np.abs(wn))[rows, a.indices]
        slack = (mag + np.bincount(rows, np.abs(u[rows, a.indices]) * mag, a.n_rows)[rows]
                 * np.abs(u[rows, a.indices])) * inv[rows] * (2 * dz + 100 * U)
        listed = (w.max() / tau) * 2 * dz * inv[rows] * 4  # (q - p) where the two nearly cancel
        close(got, want, bar + slack + listed)
    h = 1e-4
    for side, got in ((0, gq), (1, gi)):
        v = r.randn(len((qv, iv)[side]))
        up = [qv, iv]
        dn = [qv, iv]
        up[side], dn[side] = up[side] + h * v, dn[side] - h * v
        diff = ((total(*up)[0] - total(*dn)[0]) * w).sum() / (2 * h)
        d = float((got.double().cpu().numpy() * v).sum())
        scale = float(np.abs(got.double().cpu().numpy() * v).sum())
        # h^2 of the third derivative along a unit-size direction; float32 work of many entries
        assert abs(diff - d) <= 1e-4 * scale + 1e-9


@pytest.mark.parametrize("nq,ni,per_row", [(0, 5, 3), (5, 0, 3), (0, 0, 3), (5, 7, 0), (1, 1, 1)])
def test_corpus_calls_of_nothing(env, nq, ni, per_row):
    """No queries, no items, no entries: best lists, losses and gradients of the same sizes."""
    torch, sps, dev = env
    r = np.random.RandomState(nq + ni)
    q, it = corpus(r, nq, 9, lambda i: per_row, False), corpus(r, ni, 9, lambda i: per_row, False)
    qc, ic = sps.CSR.from_host(q, dev), sps.CSR.from_host(it, dev)
    top = sps.bulk_select(qc, ic, 3)
    n = min(ni, 3)
    assert top.cols.shape == (nq, 3) and (top.cols[:, n:] == -1).all()
    assert (top.cols[:, :n] >= 0).all() and (top.scores[:, n:] == -np.inf).all()
    ids = torch.zeros(nq, 2, dtype=torch.int32, device=dev)
    loss, gq, gi = sps.bulk_distill(qc, ic, ids, torch.zeros(nq, 2, device=dev), 0.1)
    assert loss.shape == (nq,) and gq.shape == (qc.nnz,) and gi.shape == (ic.nnz,)
    scores = sps.bulk_similarity(qc, ic) if nq and ni else torch.zeros(nq, ni, device=dev)
    want, g, l_bound, _ = do.batch(scores.double().cpu().numpy(), ids.cpu().numpy(), np.zeros((nq, 2)), 0.1)
    assert (np.abs(loss.double().cpu().numpy() - want) <= l_bound + 4 * U).all()
    gq2, gi2 = sps.cosine_grad(qc, ic, torch.from_numpy(g.astype(np.float32)).view(nq, ni).to(dev))
    assert gq2.shape == gq.shape and gi2.shape == gi.shape
    for a in (gq, gi, gq2, gi2):
        assert torch.isfinite(a).all()
