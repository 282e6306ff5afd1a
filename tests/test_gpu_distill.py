"""Distillation from a teacher's top list against the float64 oracle, within the bounds
that the oracle derives for float32 work, plus half a step of each output's type."""
import numpy as np
import pytest

import distill_oracle as do
import synth

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_embedding_exact_amd as sps
    sps.load_library()
    return torch, sps, torch.device("cuda:0")


def make(env, rows, cols, k, dtype, seed, spread=3.0):
    torch, _, dev = env
    r = np.random.RandomState(seed)
    x = torch.from_numpy((r.randn(rows, cols) * spread).astype(np.float32)).to(getattr(torch, dtype))
    ids = np.full((rows, k), -1, np.int32)
    for i in range(rows):
        n = min(k, cols, 1 + r.randint(k))
        ids[i, :n] = r.choice(cols, n, replace=False)
    t = (r.randn(rows, k) * spread).astype(np.float32)
    w = r.rand(rows).astype(np.float32)
    return x.to(dev), ids, t, w


def dev_of(env, a):
    return None if a is None else env[0].from_numpy(a).to(env[2])


def compare(env, loss, grad, x, ids, t, tau, lse, w, rows=None):
    torch = env[0]
    rows = range(len(ids)) if rows is None else rows
    x64 = x[list(rows)].double().cpu().numpy()
    want = do.batch(x64, ids[list(rows)], t[list(rows)], tau, None if lse is None else lse[list(rows)])
    got_l = loss.double().cpu().numpy()[list(rows)]
    same = np.isnan(want[0]) & np.isnan(got_l)
    with np.errstate(invalid="ignore"):
        close = np.abs(got_l - want[0]) <= want[2] + 1e-37
    assert (same | close | (got_l == want[0])).all(), (got_l, want[0], want[2])
    if grad is None:
        return
    ww = np.ones(len(want[0])) if w is None else w[list(rows)].astype(np.float64)
    g = want[1] * ww[:, None]
    info = torch.finfo(grad.dtype)
    # half a step, and below the smallest normal half of the smallest subnormal; products of the
    # factors below float32's smallest normal may be flushed
    bar = want[3] * ww[:, None] + np.abs(g) * (info.eps / 2 + 2 * do.U) + info.tiny * info.eps / 2 \
        + 2.0 ** -126 * (1 + ww[:, None] / tau)
    got = grad[list(rows)].double().cpu().numpy()
    big = np.abs(g) > info.max  # a gradient past the type's range is its infinity
    with np.errstate(invalid="ignore"):
        ok = np.abs(got - g) <= bar
    ok |= np.isnan(got) & np.isnan(g)
    ok |= big & np.isinf(got)
    worst = np.nanmax(np.where(ok, 0, np.abs(got - g) / bar)) if not ok.all() else 0
    assert ok.all(), (np.argwhere(~ok)[:5], got[~ok][:5], g[~ok][:5], worst)


def teacher_lse(ids, t, tau, n_cols, outside, seed):
    r = np.random.RandomState(seed)
    out = np.zeros(len(ids), np.float32)
    for i in range(len(ids)):
        c, v = do.entries(ids[i], t[i], n_cols)
        if len(c):
            out[i] = np.log(np.exp(v / tau - (v / tau).max()).sum()) + (v / tau).max() \
                - np.log1p(-outside * r.rand())
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("rows,cols,k,tau", [(3, 1, 1, 1.0), (5, 7, 3, 0.5), (4, 255, 64, 1.0),
                                             (6, 1000, 8, 0.05), (3, 8192, 100, 2.0),
                                             (7, 8193, 33, 1.0), (2, 40000, 1024, 3.0),
                                             (1030, 300, 5, 0.7)])
def test_whole_rows(env, dtype, rest, rows, cols, k, tau):
    torch, sps, dev = env
    x, ids, t, w = make(env, rows, cols, k, dtype, rows + cols, 3.0 * min(tau, 1.0))
    lse = teacher_lse(ids, t, tau, cols, 0.6, 1) if rest else None
    args = (dev_of(env, ids), dev_of(env, t), tau, dev_of(env, lse))
    loss, grad = sps.distill(x, *args, row_weights=dev_of(env, w))
    compare(env, loss, grad, x, ids, t, tau, lse, w)
    loss2, none = sps.distill(x, *args, need_grad=False)
    assert none is None and torch.equal(loss, loss2)
    out = torch.empty(rows, cols, device=dev)
    _, g32 = sps.distill(x, *args, out=out)
    assert g32 is out
    compare(env, loss, g32, x, ids, t, tau, lse, None)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("rows", [5, 1100])
def test_chunks(env, dtype, rest, rows):
    """Chunks of uneven widths in two orders, one of them empty; gradients in place."""
    torch, sps, dev = env
    cols, k, tau = 20000 if rows == 5 else 900, 40, 0.8
    x, ids, t, w = make(env, rows, cols, k, dtype, 3, 2.0)
    lse = teacher_lse(ids, t, tau, cols, 0.6, 1) if rest else None
    cuts = [0, 3, 3, cols // 2 - 1, cols - 1, cols]
    d = sps.distill_prepare(dev_of(env, ids), dev_of(env, t), cols, tau, dev_of(env, lse))
    for order in ([0, 1, 2, 3, 4], [3, 0, 4, 2, 1]):
        for j, c in enumerate(order):
            sps.distill_chunk(d, x[:, cuts[c]:cuts[c + 1]], cuts[c], first=j == 0)
        loss, slse = sps.distill_loss(d, return_lse=True)
        g = x.clone()
        for c in order:
            part = g[:, cuts[c]:cuts[c + 1]]
            assert sps.distill_chunk_grad(d, part, cuts[c], dev_of(env, w), out=part) is part
        compare(env, loss, g, x, ids, t, tau, lse, w, range(min(rows, 64)))
        ref = torch.logsumexp(x.double() / tau, 1)
        # 40 U of the sum, 3 U of exponents that reach |x - m| / tau <= 40 / ln 2
        assert float((slse.double() - ref).abs().max()) <= do.U * (160 + float(ref.abs().max()))


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("rows", [2559, 2560, 2573])
def test_chunks_of_many_rows(env, rest, rows):
    """About 64 rows an entry of the list; lists with no entry and rows with no score among them,
    the last rows too."""
    torch, sps, dev = env
    cols, k, tau = 150, 40, 1.5
    x, ids, t, w = make(env, rows, cols, k, "float32", 17)
    ids[5::7] = -1
    x[3::11, 2:] = -np.inf
    x[4::11] = -np.inf
    ids[rows - 2] = -1
    lse = teacher_lse(ids, t, tau, cols, 0.6, 1) if rest else None
    d = sps.distill_prepare(dev_of(env, ids), dev_of(env, t), cols, tau, dev_of(env, lse))
    cuts = ((0, 80), (80, cols))
    for c0, c1 in cuts:
        sps.distill_chunk(d, x[:, c0:c1], c0, first=c0 == 0)
    loss = sps.distill_loss(d)
    g = torch.empty_like(x)
    for c0, c1 in cuts:
        sps.distill_chunk_grad(d, x[:, c0:c1], c0, dev_of(env, w), out=g[:, c0:c1])
    compare(env, loss, g, x, ids, t, tau, lse, w, [*range(96), *range(rows - 40, rows)])


def test_long_rows_of_many(env):
    """Rows longer than the columns whose list bits fit LDS at a time."""
    torch, sps, dev = env
    rows, cols, k = 1030, 66001, 16
    x = torch.randn(rows, cols, device=dev, generator=torch.Generator(dev).manual_seed(1)).to(torch.bfloat16)
    r = np.random.RandomState(1)
    ids = (r.randint(0, cols // k - 1, (rows, 1)) + np.arange(k) * (cols // k)).astype(np.int32)
    ids[:, -1] = cols - 1
    t = r.randn(rows, k).astype(np.float32)
    lse = teacher_lse(ids, t, 1.0, cols, 0.6, 1)
    loss, grad = sps.distill(x, dev_of(env, ids), dev_of(env, t), 1.0, dev_of(env, lse))
    compare(env, loss, grad, x, ids, t, 1.0, lse, None, [0, 1, 511, 1029])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rest", [False, True])
def test_masks_and_odd_lists(env, dtype, rest):
    torch, sps, dev = env
    low = float(torch.finfo(getattr(torch, dtype)).min)
    cols, k, tau = 3001, 6, 0.5
    x, ids, t, w = make(env, 14, cols, k, dtype, 4, 1.0)
    ids[:] = np.arange(k) * 17 + 5
    x[0] = -np.inf                      # nothing left of the row
    x[1] = low                          # masked by the lowest value throughout: uniform
    x[2, 100:] = low                    # mostly
    x[3, 100:] = -np.inf
    x[4, :] = -np.inf
    x[4, ids[4, 0]] = 1.0               # nothing outside the list (and listed ones at -inf)
    x[5, ids[5, 2]] = -np.inf           # a listed one struck out
    x[6, 50] = np.nan
    x[7, ids[7, 1]] = np.nan
    x[8, 60] = np.inf
    ids[9] = -1                         # an empty list
    ids[10] = [5, 5, -7, cols, 22, 5]   # repeated, outside
    t[11] = -np.inf                     # no logit
    t[12, 1:] = -np.inf
    t[13, 2] = np.nan
    lse = None
    if rest:
        lse = np.full(14, 9.0, np.float32)
        lse[2] = -2.0                   # the list's mass is above 1: nothing outside it
    loss, grad = sps.distill(x, dev_of(env, ids), dev_of(env, t), tau, dev_of(env, lse),
                             row_weights=dev_of(env, w))
    rows = [i for i in range(14) if not (rest and i == 4)]
    compare(env, loss, grad, x, ids, t, tau, lse, w, [i for i in rows if i not in (6, 7, 8, 13)])
    for i in (6, 7, 8, 13):             # NaN and +inf: their own rows, whole
        assert torch.isnan(loss[i]) and torch.isnan(grad[i]).all()
    for i in (0, 9, 11):
        assert loss[i] == 0 and (grad[i] == 0).all()
    if rest:                            # a class with teacher's mass and none of the student's
        assert torch.isinf(loss[4]) and loss[4] > 0 and torch.isfinite(grad[4]).all()


@pytest.mark.parametrize("chunked", [False, True])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("cols", [700, 40000])
def test_list_far_above_the_rest(env, chunked, rest, cols):
    """A sharp student: what lies outside the list is e^-150 to e^-400 of the whole, below
    float32's range, and still a class of its own with a finite loss; and far below the list
    in the other direction."""
    torch, sps, dev = env
    x, ids, t, w = make(env, 6, cols, 4, "float32", 9, 0.01)
    ids[:] = np.arange(4) * 31
    tau = 0.01
    for i, gap in enumerate((1.5, 2.5, 4.0, -1.5, -4.0, 0.0)):
        x[i, ids[i]] += gap
    t *= 0.01
    lse = teacher_lse(ids, t, tau, cols, 0.6, 1) if rest else None
    a = (dev_of(env, ids), dev_of(env, t))
    if chunked:
        d = sps.distill_prepare(*a, cols, tau, dev_of(env, lse))
        sps.distill_chunk(d, x[:, :300], 0, first=True)
        sps.distill_chunk(d, x[:, 300:], 300)
        loss = sps.distill_loss(d)
        grad = torch.cat([sps.distill_chunk_grad(d, x[:, :300], 0, dev_of(env, w)),
                          sps.distill_chunk_grad(d, x[:, 300:], 300, dev_of(env, w))], 1)
    else:
        loss, grad = sps.distill(x, *a, tau, dev_of(env, lse), row_weights=dev_of(env, w))
    assert torch.isfinite(loss).all() and torch.isfinite(grad).all()
    compare(env, loss, grad, x, ids, t, tau, lse, w)


def test_strides(env):
    torch, sps, dev = env
    for dtype in TYPES:
        wide, ids, t, w = make(env, 4, 5000, 9, dtype, 8, 1.0)
        ids = np.minimum(ids, 1000)
        for a, b in ((1, 4999), (3, 2060), (7, 1010)):
            x = wide[:, a:b]
            out = torch.full((4, 6000), 7.0, device=dev, dtype=x.dtype)
            loss, grad = sps.distill(x, dev_of(env, ids), dev_of(env, t), 0.9, out=out[:, 5:5 + b - a])
            compare(env, loss, grad, x, ids, t, 0.9, None, None)
            assert (out[:, :5] == 7).all() and (out[:, 5 + b - a:] == 7).all()


def test_gradient_beside_the_scores(env):
    """Scores and their gradient in one wide matrix, chunk by chunk and whole."""
    torch, sps, dev = env
    for dtype in TYPES:
        x, ids, t, w = make(env, 5, 700, 9, dtype, 21, 1.0)
        a = (dev_of(env, ids), dev_of(env, t))
        wide = torch.full((5, 1501), 3.0, device=dev, dtype=x.dtype)
        wide[:, 1:701] = x
        loss, g = sps.distill(wide[:, 1:701], *a, 0.8, out=wide[:, 701:1401])
        compare(env, loss, g, x, ids, t, 0.8, None, None)
        assert torch.equal(wide[:, 1:701], x) and (wide[:, 1401:] == 3).all() and (wide[:, 0] == 3).all()
        d = sps.distill_prepare(*a, 700, 0.8)
        sps.distill_chunk(d, wide[:, 1:701], 0, first=True)
        loss = sps.distill_loss(d)
        sps.distill_chunk_grad(d, wide[:, 1:701], 0, out=wide[:, 701:1401])
        compare(env, loss, g, x, ids, t, 0.8, None, None)
        assert torch.equal(wide[:, 1:701], x) and (wide[:, 1401:] == 3).all()


@pytest.mark.parametrize("chunked", [False, True])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("cols", [700, 40000])
def test_masses_below_float32(env, chunked, rest, cols):
    """A sharp teacher's last entries have masses of e^-50 to e^-700: next to nothing where the
    student has the column, an infinite loss where it is struck out."""
    torch, sps, dev = env
    x, ids, t, w = make(env, 7, cols, 4, "float32", 13, 0.05)
    ids[:] = np.arange(4) * 31
    tau = 0.01
    t[:] = [0.0, -0.02, -0.01, 0.0]
    for i, gap in enumerate((0.5, 0.85, 0.95, 1.05, 1.5, 7.0, 1.5)):
        t[i, 3] = -gap
        if i < 6:
            x[i, ids[i, 3]] = -np.inf
    lse = teacher_lse(ids, t, tau, cols, 0.6, 1) if rest else None
    a = (dev_of(env, ids), dev_of(env, t))
    if chunked:
        d = sps.distill_prepare(*a, cols, tau, dev_of(env, lse))
        sps.distill_chunk(d, x[:, :300], 0, first=True)
        sps.distill_chunk(d, x[:, 300:], 300)
        loss = sps.distill_loss(d)
        grad = torch.cat([sps.distill_chunk_grad(d, x[:, :300], 0, dev_of(env, w)),
                          sps.distill_chunk_grad(d, x[:, 300:], 300, dev_of(env, w))], 1)
    else:
        loss, grad = sps.distill(x, *a, tau, dev_of(env, lse), row_weights=dev_of(env, w))
    assert (loss[:6] == np.inf).all() and torch.isfinite(loss[6]) and torch.isfinite(grad).all()
    # the temperature is a float32 (a mass of e^-50 moves by 50 parts in 2^25 with its rounding,
    # which is the definition's, not an error)
    compare(env, loss, grad, x, ids, t, float(np.float32(tau)), lse, w)


def test_memory_of_whole_rows(env):
    """Rows in one launch need their outputs' memory, not the lists' again."""
    torch, sps, dev = env
    x, ids, t, _ = make(env, 600, 2000, 1024, "float32", 6, 1.0)
    a = (dev_of(env, ids), dev_of(env, t))
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    loss, grad = sps.distill(x, *a, 0.8)
    more = torch.cuda.max_memory_allocated() - before
    # torch counts whole blocks: of 512 bytes up to 1 MiB, above it (the gradient) a kept block
    # whose rest below 1 MiB is not cut off. The lists' workspace would be 7.4 MB
    assert more <= grad.numel() * 4 + loss.numel() * 4 + 2**20 + 8192
    compare(env, loss, grad, x, ids, t, 0.8, None, None, range(4))


def test_against_differences(env):
    """The kernels' gradient against differences of the kernels' own losses: a step of 2^-4
    changes float32 losses near 5 by parts that float32 still resolves."""
    torch, sps, dev = env
    x, ids, t, _ = make(env, 2, 50, 6, "float32", 2, 1.0)
    ids[:] = np.arange(6) * 5
    a = (dev_of(env, ids), dev_of(env, t), 1.0)
    loss, grad = sps.distill(x, *a)
    h = 2.0 ** -4
    for j in (0, 3, 5, 25, 49):
        up, dn = x.clone(), x.clone()
        up[:, j] += h
        dn[:, j] -= h
        lu, ld = (sps.distill(v, *a, need_grad=False)[0].double() for v in (up, dn))
        d = (lu - ld) / (2 * h)
        # third derivative of log-sum-exp: at most 1/6 of h^2 / 6; two losses below 8 off by 64 U
        bar = h * h / 36 + 2 * 64 * do.U * 8 / (2 * h)
        assert float((d - grad[:, j].double()).abs().max()) <= bar


def test_reproducible_streams_and_graphs(env):
    torch, sps, dev = env
    x, ids, t, w = make(env, 6, 30000, 50, "float16", 5, 2.0)
    a = (dev_of(env, ids), dev_of(env, t), 0.7)
    l0, g0 = sps.distill(x, *a)
    torch.cuda.synchronize()
    for s in [torch.cuda.Stream() for _ in range(2)]:
        l1, g1 = sps.distill(x, *a, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(l0, l1) and torch.equal(g0, g1)
    # a graph over the chunked calls of one handle, replayed with eager calls between
    buf = x.clone()
    d = sps.distill_prepare(a[0], a[1], 30000, 0.7)
    e = sps.distill_prepare(a[0], a[1], 30000, 0.7)

    def step(h):
        sps.distill_chunk(h, buf[:, :8192], 0, first=True)
        sps.distill_chunk(h, buf[:, 8192:], 8192)
        return sps.distill_loss(h), sps.distill_chunk_grad(h, buf[:, 8192:], 8192)
    step(d)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        loss, grad = step(d)
    for i in range(4):
        buf.copy_(x.roll(i, 1))
        g.replay()
        le, ge = step(e)
        torch.cuda.synchronize()
        assert torch.equal(loss, le) and torch.equal(grad, ge)
        compare(env, loss, None, buf, ids, t, 0.7, None, None)


def test_binding_refusals(env):
    torch, sps, dev = env
    x = torch.zeros(4, 20, device=dev)
    ids = torch.zeros(4, 3, dtype=torch.int32, device=dev)
    t = torch.zeros(4, 3, device=dev)
    for bad in (lambda: sps.distill(x, ids.long(), t), lambda: sps.distill(x, ids, t.half()),
                lambda: sps.distill(x, ids, t[:, :2]), lambda: sps.distill(x[:3], ids, t),
                lambda: sps.distill(x.double(), ids, t), lambda: sps.distill(x.cpu(), ids, t),
                lambda: sps.distill(x, ids, t, out=torch.zeros(4, 20, device=dev, dtype=torch.half)),
                lambda: sps.distill(x, ids, t, row_weights=t[0])):
        with pytest.raises(AssertionError):
            bad()
    d = sps.distill_prepare(ids, t, 20)
    for bad in (lambda: sps.distill(x, ids, t, temperature=0.0),
                lambda: sps.distill(x, ids, t, temperature=float("nan")),
                lambda: sps.distill(x[:, :10], ids, t, out=x[:, 5:15]),
                lambda: sps.distill_chunk(d, x, 1, first=True),
                lambda: sps.distill_chunk(d, x[:3], 0, first=True),
                lambda: sps.distill_chunk_grad(d, x, 1)):
        with pytest.raises(sps.SpsError):
            bad()


def test_over_a_corpus(env):
    """Teacher's lists from bulk_select, the student's chunks from the half-precision path:
    scores, sums, losses and gradients chunk by chunk equal the whole rows' ones."""
    torch, sps, dev = env
    q, items, _ = synth.make_workload("mid", n_item=18000, n_query=50)
    qc, ic = sps.CSR.from_host(q, dev), sps.CSR.from_host(items, dev)
    top = sps.bulk_select(qc, ic, 20)
    it = sps.prepare(ic, 8192)
    it.enable_half()
    qq = sps.prepare_queries(qc, it)
    tau = 0.05
    d = sps.distill_prepare(top.cols, top.scores, it.n_items, tau)
    whole = torch.empty(50, it.n_items, dtype=torch.float16, device=dev)
    buf = torch.empty(50, 8192, dtype=torch.float16, device=dev)
    for c in range(it.num_chunks):
        sps.cosine_chunk_half(qq, it, c, buf)
        n = it.chunk_len(c)
        whole[:, c * 8192:c * 8192 + n] = buf[:, :n]
        sps.distill_chunk(d, buf[:, :n], c * 8192, first=c == 0)
    loss = sps.distill_loss(d)
    ids, t = top.cols.cpu().numpy(), top.scores.cpu().numpy()
    grads = []
    for c in range(it.num_chunks):
        n = it.chunk_len(c)
        grads.append(sps.distill_chunk_grad(d, whole[:, c * 8192:c * 8192 + n], c * 8192))
    compare(env, loss, torch.cat(grads, 1), whole, ids, t, tau, None, None, range(10))
