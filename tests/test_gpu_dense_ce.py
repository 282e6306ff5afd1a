"""Cross entropy of dense rows and its gradients against the float64 oracle, within the bounds
that it derives."""
import numpy as np
import pytest

import dense_oracle as do

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


def make(env, n, m, d, dtype, seed, masked=True, weighted=True, spread=1.0):
    """Rows, items, targets (some outside), bias (some -inf, never a target's) and weights."""
    torch, _, dev = env
    r = np.random.RandomState(seed)
    t = r.randint(0, m, n).astype(np.int32)
    w = r.randn(m, d) * spread / np.sqrt(d)
    x = w[t] * (d ** 0.5) * r.rand(n, 1) + r.randn(n, d)
    to = lambda a: torch.from_numpy(a.astype(np.float32)).to(getattr(torch, dtype)).to(dev)  # noqa: E731
    bias = weights = None
    if masked:
        bias = r.randn(m).astype(np.float32)
        bias[r.rand(m) < 0.1] = -np.inf
        bias[t] = 0.5
        out = r.rand(n) < 0.1
        t[out] = r.choice([-1, m, -7, 2 ** 31 - 1], out.sum())
    if weighted:
        weights = r.rand(n).astype(np.float32)
        weights[r.rand(n) < 0.05] = 0.0
    dv = lambda a: None if a is None else torch.from_numpy(a).to(dev)  # noqa: E731
    return to(x), to(w), dv(t), dv(bias), dv(weights)


def check(env, got, x, w, t, tau, bias, weights, out=None):
    n64 = lambda a: None if a is None else a.double().cpu().numpy()  # noqa: E731
    dtype = str(x.dtype).split(".")[1]
    loss, e_loss, gq, gi, bars = do.cross_entropy(n64(x), n64(w), t.cpu().numpy().astype(np.int64),
                                                  tau, n64(bias), n64(weights), dtype)
    bq, bi = bars(dtype if out is None else out)
    worst = []
    for name, g, want, bar in (("loss", got[0], loss, e_loss), ("queries", got[1], gq, bq),
                               ("items", got[2], gi, bi)):
        if g is None:
            continue
        g = n64(g)
        same = (np.isnan(g) & np.isnan(want)) | (g == want)
        with np.errstate(invalid="ignore", divide="ignore"):
            off = np.where(same, 0.0, np.abs(g - want) / bar)
        assert (off <= 1).all(), (name, np.argwhere(~(off <= 1))[:5], g[~(off <= 1)][:5],
                                  want[~(off <= 1)][:5], np.nanmax(off))
        worst.append(off.max() if off.size else 0.0)
    return worst


SHAPES = [(1, 1, 1), (1, 5, 3), (7, 130, 64), (130, 257, 72), (65, 300, 333), (64, 64, 128),
          (128, 128, 64), (300, 1000, 100), (257, 520, 8), (130, 5000, 40), (31, 4099, 513)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,m,d", SHAPES)
def test_loss_and_gradients(env, n, m, d, dtype):
    _, sps, _ = env
    for masked, weighted, tau in ((True, True, 0.25), (False, False, 1.0)):
        x, w, t, b, ww = make(env, n, m, d, dtype, n + m + d, masked, weighted)
        got = sps.dense_cross_entropy(x, w, t, tau, b, ww)
        check(env, got, x, w, t, tau, b, ww)


@pytest.mark.parametrize("dtype", TYPES)
def test_large_tiles(env, dtype):
    """Enough tiles for the large form of each product, with odd edges."""
    _, sps, _ = env
    x, w, t, b, ww = make(env, 4097, 4199, 72, dtype, 3)
    check(env, sps.dense_cross_entropy(x, w, t, 0.5, b, ww), x, w, t, 0.5, b, ww)


def test_large_dims(env):
    _, sps, _ = env
    x, w, t, b, ww = make(env, 2200, 2300, 2056, "bfloat16", 3)
    check(env, sps.dense_cross_entropy(x, w, t, 1.0, b, ww), x, w, t, 1.0, b, ww)


@pytest.mark.parametrize("dtype", TYPES)
def test_pieces(env, dtype):
    """More rows than a piece of the logits holds: the items' gradient is a sum over pieces."""
    torch, sps, dev = env
    n, m, d = 600, 1700001, 8
    x, w, t, b, ww = make(env, n, m, d, dtype, 3)
    got = sps.dense_cross_entropy(x, w, t, 0.5, b, ww)
    # by parts of the rows that are a piece each: equal losses and rows, and sums that add up
    gi, size = torch.zeros(m, d, dtype=torch.float64, device=dev), 0
    for a in range(0, n, 200):
        part = sps.dense_cross_entropy(x[a:a + 200], w, t[a:a + 200], 0.5, b, ww[a:a + 200],
                                       grad_dtype=torch.float32)
        assert torch.equal(part[0], got[0][a:a + 200])
        assert torch.allclose(part[1].double(), got[1][a:a + 200].double(),
                              rtol=2 * do.HALF[dtype] + 1e-4, atol=1e-6)
        gi += part[2].double()
        size = size + part[2].double().abs()
    # the parts round G apart (fp16 by another power of two): half a step each
    bar = size * (2 * do.HALF[dtype] + 2.0 ** -12 * (dtype != "float32") + 2.0 ** -20)
    off = (gi - got[2].double()).abs() - gi.abs() * do.HALF[dtype] - 1e-7
    assert (off <= bar).all()


def exact_on_gpu(env, x, w, t, tau, weights, rows=2048):
    """Losses and gradients in float64, and the bars of both gradients, a batch of rows at a time."""
    torch = env[0]
    d = str(x.dtype).split(".")[1]
    half = 2.0 ** -22 if d == "float32" else do.HALF[d]
    planes = do.PLANES * (d == "float32")
    w64 = w.double()
    wt = w64.t().contiguous()
    loss, gq, bq = [], [], []
    gi, bi = torch.zeros_like(w64), torch.zeros_like(w64)
    for a in range(0, len(x), rows):
        xb, tb = x[a:a + rows].double(), t[a:a + rows].long()
        live = tb >= 0
        z = xb @ wt / tau
        r = torch.arange(len(xb), device=x.device)
        lse = z.logsumexp(1)
        loss.append(torch.where(live, lse - z[r, tb.clamp(min=0)], 0.0))
        p = torch.exp(z - lse[:, None])
        # Logits in float32 are off by ez: a sum of dim products by 2 dim u of their magnitudes, the
        # factor and the maximum by a few u; a p by a factor of 1 + 2 ez and its sums' 200 u, and the
        # target's 1 - p, which comes from the loss, by as much as the loss, whatever is left of it
        size = xb.abs() @ wt.abs() / tau
        ez = (((2 * x.shape[1] + 8) * do.U + planes) * size + 4 * do.U * z.abs()).amax(1) + 8 * do.U * z.abs().amax(1)
        eg = p * (4 * ez[:, None] + 200 * do.U + half * 2.0 ** -3)
        eg[r[live], tb[live]] = 2 * ez[live] + 160 * do.U
        p[r[live], tb[live]] -= 1
        factor = torch.where(live, weights[a:a + rows].double() / tau, 0.0)[:, None]
        eg = (eg + half * (p.abs() + eg)) * factor
        p *= factor
        # float32 sums of the products
        eg += p.abs() * (2 * max(w64.shape[0], len(x)) * do.U + planes)
        gq.append(p @ w64)
        bq.append(eg @ w64.abs())
        xt = xb.t().contiguous()
        gi += (xt @ p).t()
        bi += (xt.abs() @ eg).t()
    return torch.cat(loss), torch.cat(gq), gi, torch.cat(bq), bi


@pytest.mark.parametrize("n,m,d,dtype", [
    (1024, 70000, 256, "bfloat16"),   # whole rounds of tiles of the items' product, then a split rest
    (1000, 66000, 264, "float32"),
    (8200, 66304, 256, "float16"),    # two pieces of rows: sums that go on, whole and split
    (8200, 70001, 250, "bfloat16"),
    (130, 300000, 520, "float16"),    # a long k in many parts
])
def test_rounds_and_parts(env, n, m, d, dtype):
    torch, sps, dev = env
    x, w, t, _, ww = make(env, n, m, d, dtype, 5, masked=False)
    t[::17] = -1
    loss, gq, gi, bq, bi = exact_on_gpu(env, x, w, t, 0.5, ww)
    got = sps.dense_cross_entropy(x, w, t, 0.5, row_weights=ww)
    assert ((got[0].double() - loss).abs() <= 1e-5 * (1 + loss.abs())).all()
    for g, want, bar in ((got[1], gq, bq), (got[2], gi, bi)):
        off = (g.double() - want).abs() - bar - want.abs() * do.HALF[dtype] - do.STEP[dtype]
        if dtype != "bfloat16":  # G's step below 2^-14 of the largest weight's range
            off -= 2.0 ** -38 * 64
        assert (off <= 0).all(), (float(off.max()), int((off > 0).sum()))


@pytest.mark.parametrize("dtype", TYPES)
def test_choices(env, dtype):
    """Losses alone, one side's gradient, float32 gradients: the same numbers."""
    torch, sps, _ = env
    x, w, t, b, ww = make(env, 100, 900, 72, dtype, 5)
    loss, gq, gi = sps.dense_cross_entropy(x, w, t, 0.5, b, ww)
    a = sps.dense_cross_entropy(x, w, t, 0.5, b, ww, need_grad=False)
    assert a[1] is None and a[2] is None and torch.equal(a[0], loss)
    a = sps.dense_cross_entropy(x, w, t, 0.5, b, ww, need_grad="queries")
    assert a[2] is None and torch.equal(a[0], loss) and torch.equal(a[1], gq)
    a = sps.dense_cross_entropy(x, w, t, 0.5, b, ww, need_grad="items")
    assert a[1] is None and torch.equal(a[0], loss) and torch.equal(a[2], gi)
    a = sps.dense_cross_entropy(x, w, t, 0.5, b, ww, grad_dtype=torch.float32)
    assert a[1].dtype == torch.float32
    assert torch.equal(a[1].to(x.dtype), gq) and torch.equal(a[2].to(x.dtype), gi)
    check(env, a, x, w, t, 0.5, b, ww, out="float32")


@pytest.mark.parametrize("dtype", TYPES)
def test_differences(env, dtype):
    """The gradient against central differences of the losses, in float64 of the oracle's and of
    the kernel's own losses at float32 rows."""
    torch, sps, dev = env
    x, w, t, b, ww = make(env, 6, 40, 16, dtype, 9)
    _, gq, gi = sps.dense_cross_entropy(x, w, t, 0.5, b, ww, grad_dtype=torch.float32)
    h = 2.0 ** -8

    def total(a, c):
        loss = sps.dense_cross_entropy(a, c, t, 0.5, b, ww, need_grad=False)[0]
        return float((loss.double() * ww.double()).sum())

    xf, wf = x.float(), w.float()
    for i, j in ((0, 0), (3, 7), (5, 15)):
        for side, rows, g in ((0, xf, gq), (1, wf, gi)):
            up, down = rows.clone(), rows.clone()
            up[i, j] += h
            down[i, j] -= h
            args = [(up, wf), (down, wf)] if side == 0 else [(xf, up), (xf, down)]
            diff = (total(*args[0]) - total(*args[1])) / (2 * h)
            # losses to 1e-6 each, the third derivative's h^2 term, G's rounding
            assert abs(diff - float(g[i, j])) < 2e-3 + 12 * do.HALF[dtype], (i, j, side)


def test_rows_without_part_hold_anything(env):
    """NaN and infinities in padded rows, rows of weight 0 and struck items reach nothing."""
    torch, sps, dev = env
    for dtype in TYPES:
        x, w, t, b, ww = make(env, 200, 500, 72, dtype, 5)
        want = sps.dense_cross_entropy(x, w, t, 0.5, b, ww)
        x2, w2 = x.clone(), w.clone()
        pad = (t < 0) | (t >= 500)
        assert pad.any() and torch.isneginf(b).any()
        x2[pad], w2[torch.isneginf(b)] = float("nan"), float("inf")
        w2[torch.isneginf(b).nonzero()[0]] = float("nan")
        for got in (sps.dense_cross_entropy(x2, w2, t, 0.5, b, ww),):
            for g, e in zip(got, want):
                assert torch.equal(g, e)
        assert (want[0][pad] == 0).all() and (want[1][pad] == 0).all()
        assert (want[1][ww == 0] == 0).all() and (want[2][torch.isneginf(b)] == 0).all()
        big = torch.finfo(torch.float16 if dtype == "float16" else torch.float32).max
        for x3, w3 in ((x2.clone(), w2.clone()),):  # and neither does what is large there
            x3[pad], w3[torch.isneginf(b)] = big, -big
            for g, e in zip(sps.dense_cross_entropy(x3, w3, t, 0.5, b, ww), want):
                assert torch.equal(g, e)
        x2[ww == 0] = float("nan")  # its loss is its own affair
        got = sps.dense_cross_entropy(x2, w2, t, 0.5, b, ww)
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_special_rows(env):
    torch, sps, dev = env
    for dtype in TYPES:
        x, w, t, b, ww = make(env, 20, 70, 24, dtype, 6, masked=False, weighted=False)
        # a target that is struck out: infinite loss, finite gradient
        b = torch.zeros(70, device=dev)
        t[3] = 9
        b[9] = -float("inf")
        loss, gq, gi = sps.dense_cross_entropy(x, w, t, 1.0, b)
        assert torch.isposinf(loss[3]) and gq.isfinite().all() and gi.isfinite().all()
        check(env, (loss, gq, gi), x, w, t, 1.0, b, None)
        # every item struck out
        none = torch.full((70,), -float("inf"), device=dev)
        loss, gq, gi = sps.dense_cross_entropy(x, w, t, 1.0, none)
        assert (loss == 0).all() and (gq == 0).all() and (gi == 0).all()
        # the type's lowest value is a mask that leaves something
        low = torch.full((70,), torch.finfo(torch.float32).min / 4, device=dev)
        low[5] = 0.0
        t[:] = 5
        loss, gq, gi = sps.dense_cross_entropy(x, w, t, 1.0, low)
        assert (loss.abs() <= 1e-6).all() and gq.abs().max() <= 1e-5
        # NaN and infinity in a row that takes part stay its own in the losses and its gradient
        x2 = x.clone()
        x2[2, 1], x2[4, 0] = float("nan"), float("inf")
        l0, q0, _ = sps.dense_cross_entropy(x, w, t, 1.0)
        l2, q2, _ = sps.dense_cross_entropy(x2, w, t, 1.0)
        others = [i for i in range(20) if i not in (2, 4)]
        assert l2[[2, 4]].isnan().all() and q2[[2, 4]].isnan().all()
        assert torch.equal(l2[others], l0[others]) and torch.equal(q2[others], q0[others])


@pytest.mark.parametrize("dtype", TYPES)
def test_large_logits(env, dtype):
    """Logits in the hundreds, rows that are certain and rows that are far off."""
    torch, sps, dev = env
    x, w, t, b, ww = make(env, 90, 400, 64, dtype, 8, spread=40.0)
    got = sps.dense_cross_entropy(x, w, t, 0.05, b, ww)
    check(env, got, x, w, t, 0.05, b, ww)
    assert got[0].max() > 100


def test_float32_scales(env):
    """Rows of very different lengths, and matrices of very large and very small values."""
    torch, sps, dev = env
    for sx, sw in ((1.0, 1.0), (1e15, 1e-15), (1e-20, 1e20), (1e-30, 1e30)):
        x, w, t, b, ww = make(env, 70, 300, 40, "float32", 8)
        x *= torch.logspace(-3, 0, 70, device=dev)[:, None] * sx
        w *= torch.logspace(0, -3, 300, device=dev)[:, None] * sw
        got = sps.dense_cross_entropy(x, w, t, 0.1, b, ww)
        check(env, got, x, w, t, 0.1, b, ww)


@pytest.mark.parametrize("ex,ew", [(-112, 114), (114, -112), (-60, 60), (100, -100)])
def test_float32_rows_near_the_range_s_ends(env, ex, ew):
    """Sums that leave the range when one side's scale is taken out, logits that do not."""
    torch, sps, dev = env
    x, w, t, b, ww = make(env, 70, 300, 40, "float32", 9)
    x, w = x * 2.0 ** ex, w * 2.0 ** ew
    got = sps.dense_cross_entropy(x, w, t, 0.3, b, ww)
    assert got[0].isfinite().all() and got[1].isfinite().all() and got[2].isfinite().all()
    check(env, got, x, w, t, 0.3, b, ww)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("scale", [1e-6, 65536.0])
def test_scaled_losses(env, dtype, scale):
    _, sps, _ = env
    x, w, t, b, ww = make(env, 90, 400, 64, dtype, 8)
    ww = ww * scale
    got = sps.dense_cross_entropy(x, w, t, 1.0, b, ww, grad_dtype=env[0].float32)
    check(env, got, x, w, t, 1.0, b, ww, out="float32")


@pytest.mark.parametrize("dtype", TYPES)
def test_views(env, dtype):
    """Rows of wider matrices, on any boundary; gradients do not depend on it."""
    torch, sps, dev = env
    x, w, t, b, ww = make(env, 70, 330, 64, dtype, 4)
    want = sps.dense_cross_entropy(x, w, t, 1.0, b, ww)
    for off, wide in ((0, 64), (0, 80), (1, 67), (8, 96), (3, 72)):
        xs = torch.full((70, wide), float("nan"), dtype=x.dtype, device=dev)[:, off:off + 64]
        ws = torch.full((330, wide), float("nan"), dtype=x.dtype, device=dev)[:, off:off + 64]
        if xs.shape[1] < 64:
            continue
        xs.copy_(x)
        ws.copy_(w)
        for a, c in ((xs, w), (x, ws), (xs, ws)):
            for g, e in zip(sps.dense_cross_entropy(a, c, t, 1.0, b, ww), want):
                assert torch.equal(g, e)


def test_empty(env):
    torch, sps, dev = env
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=dev)  # noqa: E731
    loss, gq, gi = sps.dense_cross_entropy(torch.ones(0, 8, device=dev), torch.ones(5, 8, device=dev),
                                           i32(0))
    assert loss.shape == (0,) and gq.shape == (0, 8) and (gi == 0).all() and gi.shape == (5, 8)
    loss, gq, gi = sps.dense_cross_entropy(torch.ones(3, 8, device=dev).half(),
                                           torch.ones(0, 8, device=dev).half(), i32(3))
    assert (loss == 0).all() and (gq == 0).all() and gi.shape == (0, 8)


@pytest.mark.parametrize("dtype", TYPES)
def test_same_bits_again(env, dtype):
    torch, sps, _ = env
    x, w, t, b, ww = make(env, 500, 3000, 96, dtype, 4)
    first = sps.dense_cross_entropy(x, w, t, 0.2, b, ww)
    for _ in range(3):
        for g, e in zip(sps.dense_cross_entropy(x, w, t, 0.2, b, ww), first):
            assert torch.equal(g, e)


def test_graphs_and_streams(env):
    """Two captured steps, replayed in turn with eager work between, and a call on another
    stream; every replay against the eager result."""
    torch, sps, dev = env
    sets = [make(env, 100, 700, 64, dt, 3) for dt in ("bfloat16", "float16")]
    side = torch.cuda.Stream()
    graphs = []
    for x, w, t, b, ww in sets:
        with torch.cuda.stream(side):
            sps.dense_cross_entropy(x, w, t, 0.3, b, ww)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = sps.dense_cross_entropy(x, w, t, 0.3, b, ww)
        graphs.append((g, out))
    for seed in range(3):
        for (x, w, t, b, ww), (g, out) in zip(sets, graphs):
            x.copy_(torch.randn(x.shape, device=dev) * (seed + 1))
            g.replay()
        torch.cuda.synchronize()
        for (x, w, t, b, ww), (g, out) in zip(sets, graphs):
            for a, e in zip(out, sps.dense_cross_entropy(x, w, t, 0.3, b, ww)):
                assert torch.equal(a, e)
    x, w, t, b, ww = sets[0]
    want = sps.dense_cross_entropy(x, w, t, 0.3, b, ww)
    torch.cuda.synchronize()
    got = sps.dense_cross_entropy(x, w, t, 0.3, b, ww, stream=side)
    side.synchronize()
    for a, e in zip(got, want):
        assert torch.equal(a, e)


def test_together(env):
    """A step of training dense rows against a corpus, the corpus into 8 bits, and an answer: the
    gradients lower the loss, and the best items of the 8-bit scores are those of their exact
    products."""
    torch, sps, dev = env
    x, w, t, _, _ = make(env, 300, 2000, 64, "float32", 2, masked=False, weighted=False)
    loss, gq, gi = sps.dense_cross_entropy(x, w, t, 0.5, row_weights=torch.full((300,), 1 / 300,
                                                                               device=dev))
    x2, w2 = x - 0.1 * gq, w - 0.1 * gi
    q, i = sps.quantize_rows(x2), sps.quantize_rows(w2)
    top = sps.int8_select(q, i, 10, chunk_size=700)
    a = sps.dequantize_rows(q).double() @ sps.dequantize_rows(i).double().t().contiguous()
    best = a.topk(10, dim=1)
    assert torch.allclose(top.scores.double(), best.values, rtol=1e-6, atol=1e-9)
    # the list distils into sparse or dense students alike
    s = sps.int8_scores(q, i)
    d_loss, d_grad = sps.distill(s, top.cols, top.scores, temperature=0.5)
    assert d_loss.isfinite().all() and d_grad.shape == s.shape
