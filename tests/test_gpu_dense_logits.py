"""Cross entropy of dense rows whose logits are large: finite masks over some items or all, and
products over a small temperature. Every logit here is a number that float32 holds, so that the
results are known whatever their size."""
import numpy as np
import pytest

import dense_oracle as do
from test_gpu_dense_ce import TYPES, check, env, make  # noqa: F401

pytestmark = pytest.mark.gpu


def check_exact(env, got, x, w, t, tau, weights=None, bias=None):  # noqa: F811
    """Against float64 where the logits are exact. What is left: a p is off by its exponential and
    its row's sums (200 u, as in the oracle's bars), its code (2^-11 of 16-bit types at the most)
    and G's rounding; then the products."""
    n64 = lambda a: None if a is None else a.double().cpu().numpy()  # noqa: E731
    dtype = str(x.dtype).split(".")[1]
    wide = dtype == "float32"
    xs, ws, ts = n64(x), n64(w), t.cpu().numpy()
    n, m = len(xs), len(ws)
    z = xs @ ws.T / tau + (0.0 if bias is None else n64(bias))
    top = z.max(1, keepdims=True)
    e = np.exp(z - top)
    total = e.sum(1, keepdims=True)
    p, rows = e / total, np.arange(n)
    loss = (top[:, 0] - z[rows, ts]) + np.log(total[:, 0])  # (in this order: the log beside 1e11)
    # the difference of maximum and target is rounded once, as the loss is
    off = np.abs(n64(got[0]) - loss) / (200 * do.U + 4 * do.U * np.abs(loss))
    assert (off <= 1).all(), (np.argwhere(~(off <= 1))[:5], n64(got[0])[:5], loss[:5])
    g = p.copy()
    g[rows, ts] -= 1
    f = (np.ones(n) if weights is None else n64(weights))[:, None] / tau
    half = 2.0 ** -22 if wide else do.HALF[dtype]
    eg = p * (200 * do.U + (0.0 if wide else 2.0 ** -11))
    eg[rows, ts] = np.abs(g[rows, ts]) * 200 * do.U + 200 * do.U + 4 * do.U * np.minimum(np.abs(loss), 100)
    eg = eg + half * (np.abs(g) + eg)
    G, eG = g * f, eg * f + 2.0 ** -39 * f.max()
    planes = do.PLANES if wide else 0.0
    for a, b, v, k in ((1, G, ws, m), (2, G.T, xs, n)):
        eb = eG if a == 1 else eG.T
        want, size = b @ v, np.abs(v)
        bar = eb @ size + (np.abs(b) @ size) * ((2 * (k + 8) + 4) * do.U + planes)
        if wide:
            bar += do.FLOOR * size.max() * np.abs(b).sum(1)[:, None]
        bar += do.rounding(np.abs(want) + bar, str(got[a].dtype).split(".")[1])
        off = np.abs(n64(got[a]) - want) / np.maximum(bar, 1e-300)
        assert (off <= 1).all(), (a, np.argwhere(~(off <= 1))[:5], np.nanmax(off))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("low", [-1.2e7, -1.5e7, -2e7, -3e7, -5e7, -1e8, -1.5e8, -1.8e8, -1e9, -1e12, -1e30])
def test_finite_masks_over_whole_blocks(env, dtype, low):  # noqa: F811
    """Items under a finite mask count as much as those under -inf: nothing, to the last bit."""
    torch, sps, dev = env
    x, w, t, b, ww = make(env, 150, 700, 72, dtype, 4, masked=False)
    t = torch.where((t >= 64) & (t < 512), t % 64, t)
    for a, e in ((64, 256), (70, 500)):
        none = torch.zeros(700, device=dev)
        none[a:e] = -float("inf")
        some = none.clone()
        some[a:e] = low
        want = sps.dense_cross_entropy(x, w, t, 0.5, none, ww)
        got = sps.dense_cross_entropy(x, w, t, 0.5, some, ww)
        for g, v in zip(got, want):
            assert g.isfinite().all() and torch.equal(g, v), (a, e)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("low", [-1e5, -1.3e7, -2e7, -1e8, -1e9, -1e20])
def test_a_mask_on_every_item(env, dtype, low):  # noqa: F811
    """Takes part in every logit alike, so in no loss and no gradient."""
    torch, sps, dev = env
    for n, m in ((5, 64), (150, 300)):
        _, w, t, _, ww = make(env, n, m, 24, dtype, 6, masked=False)
        x = torch.zeros(n, 24, device=dev, dtype=w.dtype)
        bias = torch.full((m,), low, device=dev)
        got = sps.dense_cross_entropy(x, w, t, 1.0, bias, ww)
        check_exact(env, got, x, w, t, 1.0, ww)
        alone = sps.dense_cross_entropy(x, w, t, 1.0, bias, ww, need_grad=False)[0]
        assert torch.equal(alone, got[0])


def whole(env, shape, most, dtype, seed):  # noqa: F811
    torch, _, dev = env
    a = np.random.RandomState(seed).randint(-most, most + 1, shape).astype(np.float32)
    return torch.from_numpy(a).to(getattr(torch, dtype)).to(dev)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("up", [1, 2, 8, 128])
def test_products_over_a_small_temperature(env, dtype, up):  # noqa: F811
    """Whole numbers, so that products are exact: logits of some 1e6 to 1e10 and more, ties among
    the largest. (300 items: whole tiles and an edge.)"""
    torch, sps, dev = env
    tau = 2.0 ** -16
    x, w = whole(env, (150, 64), 4, dtype, 1) * up, whole(env, (300, 64), 4, dtype, 2) * up
    w[40] = w[7]
    w[290] = w[7]
    x[::3] = w[7]
    t = torch.arange(150, device=dev, dtype=torch.int32) * 2
    t[::3] = 40
    f32 = torch.float32  # (gradients of 65536 and more are infinite in fp16)
    got = sps.dense_cross_entropy(x, w, t, tau, grad_dtype=f32)
    check_exact(env, got, x, w, t, tau)
    ww = torch.rand(150, device=dev) + 0.1
    got = sps.dense_cross_entropy(x, w, t, tau, row_weights=ww, grad_dtype=f32)
    check_exact(env, got, x, w, t, tau, ww)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", [64, 256, 300, 2000])
def test_logits_that_differ_by_little(env, dtype, m):  # noqa: F811
    """2^24 and a few: a softmax over many items all the same."""
    torch, sps, dev = env
    tau = 2.0 ** -4
    x, w = torch.full((150, 32), 256.0, device=dev), torch.full((m, 32), 256.0, device=dev)
    x[:, 16:] = whole(env, (150, 16), 1, "float32", 1) / 8  # 2^20 and eighths: 24 bits
    w[:, 16:] = whole(env, (m, 16), 1, "float32", 2)
    x, w = x.to(getattr(torch, dtype)), w.to(getattr(torch, dtype))
    t = (torch.arange(150, device=dev, dtype=torch.int32) * 7) % m
    got = sps.dense_cross_entropy(x, w, t, tau)
    assert 1 < got[0].median() < 30
    check_exact(env, got, x, w, t, tau)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("low", [-1.5e38, -3e38, float(np.finfo(np.float32).min)])
def test_the_lowest_finite_masks(env, dtype, low):  # noqa: F811
    """A finite bias strikes nothing out: some items, all of them, and targets that have it."""
    torch, sps, dev = env
    x, w, t, b, ww = make(env, 150, 700, 72, dtype, 4, masked=False)
    some = torch.zeros(700, device=dev)
    some[64:256] = low
    some[3] = low
    none = torch.where(some < 0, -float("inf"), some)
    free = torch.where(some[t.long()] < 0, 5, t)
    want = sps.dense_cross_entropy(x, w, free, 0.5, none, ww)
    for g, v in zip(sps.dense_cross_entropy(x, w, free, 0.5, some, ww), want):
        assert g.isfinite().all() and torch.equal(g, v)
    # a target under the mask: the loss is its bias, the gradient that of a row that is all wrong
    t[:] = 100
    got = sps.dense_cross_entropy(x, w, t, 0.5, some, ww, grad_dtype=torch.float32)
    assert torch.allclose(got[0], torch.full_like(got[0], -low), rtol=2.0 ** -22)
    live = sps.dense_cross_entropy(x, w, t * 0 - 1, 0.5, some, ww, grad_dtype=torch.float32)
    assert (live[2] == 0).all()
    item = got[2][100].double()
    exact = -(ww.double()[:, None] * x.double()).sum(0) / 0.5
    size = (ww.double()[:, None] * x.double().abs()).sum(0) / 0.5
    half = 2.0 ** -22 if dtype == "float32" else do.HALF[dtype]
    assert ((item - exact).abs() <= size * (half + do.PLANES + 320 * do.U) + 2.0 ** -30).all()
    # on every item (the products vanish beside it)
    x = torch.zeros_like(x)
    every = torch.full((700,), low, device=dev)
    check_exact(env, sps.dense_cross_entropy(x, w, t, 1.0, every, ww), x, w, t, 1.0, ww)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_mask_and_products(env, dtype):  # noqa: F811
    """-1e9 on every item and products of whole 64, which float32 holds beside it: the mask is taken
    as it is, not rounded with a factor of the logarithm."""
    torch, sps, dev = env
    x, w = whole(env, (150, 16), 1, dtype, 1) * 16, whole(env, (300, 16), 1, dtype, 2) * 8
    t = torch.arange(150, device=dev, dtype=torch.int32) * 2
    for tau in (1.0, 2.0):
        bias = torch.full((300,), -1e9, device=dev)
        got = sps.dense_cross_entropy(x, w, t, tau, bias)
        check_exact(env, got, x, w, t, tau)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_large_bias(env, dtype):  # noqa: F811
    """The largest value on some items: they share the softmax."""
    torch, sps, dev = env
    w = whole(env, (300, 16), 2, dtype, 1)
    x = torch.zeros(40, 16, device=dev, dtype=w.dtype)
    bias = torch.zeros(300, device=dev)
    bias[[7, 8, 290]] = torch.finfo(torch.float32).max
    t = torch.full((40,), 8, device=dev, dtype=torch.int32)
    check_exact(env, sps.dense_cross_entropy(x, w, t, 1.0, bias), x, w, t, 1.0, bias=bias)
