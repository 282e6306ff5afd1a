"""Dense rows in 8 bits: integers and scales exactly, products within the roundings that the
header names."""
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


def rows_of(env, n, dim, dtype, seed, spread=1.0):
    torch, _, dev = env
    r = np.random.RandomState(seed)
    x = r.randn(n, dim) * spread * np.exp(r.randn(n, 1))
    return torch.from_numpy(x.astype(np.float32)).to(getattr(torch, dtype)).to(dev)


def check_quantized(env, x, q):
    want, scales = do.quantize(x.double().cpu().numpy())
    dim = x.shape[1]
    v = q.values.cpu().numpy()
    assert (v[:, :dim] == want).all()
    assert (v[:, dim:] == 0).all()
    np.testing.assert_array_equal(q.scales.cpu().numpy(), scales)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,dim", [(1, 1), (1, 16), (3, 7), (5, 17), (64, 64), (33, 333), (9, 1024),
                                   (4, 2049), (3, 5000), (1000, 384)])
def test_quantize(env, n, dim, dtype):
    _, sps, _ = env
    x = rows_of(env, n, dim, dtype, n * 1000 + dim)
    check_quantized(env, x, sps.quantize_rows(x))


def test_quantize_ties(env):
    """Every half between two integers, and its neighbours in float32."""
    torch, sps, dev = env
    half = np.arange(-126.5, 127, 1.0, dtype=np.float32)
    rows = []
    for a in (np.float32(254), np.float32(254 * 2.0 ** -40), np.float32(254 * 2.0 ** 100),
              np.float32(127) * np.float32(1.7)):
        t = (half * (np.float64(a) / 127)).astype(np.float32)
        for v in (t, np.nextafter(t, np.float32(np.inf)), np.nextafter(t, np.float32(-np.inf))):
            rows.append(np.concatenate([[a], v]))
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).to(dev)
    check_quantized(env, x, sps.quantize_rows(x))


def test_quantize_extremes(env):
    torch, sps, dev = env
    big, tiny = float(np.finfo(np.float32).max), 2.0 ** -149
    x = torch.zeros(9, 20, device=dev)
    x[1, 3] = big
    x[1, 4] = -big / 3
    x[2] = torch.arange(20, device=dev) * tiny
    x[3, :] = 2.0 ** -126
    x[3, 5] = -(2.0 ** -120)
    x[4, 0] = float("inf")
    x[5, 19] = float("nan")
    x[6, 7] = -0.0
    x[7, 2] = -float("inf")
    x[8, :3] = torch.tensor([2.0 ** -60, -(2.0 ** -61), 2.0 ** -67], device=dev)
    q = sps.quantize_rows(x)
    check_quantized(env, x, q)
    assert q.scales.isnan().nonzero().view(-1).tolist() == [4, 5, 7]


def test_quantize_views(env):
    """Parts of a wider matrix, and rows on any boundary of an element."""
    torch, sps, dev = env
    wide = rows_of(env, 40, 130, "bfloat16", 5)
    for x in (wide[:, 1:100], wide[3:30:2, 17:18], wide[:1, 5:], wide[:, :64]):
        check_quantized(env, x, sps.quantize_rows(x))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,dim", [(1, 1), (5, 17), (64, 64), (33, 333), (1000, 384)])
def test_dequantize(env, n, dim, dtype):
    torch, sps, dev = env
    q = sps.quantize_rows(rows_of(env, n, dim, "float32", dim))
    t = getattr(torch, dtype)
    got = sps.dequantize_rows(q, t)
    want = (q.values[:, :dim].double() * q.scales.double()[:, None]).cpu().numpy()
    # exact in float64 (7 + 24 bits); at most a rounding to float32 and one to the type
    bar = np.abs(want) * do.U + do.rounding(np.abs(want) * (1 + do.U), dtype)
    assert (np.abs(got.double().cpu().numpy() - want) <= bar).all()
    if dtype == "float32":
        assert torch.equal(got, q.values[:, :dim].float() * q.scales[:, None])
    want = got
    out = torch.full((n, dim + 3), 7.0, dtype=t, device=dev)
    sps.dequantize_rows(q, out=out[:, 1:dim + 1])
    assert torch.equal(out[:, 1:dim + 1], want)
    assert (out[:, 0] == 7).all() and (out[:, dim + 1:] == 7).all()


def check_scores(env, q, i, got):
    torch = env[0]
    a = q.values[:, :q.dim].double() @ i.values[:, :i.dim].double().t().contiguous()  # exact
    want = (a * q.scales.double()[:, None] * i.scales.double()).cpu().numpy()
    g = got.double().cpu().numpy()
    dtype = str(got.dtype).split(".")[1]
    # the sum's float32, two products, the type
    bar = np.abs(want) * (3 * do.U * 1.01) + do.rounding(np.abs(want) * (1 + 4 * do.U), dtype) \
        + 2 * do.STEP["float32"]
    same = np.isnan(want) & np.isnan(g)
    big = np.abs(want) >= torch.finfo(got.dtype).max
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(g - want) <= bar) | (big & np.isinf(g))
    assert ok.all(), (np.argwhere(~ok)[:5], g[~ok][:5], want[~ok][:5])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,m,dim", [
    (1, 1, 1), (1, 1000, 384), (2, 15, 16), (16, 33, 64), (17, 500, 100), (33, 257, 200), (64, 129, 48),
    (65, 130, 333), (100, 100, 65), (129, 1000, 768), (300, 129, 1000), (513, 777, 20)])
def test_scores(env, n, m, dim, dtype):
    torch, sps, _ = env
    q = sps.quantize_rows(rows_of(env, n, dim, "float32", n))
    i = sps.quantize_rows(rows_of(env, m, dim, "float32", m + 7))
    check_scores(env, q, i, sps.int8_scores(q, i, dtype=getattr(torch, dtype)))


def test_scores_large_tiles(env):
    """More than 256 tiles of 256 x 256, odd edges; the largest magnitudes in long rows."""
    torch, sps, dev = env
    q = sps.quantize_rows(rows_of(env, 4097, 72, "float32", 1))
    i = sps.quantize_rows(rows_of(env, 4099, 72, "float32", 2))
    check_scores(env, q, i, sps.int8_scores(q, i))
    for n in (1, 70):
        full = torch.full((n, 131072), -127, dtype=torch.int8, device=dev)
        one = sps.Int8Rows(full, torch.ones(n, device=dev), 131072)
        assert (sps.int8_scores(one, one[:1]) == float(127 * 127 * 131072)).all()


def test_scores_do_not_depend_on_the_batch(env):
    """A query's scores are the same bits alone, among few and among many, and in chunks."""
    torch, sps, _ = env
    q = sps.quantize_rows(rows_of(env, 200, 300, "float32", 3))
    i = sps.quantize_rows(rows_of(env, 1000, 300, "float32", 4))
    whole = sps.int8_scores(q, i)
    for n in (1, 16, 17, 40, 64, 65):
        assert torch.equal(sps.int8_scores(q[:n], i), whole[:n])
    out = torch.empty_like(whole)
    for b in range(0, 1000, 130):
        sps.int8_scores(q, i[b:b + 130], out[:, b:b + 130])
    assert torch.equal(out, whole)


def test_scores_leave_the_rest_alone(env):
    torch, sps, dev = env
    for n in (3, 70):
        q = sps.quantize_rows(rows_of(env, n, 50, "float32", 3))
        i = sps.quantize_rows(rows_of(env, 77, 50, "float32", 4))
        out = torch.full((n + 2, 90), 5.0, device=dev)
        sps.int8_scores(q, i, out[1:n + 1, 3:80])
        assert torch.equal(out[1:n + 1, 3:80], sps.int8_scores(q, i))
        out[1:n + 1, 3:80] = 5.0
        assert (out == 5.0).all()


def test_rows_that_hold_nan(env):
    """Their scores are NaN, nobody else's."""
    torch, sps, _ = env
    x, y = rows_of(env, 70, 40, "float32", 3), rows_of(env, 90, 40, "float32", 4)
    x[3, 5], y[8, 1] = float("nan"), float("inf")
    for n in (5, 70):
        s = sps.int8_scores(sps.quantize_rows(x[:n]), sps.quantize_rows(y))
        bad = s.isnan()
        assert bad[3].all() and bad[:, 8].all() and int(bad.sum()) == 90 + n - 1


def test_scores_of_scales_far_apart(env):
    """Scales of either side near the ends of float32's range: the scores are inside it."""
    torch, sps, dev = env
    for sq, si in ((2.0 ** 110, 2.0 ** -115), (2.0 ** -115, 2.0 ** 110)):
        for n in (5, 70):
            q = sps.quantize_rows(rows_of(env, n, 200, "float32", 3))
            i = sps.quantize_rows(rows_of(env, 90, 200, "float32", 4))
            q.scales *= sq
            i.scales *= si
            got = sps.int8_scores(q, i)
            assert got.isfinite().all()
            check_scores(env, q, i, got)


def test_empty(env):
    torch, sps, dev = env
    none = sps.quantize_rows(torch.empty(0, 24, device=dev))
    some = sps.quantize_rows(rows_of(env, 5, 24, "float32", 3))
    assert sps.int8_scores(none, some).shape == (0, 5)
    assert sps.int8_scores(some, none).shape == (5, 0)
    assert sps.dequantize_rows(none).shape == (0, 24)
    top = sps.int8_select(some, none, 3)
    assert (top.cols == -1).all() and torch.isneginf(top.scores).all()


@pytest.mark.parametrize("n,m,k,chunk", [(1, 5000, 10, 700), (70, 3001, 16, 1000), (3, 7, 9, 4)])
def test_select(env, n, m, k, chunk):
    torch, sps, _ = env
    q = sps.quantize_rows(rows_of(env, n, 96, "bfloat16", 3))
    i = sps.quantize_rows(rows_of(env, m, 96, "bfloat16", 4))
    top = sps.int8_select(q, i, k, chunk_size=chunk)
    s = sps.int8_scores(q, i)
    order = torch.sort(-s.double(), dim=1, stable=True).indices[:, :k]
    kk = min(k, m)
    assert torch.equal(top.cols[:, :kk].long(), order)
    assert torch.equal(top.scores[:, :kk], s.gather(1, order))
    assert (top.cols[:, kk:] == -1).all()


def test_graph_and_stream(env):
    """A captured answer to one question, replayed with new questions, and the same calls on
    another stream."""
    torch, sps, dev = env
    i = sps.quantize_rows(rows_of(env, 3000, 128, "bfloat16", 4))
    x = rows_of(env, 1, 128, "bfloat16", 5).clone()

    def answer():
        s = sps.int8_scores(sps.quantize_rows(x), i)
        top = sps.top_rows(1, 5, dev)
        sps.select_chunk(s, top, 0, first=True)
        return top

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        answer()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = answer()
    for seed in range(4):
        x.copy_(rows_of(env, 1, 128, "bfloat16", seed))
        g.replay()
        torch.cuda.synchronize()
        want = answer()
        assert torch.equal(got.cols, want.cols) and torch.equal(got.scores, want.scores)
    with torch.cuda.stream(side):
        other = sps.int8_scores(sps.quantize_rows(x, stream=side), i, stream=side)
    side.synchronize()
    assert torch.equal(other, sps.int8_scores(sps.quantize_rows(x), i))
