"""One side's gradient of the cross entropy at the sizes of every plan, pieces under a mask against
float64, and answers from a corpus of many chunks."""
import pytest

import dense_oracle as do
from test_gpu_dense_ce import TYPES, check, env, exact_on_gpu, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("side", ["queries", "items"])
@pytest.mark.parametrize("n,m,d", [(1, 1, 1), (1, 5, 3), (65, 300, 333), (257, 520, 8), (130, 5000, 40),
                                   (31, 4099, 513), (1500, 100, 64)])
def test_one_side(env, n, m, d, side, dtype):  # noqa: F811
    _, sps, _ = env
    x, w, t, b, ww = make(env, n, m, d, dtype, n + m + d)
    got = sps.dense_cross_entropy(x, w, t, 0.25, b, ww, need_grad=side)
    assert got[2 if side == "queries" else 1] is None
    check(env, got, x, w, t, 0.25, b, ww)


@pytest.mark.parametrize("side", ["queries", "items"])
@pytest.mark.parametrize("n,m,d,dtype", [(1024, 70000, 256, "bfloat16"), (1000, 66000, 264, "float32"),
                                         (8200, 66304, 256, "float16"), (130, 300000, 520, "float16"),
                                         (4097, 4199, 72, "bfloat16")])
def test_one_side_of_rounds_and_parts(env, n, m, d, dtype, side):  # noqa: F811
    torch, sps, dev = env
    x, w, t, _, ww = make(env, n, m, d, dtype, 5, masked=False)
    t[::17] = -1
    loss, gq, gi, bq, bi = exact_on_gpu(env, x, w, t, 0.5, ww)
    got = sps.dense_cross_entropy(x, w, t, 0.5, row_weights=ww, need_grad=side)
    assert ((got[0].double() - loss).abs() <= 1e-5 * (1 + loss.abs())).all()
    g, want, bar = (got[1], gq, bq) if side == "queries" else (got[2], gi, bi)
    off = (g.double() - want).abs() - bar - want.abs() * do.HALF[dtype] - do.STEP[dtype]
    if dtype != "bfloat16":
        off -= 2.0 ** -38 * 64
    assert (off <= 0).all(), (float(off.max()), int((off > 0).sum()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("low", [float("-inf"), -1e8])
def test_pieces_under_a_mask(env, dtype, low):  # noqa: F811
    """More rows than a piece holds, a run of items and single ones out: as over the items that are
    left, within the bounds of those."""
    torch, sps, dev = env
    n, m, d = 600, 1700001, 8
    x, w, t, _, ww = make(env, n, m, d, dtype, 7, masked=False)
    out = torch.rand(m, device=dev) < 0.3
    out[100000:400000] = True
    out[t.long()] = False
    t[::17] = -1
    bias = torch.zeros(m, device=dev)
    bias[out] = low
    w[out.nonzero()[::1000, 0]] = 100.0  # whatever they hold, within what -1e8 covers
    left = (~out).nonzero()[:, 0]
    place = torch.cumsum(~out, 0).int() - 1
    t2 = torch.where(t >= 0, place[t.clamp(min=0).long()], -1).int()
    loss, gq, gi, bq, bi = exact_on_gpu(env, x, w[left].contiguous(), t2, 0.5, ww, rows=300)
    got = sps.dense_cross_entropy(x, w, t, 0.5, bias, ww)
    assert ((got[0].double() - loss).abs() <= 1e-5 * (1 + loss.abs())).all()
    assert (got[2][out] == 0).all()
    for g, want, bar in ((got[1], gq, bq), (got[2][left], gi, bi)):
        # G is formed among all items' blocks: sums over m of them, not only those left
        off = (g.double() - want).abs() - 2 * bar - want.abs() * do.HALF[dtype] - do.STEP[dtype]
        if dtype != "bfloat16":
            off -= 2.0 ** -38 * 64
        assert (off <= 0).all(), (float(off.max()), int((off > 0).sum()))


@pytest.mark.parametrize("n,m,k", [(1, 300001, 64), (3, 200003, 10), (40, 131073, 33)])
def test_answers_from_many_chunks(env, n, m, k):  # noqa: F811
    """The default chunks; among them items that are equal."""
    torch, sps, dev = env
    g = torch.Generator(device=dev).manual_seed(m)
    x = torch.randn(m, 48, generator=g, device=dev)
    x[m // 2:m // 2 + 1000] = x[:1000]
    x[-7:] = x[3]
    i, q = sps.quantize_rows(x), sps.quantize_rows(torch.cat([x[3:4], x[m // 3:m // 3 + n - 1]]))
    top = sps.int8_select(q, i, k)
    s = sps.int8_scores(q, i)
    order = torch.sort(-s.double(), dim=1, stable=True).indices[:, :k]
    assert torch.equal(top.cols.long(), order)
    assert torch.equal(top.scores, s.gather(1, order))
