"""Selection over rows of scores (running best k, beam steps, states that
follow their parents) against a sort by numpy. A key is one sum of float32
values rounded once to float32 (formed here in float64, which rounds the same),
so keys, parents and columns must be equal, not close."""
import numpy as np
import pytest

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


def oracle(x, offsets, beams, k, col_begin=0):
    """(keys, parents, columns) of every group; x float64 (rows, columns)."""
    rows, cols = x.shape
    off = np.zeros(rows) if offsets is None else offsets.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        keys = (x + off[:, None]).astype(np.float32).reshape(rows // beams, beams * cols)
    out_k = np.full((rows // beams, k), -np.inf, np.float32)
    out_p = np.full((rows // beams, k), -1, np.int64)
    out_c = np.full((rows // beams, k), -1, np.int64)
    for g, row in enumerate(keys):
        cand = np.nonzero(row > -np.inf)[0]  # not NaN, not -inf
        best = cand[np.argsort(-row[cand], kind="stable")][:k]
        out_k[g, :len(best)] = row[best]
        out_p[g, :len(best)] = g * beams + best // cols
        out_c[g, :len(best)] = col_begin + best % cols
    return out_k, out_p, out_c


def check(step, want):
    np.testing.assert_array_equal(step.scores.cpu().numpy(), want[0])
    if hasattr(step, "parents"):
        np.testing.assert_array_equal(step.parents.cpu().numpy(), want[1])
    np.testing.assert_array_equal(step.cols.cpu().numpy(), want[2])


def make(env, rows, cols, dtype, seed, kind="normal"):
    torch, _, dev = env
    r = np.random.RandomState(seed)
    if kind == "normal":
        x = r.randn(rows, cols)
    elif kind == "few":        # many equal keys, both zeros
        x = r.randint(-2, 3, (rows, cols)) * 0.5
        x[x == 0] *= np.where(r.rand((x == 0).sum()) < 0.5, 1.0, -1.0)
    elif kind == "constant":
        x = np.full((rows, cols), 0.25)
    elif kind == "rising":
        x = np.arange(cols)[None, :] / cols + r.rand(rows, 1)
    elif kind == "falling":
        x = -np.arange(cols)[None, :] / cols + r.rand(rows, 1)
    elif kind == "struck":     # -inf, the type's lowest value, +inf, NaN; row 0 all -inf, 1 all NaN
        x = r.randn(rows, cols)
        x[r.rand(rows, cols) < 0.3] = -np.inf
        x[r.rand(rows, cols) < 0.3] = float(torch.finfo(getattr(torch, dtype)).min)
        x[r.rand(rows, cols) < 0.01] = np.inf
        x[r.rand(rows, cols) < 0.1] = np.nan
        x[0] = -np.inf
        if rows > 1:
            x[1] = np.nan
        if rows > 2:           # all of a row at the lowest value but one
            x[2] = float(torch.finfo(getattr(torch, dtype)).min)
            x[2, cols // 2] = 0.5
    t = torch.from_numpy(x.astype(np.float32)).to(getattr(torch, dtype))
    return t.to(dev), t.double().numpy()


KINDS = ["normal", "few", "constant", "rising", "falling", "struck"]


@pytest.mark.parametrize("cols", [1, 7, 255, 1000, 2048, 2049, 8191, 8192, 8200, 20011])
@pytest.mark.parametrize("k", [1, 5, 100, 256])
def test_lengths(env, cols, k):
    torch, sps, dev = env
    for i, dtype in enumerate(TYPES):
        x, x64 = make(env, 3, cols, dtype, cols + k + i)
        top = sps.top_rows(3, k, dev)
        sps.select_chunk(x, top, 11, first=True)
        check(top, oracle(x64, None, 1, k, 11))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols,k", [(5, 9000, 64), (4, 70001, 256), (1030, 700, 9)])
def test_kinds(env, dtype, kind, rows, cols, k):
    torch, sps, dev = env
    x, x64 = make(env, rows, cols, dtype, rows + cols, kind)
    top = sps.top_rows(rows, k, dev)
    sps.select_chunk(x, top, first=True)
    check(top, oracle(x64, None, 1, k))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["normal", "few", "rising", "struck"])
@pytest.mark.parametrize("k", [3, 130])
def test_chunks_in_any_order(env, dtype, kind, k):
    torch, sps, dev = env
    rows, cols = 6, 21000
    x, x64 = make(env, rows, cols, dtype, 7, kind)
    off = torch.linspace(-1, 1, rows, device=dev)
    want = oracle(x64, off.cpu().numpy(), 1, k)
    cuts = [0, 1, 9000, 9001, 17000, cols]
    for order in ([0, 1, 2, 3, 4], [4, 2, 0, 3, 1]):
        top = sps.top_rows(rows, k, dev)
        for j, c in enumerate(order):
            sps.select_chunk(x[:, cuts[c]:cuts[c + 1]], top, cuts[c], offsets=off, first=j == 0)
        check(top, want)


def twice(x64, offsets, k, cols):
    """Best k of each row's columns, `cols` of them given a second time."""
    both = np.concatenate([x64, x64[:, cols]], 1)
    at = np.concatenate([np.arange(x64.shape[1]), cols])
    order = np.argsort(at, kind="stable")  # equal keys go by column
    want = oracle(both[:, order], offsets, 1, k)
    return want[0], want[1], np.where(want[2] < 0, -1, at[order][want[2]])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cols,k", [(1, 3), (40, 7), (40, 100), (3000, 5), (3000, 256), (70001, 90)])
def test_columns_offered_twice(env, dtype, kind, cols, k):
    """A column offered twice takes two places, next to each other where its key is the same;
    other columns keep theirs."""
    torch, sps, dev = env
    x, x64 = make(env, 3, cols, dtype, cols + k, kind)
    off = torch.linspace(-1, 1, 3, device=dev)
    cut = cols // 3
    for parts in ([(0, cols), (0, cols)], [(0, cols), (cut, cols)], [(cut, cols), (0, cols)],
                  [(0, cols), (0, cut), (cut, cols)]):
        top = sps.top_rows(3, k, dev)
        for j, (a, b) in enumerate(parts):
            sps.select_chunk(x[:, a:b], top, 5 + a, offsets=off, first=j == 0)
        seen = np.zeros(cols, int)
        for a, b in parts:
            seen[a:b] += 1
        want = twice(x64, off.cpu().numpy(), k, np.nonzero(seen == 2)[0])
        check(top, (want[0], None, np.where(want[2] < 0, -1, want[2] + 5)))


def test_strides_and_alignment(env):
    torch, sps, dev = env
    for dtype in TYPES:
        wide, _ = make(env, 4, 5000, dtype, 3)
        for a, b in ((1, 4999), (3, 2052), (7, 8), (5, 5)):
            x = wide[:, a:b]  # any element alignment, ld above the columns, no column at all
            top = sps.top_rows(4, 10, dev)
            sps.select_chunk(x, top, a, first=True)
            check(top, oracle(x.double().cpu().numpy(), None, 1, 10, a))


def test_columns_to_the_largest(env):
    torch, sps, dev = env
    x, x64 = make(env, 2, 300, "float32", 5)
    begin = 2**31 - 2 - 300
    top = sps.top_rows(2, 40, dev)
    sps.select_chunk(x, top, begin, first=True)
    check(top, oracle(x64, None, 1, 40, begin))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("groups,beams,cols,k", [(1, 4, 1000, 4), (3, 5, 9001, 10), (2, 3, 70000, 256),
                                                 (300, 4, 500, 8), (2, 1, 40, 60), (2, 40, 3, 7),
                                                 (3, 3, 5461, 20), (1, 7, 2341, 256)])
def test_beams(env, dtype, kind, groups, beams, cols, k):
    torch, sps, dev = env
    rows = groups * beams
    x, x64 = make(env, rows, cols, dtype, rows * 3 + cols, kind)
    r = np.random.RandomState(rows)
    b = (r.randint(-3, 3, rows) * 0.5).astype(np.float32)  # sums that meet across beams
    b[r.rand(rows) < 0.2] = -np.inf                        # ended beams
    b[-1] = np.nan if groups > 1 else b[-1]
    bs = torch.from_numpy(b).to(dev)
    want = oracle(x64, b, beams, k)
    check(sps.beam_select(x, bs, beams, k), want)
    # over chunks: the lists with the beams' scores as offsets, then the join
    top = sps.top_rows(rows, min(256, k + 3), dev)
    half = cols // 2
    sps.select_chunk(x[:, half:], top, half, offsets=bs, first=True)
    sps.select_chunk(x[:, :half], top, 0, offsets=bs)
    check(sps.beam_join(top, beams, k), want)


def test_sums_that_round_together(env):
    """Scores that differ but whose sums with a large beam score are equal: the lower
    column wins, not the larger score."""
    torch, sps, dev = env
    x = torch.zeros(2, 5000, device=dev)
    x[0] = torch.linspace(0, 1e-4, 5000, device=dev)
    bs = torch.tensor([4096.0, 4096.0], device=dev)
    want = oracle(x.double().cpu().numpy(), bs.cpu().numpy(), 2, 50)
    assert (want[2][0] == np.arange(50)).all()
    check(sps.beam_select(x, bs, 2, 50), want)


def test_reproducible_and_streams(env):
    torch, sps, dev = env
    x, x64 = make(env, 8, 100000, "float16", 9, "few")
    want = oracle(x64, None, 4, 16)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    steps = [sps.beam_select(x, None, 4, 16, stream=s) for s in side for _ in range(3)]
    torch.cuda.synchronize()
    for st in steps:
        check(st, want)


def test_captured_and_replayed(env):
    """Two graphs of one program, replayed in turn with eager work between."""
    torch, sps, dev = env
    x = torch.empty(8, 30000, device=dev)
    bs = torch.zeros(8, device=dev)
    state = torch.arange(8 * 10, device=dev, dtype=torch.float32).view(8, 10)
    graphs = []
    side = torch.cuda.Stream()
    for k in (4, 12):
        sps.beam_select(x.zero_(), bs, 4, k)  # sizes known before capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step = sps.beam_select(x, bs, 4, k)
            out = sps.reorder_states([state], step.parents)[0]
        graphs.append((g, step, out, k))
    for i in range(4):
        src, x64 = make(env, 8, 30000, "float32", 100 + i)
        x.copy_(src)
        for g, step, out, k in graphs:
            g.replay()
            eager = sps.beam_select(x, bs, 4, k)
            torch.cuda.synchronize()
            want = oracle(x64, bs.cpu().numpy(), 4, k)
            check(step, want)
            check(eager, want)
            np.testing.assert_array_equal(out.cpu().numpy(),
                                          state.cpu().numpy()[want[1].reshape(-1)])


@pytest.mark.parametrize("shape,dtype", [((37,), "int32"), ((3, 5), "float16"), ((), "int64"),
                                         ((16385,), "uint8"), ((1,), "uint8"), ((4096,), "float32"),
                                         ((0,), "float32")])
def test_reorder(env, shape, dtype):
    torch, sps, dev = env
    r = np.random.RandomState(1)
    rows, n = 9, 14
    t = torch.from_numpy(r.randint(0, 100, (rows,) + shape)).to(getattr(torch, dtype)).to(dev)
    p = r.randint(-1, rows, n).astype(np.int32)
    p[:3] = (-1, 2**31 - 1, -2**31)
    par = torch.from_numpy(p).to(dev)
    want = np.where(((p >= 0) & (p < rows)).reshape((n,) + (1,) * len(shape)),
                    t.cpu().numpy()[np.clip(p, 0, rows - 1)], 0)
    np.testing.assert_array_equal(sps.reorder_states([t], par)[0].cpu().numpy(), want)


def test_reorder_many_strided(env):
    """More states than one launch takes, rows inside wider tensors; what lies between
    the rows stays as it was."""
    torch, sps, dev = env
    par = torch.tensor([[2, -1], [0, 2]], dtype=torch.int32, device=dev)
    states, outs, wides = [], [], []
    for i in range(11):
        w = 1 + 13 * i
        src = torch.arange(3 * (w + 5), device=dev, dtype=torch.int32).view(3, w + 5)
        dst = torch.full((4, w + 3), -7, device=dev, dtype=torch.int32)
        states.append(src[:, 2:2 + w])
        outs.append(dst[:, 1:1 + w])
        wides.append(dst)
    sps.reorder_states(states, par, outs)
    for s, o, wide in zip(states, outs, wides):
        want = s.cpu().numpy()[[2, 0, 0, 2]]
        want[1] = 0
        np.testing.assert_array_equal(o.cpu().numpy(), want)
        edges = wide.cpu().numpy()
        assert (edges[:, 0] == -7).all() and (edges[:, -2:] == -7).all()


def test_reorder_inside_one_buffer(env):
    """From one half of a buffer to the other, the halves' rows side by side."""
    torch, sps, dev = env
    par = torch.tensor([3, 3, -1, 0, 1], dtype=torch.int32, device=dev)
    for width in (1, 7, 64, 5000):
        t = torch.arange(5 * 2 * width, device=dev, dtype=torch.int32).view(5, 2, width)
        was = t.clone()
        out = sps.reorder_states([t[:, 0]], par, [t[:, 1]])[0]
        want = was[:, 0][par.clamp(min=0).long()] * (par >= 0).view(-1, 1)
        assert torch.equal(out, want) and torch.equal(t[:, 1], want)
        assert torch.equal(t[:, 0], was[:, 0])
    with pytest.raises(sps.SpsError):  # two outputs in one place
        a, o = torch.zeros(2, 5, 8, device=dev), torch.zeros(5, 12, device=dev)
        sps.reorder_states([a[0], a[1]], par, [o[:, :8], o[:, 4:]])


def test_reorder_refuses_overlap(env):
    torch, sps, dev = env
    t = torch.zeros(8, 16, device=dev)
    par = torch.zeros(8, dtype=torch.int32, device=dev)
    with pytest.raises(sps.SpsError):
        sps.reorder_states([t], par, [t])


def test_binding_refusals(env):
    torch, sps, dev = env
    x = torch.zeros(6, 10, device=dev)
    top = sps.top_rows(6, 4, dev)
    for bad in (lambda: sps.select_chunk(x.double(), top, first=True),
                lambda: sps.select_chunk(x.t(), top, first=True),
                lambda: sps.select_chunk(x.cpu(), top, first=True),
                lambda: sps.select_chunk(x[:5], top, first=True),
                lambda: sps.select_chunk(x, top, offsets=torch.zeros(5, device=dev), first=True),
                lambda: sps.beam_select(x, None, 4),
                lambda: sps.beam_join(top, 4),
                lambda: sps.reorder_states([x], torch.zeros(3, dtype=torch.int64, device=dev)),
                lambda: sps.reorder_states([x, x[:5]], torch.zeros(3, dtype=torch.int32, device=dev))):
        with pytest.raises(AssertionError):
            bad()
    for bad in (lambda: sps.select_chunk(x, sps.top_rows(6, 257, dev), first=True),
                lambda: sps.select_chunk(x[:1].expand(6, 10), top, first=True),
                lambda: sps.select_chunk(x, top, col_begin=-1, first=True),
                lambda: sps.beam_select(x, None, 2, 0)):
        with pytest.raises(sps.SpsError):
            bad()


def test_bulk_select_and_hops(env, orc):
    """The best items of every query over a whole corpus, then a second hop whose beams are
    those items: chunks scored, joined with the first hop's scores, states following."""
    torch, sps, dev = env
    q, items, _ = synth.make_workload("mid", n_item=20000, n_query=60)
    qc, ic = sps.CSR.from_host(q, dev), sps.CSR.from_host(items, dev)
    k = 5
    top = sps.bulk_select(qc, ic, k)
    full = sps.bulk_similarity(qc, ic).cpu().numpy().astype(np.float64)
    want = oracle(full, None, 1, k)
    check(top, want)
    ref = orc.scores(q, items)
    assert np.abs(np.sort(ref, 1)[:, ::-1][:, :k] - top.scores.cpu().numpy()).max() <= 1e-5
    # second hop: the items found ask next
    beams = want[2].reshape(-1)
    hop = sps.CSR.from_host(items.take_rows(beams), dev)
    it = sps.prepare(ic, 8192)
    qq = sps.prepare_queries(hop, it)
    bs = top.scores.view(-1).clone()
    run = sps.top_rows(len(beams), 7, dev)
    buf = torch.empty(len(beams), 8192, device=dev)
    for c in range(it.num_chunks):
        sps.cosine_chunk(qq, it, c, buf)
        sps.select_chunk(buf[:, :it.chunk_len(c)], run, c * 8192, offsets=bs, first=c == 0)
    step = sps.beam_join(run, k, 7)
    full2 = sps.bulk_similarity(hop, ic)
    want2 = oracle(full2.double().cpu().numpy(), bs.cpu().numpy(), k, 7)
    check(step, want2)
    check(sps.beam_select(full2, bs, k, 7), want2)
    path = sps.reorder_states([top.cols.view(-1, 1)], step.parents)[0]
    np.testing.assert_array_equal(path.cpu().numpy()[:, 0], beams[want2[1].reshape(-1)])
