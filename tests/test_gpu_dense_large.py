"""Operators on dense rows where offsets pass 2^31 bytes or elements."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_embedding_exact_amd as sps
    sps.load_library()
    return torch, sps, torch.device("cuda:0")


def int8_rows(env, n, dim, seed):
    torch, sps, dev = env
    g = torch.Generator(device=dev).manual_seed(seed)
    v = torch.randint(-127, 128, (n, dim), generator=g, device=dev, dtype=torch.int8)
    return sps.Int8Rows(v, torch.rand(n, generator=g, device=dev) + 0.5, dim)


def check(env, q, i, out, rows, cols):
    """Some rows and columns: exact sums, two products, a rounding to the type."""
    torch = env[0]
    a, b = q.values[rows].double(), i.values[cols].double()
    want = (a @ b.t().contiguous()) * q.scales[rows, None].double() * i.scales[cols].double()
    got = out[rows][:, cols].double()
    step = torch.finfo(out.dtype).eps / 2
    assert ((got - want).abs() <= want.abs() * (3 * 2.0 ** -24 + step * 1.01)).all()


@pytest.mark.parametrize("n", [1, 70])
def test_scores_of_a_long_corpus(env, n):
    """3M items of 768 bytes: past 2^31 bytes of rows."""
    torch, sps, dev = env
    i = int8_rows(env, 3000001, 768, 1)
    q = int8_rows(env, n, 768, 2)
    out = sps.int8_scores(q, i)
    cols = torch.tensor([0, 1, 2796201, 2796202, 2796203, 2999999, 3000000], device=dev)
    check(env, q, i, out, torch.arange(n, device=dev), cols)
    check(env, q, i, out, torch.arange(n, device=dev), torch.arange(2999000, 3000001, device=dev))


def test_scores_past_2_31(env):
    """1100 x 2M scores in 16 bits, 4.4 GB of them."""
    torch, sps, dev = env
    i, q = int8_rows(env, 2000003, 16, 1), int8_rows(env, 1100, 16, 2)
    q.scales.div_(127 * 127 * 16)  # within fp16's range
    out = sps.int8_scores(q, i, dtype=torch.float16)
    assert out.numel() > 2 ** 31
    for rows in (torch.tensor([0, 1, 511, 1072, 1073, 1074, 1099], device=dev),):
        for cols in (torch.arange(3000, device=dev), torch.arange(1997000, 2000003, device=dev)):
            want = (q.values[rows].double() @ i.values[cols].double().t().contiguous()) \
                * q.scales[rows, None].double() * i.scales[cols].double()
            off = (out[rows][:, cols].double() - want).abs()
            assert (off <= want.abs() * (3 * 2.0 ** -24 + 2.0 ** -11 * 1.01) + 2.0 ** -25).all()


def test_many_rows_to_8_bits_and_back(env):
    """3M x 768: the values of some rows, from end to end."""
    torch, sps, dev = env
    x = torch.randn(3000001, 768, device=dev, dtype=torch.bfloat16)
    q = sps.quantize_rows(x)
    back = sps.dequantize_rows(q, torch.bfloat16)
    for rows in (slice(0, 100), slice(1398000, 1398200), slice(2796150, 2796250), slice(-100, None)):
        a = x[rows].double()
        step = a.abs().amax(1, keepdim=True) / 127
        assert ((back[rows].double() - a).abs() <= step / 2 * (1 + 1e-6) + back[rows].double().abs() * 2 ** -8).all()


def test_cross_entropy_of_many_items(env):
    """2.2M items: a piece's codes of 256 rows take more than 2^30 bytes, the transposed items' rows
    4.4 MB each, against the losses and rows of float64."""
    torch, sps, dev = env
    n, m, d = 300, 2200003, 24
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.randn(n, d, generator=g, device=dev).bfloat16()
    w = (torch.randn(m, d, generator=g, device=dev) * 0.3).bfloat16()
    t = torch.randint(0, m, (n,), generator=g, device=dev, dtype=torch.int32)
    t[:3] = torch.tensor([m - 1, 0, m - 200], device=dev, dtype=torch.int32)
    loss, gq, gi = sps.dense_cross_entropy(x, w, t)
    z = x.double() @ w.double().t().contiguous()
    lse = z.logsumexp(1)
    rows = torch.arange(n, device=dev)
    want = lse - z[rows, t.long()]
    assert ((loss.double() - want).abs() <= 1e-5 * want.abs()).all()
    z -= lse[:, None]
    p = z.exp_()
    p[rows, t.long()] -= 1
    size = p.abs() @ w.double().abs()
    want = p @ w.double()
    # G's half step and its code's eighth of one, the output's half step, float32 sums
    assert ((gq.double() - want).abs() <= size * (2.0 ** -8 * 1.2 + 1e-4) + want.abs() * 2.0 ** -8).all()
    for cols in (slice(0, 2000), slice(1000000, 1002000), slice(m - 2000, m)):
        a = p[:, cols].t().contiguous()
        want, size = a @ x.double(), a.abs() @ x.double().abs()
        assert ((gi[cols].double() - want).abs() <= size * (2.0 ** -8 * 1.2 + 1e-4)
                + want.abs() * 2.0 ** -8 + 2.0 ** -40).all()
