"""Rows of scores whose elements lie past 2^31 and whose bytes lie past 2^32: the last rows must
be as right as the first."""
import numpy as np
import pytest

import distill_oracle as do

pytestmark = pytest.mark.gpu
ROWS, COLS = 300000, 8192  # 2.46e9 elements of 2 bytes


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_embedding_exact_amd as sps
    sps.load_library()
    dev = torch.device("cuda:0")
    x = torch.empty(ROWS, COLS, dtype=torch.float16, device=dev).normal_(
        generator=torch.Generator(dev).manual_seed(3))
    yield torch, sps, dev, x
    del x
    torch.cuda.empty_cache()


def test_selection(env):
    torch, sps, dev, x = env
    top = sps.top_rows(ROWS, 20, dev)
    sps.select_chunk(x, top, 7, first=True)
    for part in (slice(0, 64), slice(ROWS - 64, ROWS)):
        assert torch.equal(top.scores[part], x[part].float().topk(20, 1).values)
        assert torch.equal(x[part].float().gather(1, (top.cols[part] - 7).long()), top.scores[part])
    step = sps.beam_select(x, None, 3, 5)
    assert torch.equal(step.scores[-20:], x[-60:].float().view(20, -1).topk(5, 1).values)
    assert torch.equal(x[step.parents[-20:].long(), step.cols[-20:].long()].float(), step.scores[-20:])
    assert (step.parents[-1] >= ROWS - 3).all()


def test_states(env):
    torch, sps, dev, x = env
    turned = torch.arange(ROWS - 1, -1, -1, dtype=torch.int32, device=dev)
    y = sps.reorder_states([x], turned)[0]
    assert torch.equal(y[:99], x[-99:].flip(0)) and torch.equal(y[-99:], x[:99].flip(0))


@pytest.mark.parametrize("chunked", [False, True])
def test_distillation(env, chunked):
    torch, sps, dev, x = env
    r = np.random.RandomState(0)
    ids = torch.from_numpy((r.randint(0, 1000, (ROWS, 1)) + np.arange(8) * 1000).astype(np.int32)).to(dev)
    t = torch.from_numpy(r.randn(ROWS, 8).astype(np.float32)).to(dev)
    if chunked:
        d = sps.distill_prepare(ids, t, COLS, 1.0)
        for c in (0, 4096):
            sps.distill_chunk(d, x[:, c:c + 4096], c, first=c == 0)
        loss = sps.distill_loss(d)
        grad = torch.empty_like(x)
        for c in (0, 4096):
            sps.distill_chunk_grad(d, x[:, c:c + 4096], c, out=grad[:, c:c + 4096])
    else:
        loss, grad = sps.distill(x, ids, t, 1.0)
    for part in (slice(0, 3), slice(ROWS - 3, ROWS)):
        want = do.batch(x[part].double().cpu().numpy(), ids[part].cpu().numpy(), t[part].cpu().numpy(), 1.0)
        assert (np.abs(loss[part].double().cpu().numpy() - want[0]) <= want[2]).all()
        # float16: half a step, and half the smallest subnormal
        bar = want[3] + np.abs(want[1]) * (2.0**-11 + 2 * do.U) + 2.0**-25
        assert (np.abs(grad[part].double().cpu().numpy() - want[1]) <= bar).all()
