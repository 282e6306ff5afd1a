"""Small parts of the cross entropy's gradient: items of little probability beside one that is
nearly certain, rows of little weight."""
import pytest

import dense_oracle as do
from test_gpu_dense_ce import TYPES, check, env, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("m", [64, 300])
def test_little_probability_beside_a_certain_item(env, dtype, m):  # noqa: F811
    """Items of 2^0 to 2^-28 in one block: each one's gradient to its own step. Half a step of G, of
    its code (fp16's 11 bits of mantissa 2^-12, bf16's 10 bits 2^-11) and, of logits down to -20 in
    float32, 2^-15."""
    torch, sps, dev = env
    w = torch.zeros(m, 8, device=dev)
    w[1:, 0] = torch.linspace(-19.3, -9.0, m - 1, device=dev)
    w = w.to(getattr(torch, dtype))
    x = torch.zeros(3, 8, device=dev, dtype=w.dtype)
    x[:, 0] = 1
    t = torch.zeros(3, device=dev, dtype=torch.int32)
    _, _, gi = sps.dense_cross_entropy(x[:1], w, t[:1], 1.0, grad_dtype=torch.float32)
    z = w[:, 0].double()
    p = torch.exp(z - z.logsumexp(0))
    assert p[1:].min() >= 2.0 ** -28 and p[0] > 0.9
    off = ((gi[:, 0].double() - p).abs() / p)[1:]
    code = 2.0 ** -12 if dtype == "float16" else 2.0 ** -11
    assert (off <= do.HALF[dtype] + code + 2.0 ** -15).all(), float(off.max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", [300, 20000])
def test_weights_far_apart(env, dtype, m):  # noqa: F811
    """Weights from 1 down to 2^-20 over a softmax without favourites: every row within the bound
    that goes by the weight times the probability."""
    torch, sps, dev = env
    x, w, t, _, _ = make(env, 63, m, 40, dtype, 8, masked=False, weighted=False)
    ww = torch.exp2(-torch.arange(63, device=dev) / 3.0).float()
    x = x * 0.05
    got = sps.dense_cross_entropy(x, w, t, 1.0, None, ww, grad_dtype=torch.float32)
    check(env, got, x, w, t, 1.0, None, ww, out="float32")
