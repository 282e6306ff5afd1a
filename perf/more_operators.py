"""Cases of the operators on dense rows (embeddings before they are made sparse,
or beside them): rows held in 8 bits, their products, and the loss that trains
dense rows against a whole corpus or vocabulary.

A case is a dict; its "kind" says which operator it runs:

- "rows":   rows to 8-bit integers with a scale each, and back to the values they
            stand for.
- "scores": queries to 8 bits, then their products with a corpus kept in 8 bits,
            scaled by both rows' scales.
- "loss":   softmax cross entropy of every query over all items, and with "grad"
            its gradients about both sides.
"""
import math

import torch

own = False

_DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
_DEV = "cuda"


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # a batch of fresh items joins an index: small enough that the launches count
        dict(name="rows 1000x384", kind="rows", dtype="fp32", rows=1000, dim=384),
        # a corpus of 16-bit embeddings is put into 8 bits, odd row length
        dict(name="rows 500000x333", kind="rows", dtype="bf16", rows=500000, dim=333),
        # one question against the whole 2M-item corpus
        dict(name="scores 1x2M", kind="scores", dtype="fp32", rows=1, items=1999999, dim=768,
             out="fp32"),
        # a batch of queries against one chunk of 8192 items, scores in 16 bits
        dict(name="scores 2000x8192", kind="scores", dtype="bf16", rows=2000, items=8192, dim=768,
             out="fp16"),
        # many queries against a vocabulary's rows, odd sizes, short rows: the scores' bytes count
        dict(name="scores 10001x30522", kind="scores", dtype="fp16", rows=10001, items=30522, dim=200,
             out="fp32"),
        # in-batch contrast of a small batch: latency
        dict(name="loss 256x256", kind="loss", dtype="fp32", rows=256, items=256, dim=128, tau=0.05,
             masked=False, grad=True),
        # a training batch against one chunk of items, some of them struck out
        dict(name="loss 2000x8192", kind="loss", dtype="bf16", rows=2000, items=8192, dim=768,
             tau=0.05, masked=True, grad=True),
        # a small encoder in 32 bits over a word-piece vocabulary
        dict(name="loss 1000x30522", kind="loss", dtype="fp32", rows=1000, items=30522, dim=384,
             tau=1.0, masked=False, grad=True),
        # the head of an encoder over the same vocabulary, odd number of tokens
        dict(name="loss 4095x30522", kind="loss", dtype="bf16", rows=4095, items=30522, dim=768,
             tau=1.0, masked=False, grad=True),
        # queries against all 100,000 items, odd row length, 16-bit floats with a scaled loss
        dict(name="loss 1001x100000", kind="loss", dtype="fp16", rows=1001, items=100000, dim=333,
             tau=0.05, masked=True, grad=True),
        # validation: the losses alone
        dict(name="loss 8192x30522 alone", kind="loss", dtype="fp16", rows=8192, items=30522, dim=768,
             tau=1.0, masked=False, grad=False),
        # a large batch against all 100,000 items
        dict(name="loss 8192x100000", kind="loss", dtype="bf16", rows=8192, items=100000, dim=1024,
             tau=0.05, masked=True, grad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rows", "scores", "scores", "loss", "loss", "loss"])
    dtype = rng.choice(["fp32", "fp16", "bf16"])
    if kind == "rows":
        dim = _log_int(rng, 16, 2048)
        return dict(kind=kind, dtype=dtype, dim=dim,
                    rows=_log_int(rng, 1, min(500000, 160000000 // dim)))
    if kind == "scores":
        rows, dim = _log_int(rng, 1, 10000), _log_int(rng, 32, 1536)
        return dict(kind=kind, dtype=dtype, rows=rows, dim=dim,
                    items=_log_int(rng, 500, min(500000, 300000000 // rows)),
                    out=rng.choice(["fp32", "fp16", "bf16"]))
    rows, dim = _log_int(rng, 16, 8192), _log_int(rng, 32, 1024)
    return dict(kind=kind, dtype=dtype, rows=rows, dim=dim,
                items=_log_int(rng, 100, min(150000, 300000000000 // (rows * dim))),
                tau=rng.choice([0.05, 0.1, 1.0]), masked=rng.random() < 0.5,
                grad=rng.random() < 0.75)


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=_DEV)


def _quantized(x):
    """(integers, scales) of rows: scale = largest magnitude / 127, values to the nearest
    integer of x / scale, ties to even. In 64 bits: 127 x is exact there, and its quotient is a
    tie only where the true one is."""
    q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    amax = x.abs().amax(1).float()
    for b in range(0, x.shape[0], 1 << 18):
        e = min(b + (1 << 18), x.shape[0])
        top = amax[b:e, None].double()
        ratio = x[b:e].double() * 127 / torch.where(top > 0, top, 1.0)
        q[b:e] = torch.round(ratio).to(torch.int8)
    return q, amax / 127


def prepare(case, seed):
    g, dt = _gen(seed), _DTYPES[case["dtype"]]
    n, dim = case["rows"], case["dim"]
    s = dict(case)
    if case["kind"] == "rows":
        # lengths that differ from row to row, and a row in 100 of zeros
        x = _randn(g, n, dim) * _randn(g, n, 1).exp_()
        x.masked_fill_(torch.rand(n, 1, generator=g, device=_DEV) < 0.01, 0.0)
        s["x"] = x.to(dt)
    elif case["kind"] == "scores":
        m = case["items"]
        items = torch.nn.functional.normalize(_randn(g, m, dim), dim=1)
        # every query lies near one of the items
        near = torch.randint(0, m, (n,), generator=g, device=_DEV)
        x = items[near] + _randn(g, n, dim) * (1.0 / math.sqrt(dim))
        s["x"] = torch.nn.functional.normalize(x, dim=1).to(dt)
        # the corpus as a program keeps it: 8-bit rows on 16-byte boundaries, zeros between
        q, s["scales"] = _quantized(items)
        s["values"] = torch.nn.functional.pad(q, (0, -dim % 16))
    else:
        m, tau = case["items"], case["tau"]
        if tau < 0.5:  # cosines
            w = torch.nn.functional.normalize(_randn(g, m, dim), dim=1)
            noise = 1.0 / math.sqrt(dim)
        else:  # a head's logits
            w = _randn(g, m, dim) * 0.1
            noise = 1.0
        t = torch.randint(0, m, (n,), generator=g, device=_DEV)
        x = w[t] * torch.rand(n, 1, generator=g, device=_DEV) * 2 + _randn(g, n, dim) * noise
        s["x"], s["w"] = x.to(dt), w.to(dt)
        s["bias"] = None
        if case["masked"]:  # sampling corrections, and items that a filter has struck out
            b = _randn(g, m) * 0.5
            b.masked_fill_(torch.rand(m, generator=g, device=_DEV) < 0.02, -math.inf)
            b[t] = 0.0
            s["bias"] = b
        t[torch.rand(n, generator=g, device=_DEV) < 0.02] = -1  # rows that only pad the batch
        s["targets"] = t.to(torch.int32)
        # a mean over the batch, scaled up where the gradient's type is narrow
        scale = 256.0 if case["dtype"] == "fp16" else 1.0 / n
        s["weights"] = torch.rand(n, generator=g, device=_DEV) * scale
    return s


# ---------------------------------------------------------------------------
# plain forms

def _plain_rows(s):
    q, scales = _quantized(s["x"])
    return dict(values=q.float() * scales[:, None], scales=scales)


def _plain_scores(s):
    q, scales = _quantized(s["x"])
    dots = q.float() @ s["values"][:, :s["dim"]].float().t()
    return (dots * scales[:, None] * s["scales"]).to(_DTYPES[s["out"]])


def _plain_loss(s):
    x, w, t = s["x"].float(), s["w"].float(), s["targets"].long()
    z = x @ w.t() / s["tau"]
    if s["bias"] is not None:
        z = z + s["bias"]
    valid = t >= 0
    at = t.clamp(min=0)[:, None]
    top = z.amax(1, keepdim=True)
    z_t = z.gather(1, at)[:, 0]
    e = z.sub_(top).exp_()
    total = e.sum(1)
    loss = torch.where(valid, top[:, 0] + torch.log(total) - z_t, 0.0)
    if not s["grad"]:
        return dict(loss=loss)
    g = e.div_(total[:, None])
    g.scatter_add_(1, at, torch.full_like(at, -1, dtype=g.dtype))
    g.mul_(torch.where(valid, s["weights"] / s["tau"], 0.0)[:, None])
    return dict(loss=loss, queries=(g @ w).to(s["x"].dtype), items=(g.t() @ x).to(s["x"].dtype))


# ---------------------------------------------------------------------------
# the framework's calls

def _own_rows(s):
    import sparse_embedding_exact_amd as sps
    q = sps.quantize_rows(s["x"])
    return dict(values=sps.dequantize_rows(q), scales=q.scales)


def _own_scores(s):
    import sparse_embedding_exact_amd as sps
    items = sps.Int8Rows(s["values"], s["scales"], s["dim"])
    return sps.int8_scores(sps.quantize_rows(s["x"]), items, dtype=_DTYPES[s["out"]])


def _own_loss(s):
    import sparse_embedding_exact_amd as sps
    loss, gq, gi = sps.dense_cross_entropy(s["x"], s["w"], s["targets"], temperature=s["tau"],
                                           bias=s["bias"], row_weights=s["weights"],
                                           need_grad=s["grad"])
    return dict(loss=loss, queries=gq, items=gi) if s["grad"] else dict(loss=loss)


def run(s):
    if own:
        return {"rows": _own_rows, "scores": _own_scores, "loss": _own_loss}[s["kind"]](s)
    return {"rows": _plain_rows, "scores": _plain_scores, "loss": _plain_loss}[s["kind"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    n, dim, size = case["rows"], case["dim"], _SIZE[case["dtype"]]
    if case["kind"] == "rows":
        # read, written in 8 bits, written as what they stand for
        return dict(bytes=n * dim * (size + 1 + 4) + 4 * n, flops=3 * n * dim)
    m = case["items"]
    if case["kind"] == "scores":
        return dict(bytes=n * dim * size + m * dim + 4 * m + n * m * _SIZE[case["out"]],
                    flops=2 * n * m * dim)
    fixed = (n + m) * dim * size + 8 * n
    if not case["grad"]:
        return dict(bytes=fixed, flops=2 * n * m * dim)
    # logits, and two products with their gradient
    return dict(bytes=fixed + (n + m) * dim * size + 4 * n, flops=6 * n * m * dim)


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_integers(x):
    """The nearest integer to 127 x / (the row's largest magnitude) by comparison with the
    neighbouring halves, ties to the even one; and the scales."""
    x = x.double()
    top = x.abs().max(dim=1, keepdim=True).values
    mag = 127 * x.abs()
    low = torch.floor(mag / top.masked_fill(top == 0, 1.0))
    twice = 2 * mag - (2 * low + 1) * top  # where the fraction stands about one half: exact
    up = (twice > 0) | ((twice == 0) & (low % 2 == 1))
    q = torch.where(top > 0, (low + up) * torch.sign(x), 0.0)
    return q, top[:, 0] / 127


def _exact_loss(s):
    n, m = s["rows"], s["items"]
    x, w = s["x"].double(), s["w"].double()
    z = torch.empty(n, m, dtype=torch.float64, device=_DEV)
    for b in range(0, m, 16384):
        part = torch.mm(x, w[b:b + 16384].t().contiguous()) / float(s["tau"])
        z[:, b:b + 16384] = part if s["bias"] is None else part + s["bias"][b:b + 16384].double()
    lse = torch.logsumexp(z, 1)
    rows = (s["targets"] >= 0).nonzero()[:, 0]
    cols = s["targets"][rows].long()
    loss = torch.zeros(n, dtype=torch.float64, device=_DEV)
    loss[rows] = lse[rows] - z[rows, cols]
    if not s["grad"]:
        return dict(loss=loss)
    p = torch.exp(z.sub_(lse[:, None]))
    p[rows, cols] -= 1
    factor = torch.zeros(n, dtype=torch.float64, device=_DEV)
    factor[rows] = s["weights"][rows].double() / float(s["tau"])
    p.mul_(factor[:, None])
    return dict(loss=loss, queries=p @ w, items=(x.t().contiguous() @ p).t())


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "loss":
        return _exact_loss(s)
    q, scales = _exact_integers(s["x"])
    if case["kind"] == "rows":
        return dict(values=q * scales[:, None], scales=scales)
    items = s["values"][:, :s["dim"]]
    out = torch.empty(case["rows"], case["items"], dtype=torch.float64, device=_DEV)
    for b in range(0, case["items"], 1 << 17):
        e = min(b + (1 << 17), case["items"])
        out[:, b:e] = torch.mm(q * scales[:, None],
                               (items[b:e].double() * s["scales"][b:e, None].double()).t().contiguous())
    return out
