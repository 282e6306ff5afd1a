"""Cases of the operators on rows of scores: the best of beams and columns with
the states that follow them, distillation from a teacher's top logits (loss
and gradient), and the gradient of the scores with respect to the values of
the sparse rows.

A case is a dict; its "kind" says which operator it runs:

- "beam":    rows are groups of beams; best `k` of (beam, column) of each group
             by fl32(beam score + score), ties to the lowest beam, then column;
             then the states follow their parents.
- "select":  the running best `k` of every row over two chunks of columns.
- "distill": loss and gradient of whole rows against the teacher's list.
- "stream":  the same over two chunks of columns, each a tensor of its own.
- "grad":    gradients of the values of queries and items from that of their
             score matrix.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
_DEV = "cuda"


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one question, a first hop with four beams: the smallest call, latency alone
        dict(name="beam 1x4 of 1000", kind="beam", dtype="fp32", groups=1, beams=4, cols=1000, k=4,
             state=256),
        # 32 sequences decoded with 8 beams over a vocabulary, 64 KiB of state a beam
        dict(name="beam 32x8 of 32768", kind="beam", dtype="fp16", groups=32, beams=8, cols=32768,
             k=8, state=16384),
        # multi-hop retrieval over the whole 2M-item corpus, twice as many kept as beams, odd sizes
        dict(name="beam 16x5 of 2M", kind="beam", dtype="fp32", groups=16, beams=5, cols=1999999,
             k=10, state=1001),
        # a teacher's top 100 of 50,000 queries while chunks of 8192 items stream by (two of them)
        dict(name="select 50000x8192x2", kind="select", dtype="fp32", rows=50000, cols=16384, k=100),
        # a handful of rows against 1000 candidates: latency
        dict(name="distill 8x1000", kind="distill", dtype="fp32", rows=8, cols=1000, k=8, rest=False,
             tau=0.05, masked=False),
        # a batch of 2000 queries against all 100,000 items
        dict(name="distill 2000x100000", kind="distill", dtype="fp32", rows=2000, cols=100000, k=64,
             rest=False, tau=0.05, masked=True),
        # a vocabulary's 16-bit logits, teacher's mass outside its list kept as one class, odd sizes
        dict(name="distill 4095x30522", kind="distill", dtype="bf16", rows=4095, cols=30522, k=100,
             rest=True, tau=2.0, masked=False),
        # half-precision chunks of 8192 items as they stream by, 10,000 queries
        dict(name="stream 10000x8192x2", kind="stream", dtype="fp16", rows=10000, cols=16384, k=32,
             rest=True, tau=0.05, masked=True),
        # the smallest corpus: uniform dims, few shared
        dict(name="grad 256x4096", kind="grad", dtype="fp32", rows=256, items=4096, dim=65536, nnz=20,
             zipf=0.0),
        # a training batch against one chunk, title embeddings with a skewed dictionary
        dict(name="grad 2000x8192", kind="grad", dtype="fp32", rows=2000, items=8192, dim=500000,
             nnz=43, zipf=1.1),
        # learned expansions over a word-piece vocabulary: long rows, many shared dims; 16-bit gradient
        dict(name="grad 1001x8192", kind="grad", dtype="bf16", rows=1001, items=8192, dim=30522,
             nnz=120, zipf=1.0),
        # a large batch against two chunks
        dict(name="grad 4096x16384", kind="grad", dtype="fp32", rows=4096, items=16384, dim=1200000,
             nnz=43, zipf=1.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["beam", "beam", "select", "distill", "distill", "stream", "grad", "grad"])
    dtype = rng.choice(["fp32", "fp16", "bf16"])
    if kind == "beam":
        beams, cols = rng.randint(1, 12), _log_int(rng, 500, 500000)
        groups = _log_int(rng, 1, max(1, min(256, 150000000 // (beams * cols))))
        return dict(kind=kind, dtype=dtype, groups=groups, beams=beams, cols=cols,
                    k=rng.randint(1, 2 * beams + 4), state=_log_int(rng, 1, 4096))
    if kind == "select":
        return dict(kind=kind, dtype=dtype, rows=_log_int(rng, 100, 40000),
                    cols=2 * _log_int(rng, 200, 8192), k=_log_int(rng, 1, 256))
    if kind in ("distill", "stream"):
        cols = _log_int(rng, 1000, 200000) if kind == "distill" else 2 * _log_int(rng, 300, 8192)
        return dict(kind=kind, dtype=dtype, rows=_log_int(rng, 4, min(8000, 180000000 // cols)),
                    cols=cols, k=_log_int(rng, 2, 128), rest=rng.random() < 0.5,
                    tau=rng.choice([0.05, 0.1, 1.0, 2.0]), masked=rng.random() < 0.5)
    return dict(kind=kind, dtype=dtype, rows=_log_int(rng, 32, 2500), items=_log_int(rng, 300, 12000),
                dim=_log_int(rng, 20000, 1200000), nnz=rng.randint(12, 64),
                zipf=rng.choice([0.0, 1.0, 1.1]))


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(seed)


def _scores(g, rows, cols, case):
    """Rows of scores as this library gives them (cosines, 0.1 +- 0.08), or logits."""
    x = torch.randn(rows, cols, generator=g, device=_DEV)
    x = x.mul_(0.08).add_(0.1) if case.get("tau", 0.05) < 0.5 else x.mul_(3.0)
    if case.get("masked", True):  # items that a filter has struck out
        x.masked_fill_(torch.rand(cols, generator=g, device=_DEV) < 0.02, -math.inf)
    return x


def _cdf(dim, zipf):
    w = np.arange(1, dim + 1, dtype=np.float64) ** -zipf
    return np.cumsum(w / w.sum())


def _lens(n, m, which):
    """Entries of n rows, m / 2 to 3 m / 2 and 1 row in 100 without any: the same for every seed."""
    r = np.random.RandomState(1000 * m + which)
    return r.randint(m // 2, m + m // 2 + 1, n) * (r.rand(n) >= 0.01)


def _corpus(g, n, case, which):
    """CSR of n rows: dims drawn from the law, a row's repeats moved on to the next free dim."""
    dim, m = case["dim"], case["nnz"]
    most = m + m // 2
    cdf = torch.from_numpy(_cdf(dim - most, case["zipf"])).to(_DEV)
    u = torch.rand(n, most, generator=g, device=_DEV, dtype=torch.float64)
    d = torch.searchsorted(cdf, u).clamp_(max=dim - most - 1)
    lens = torch.from_numpy(_lens(n, m, which)).to(_DEV)
    place = torch.arange(most, device=_DEV)
    d.masked_fill_(place >= lens[:, None], dim)
    d = (d.sort(dim=1).values - place).cummax(1).values + place
    indptr = torch.zeros(n + 1, dtype=torch.int32, device=_DEV)
    indptr[1:] = lens.cumsum(0)
    ix = d[place < lens[:, None]].to(torch.int32)
    v = torch.randn(ix.numel(), generator=g, device=_DEV).exp_()
    return dict(indptr=indptr, indices=ix, values=v, n=n, dim=dim)


def _shared(case, n=512):
    """Dims that a query and an item share, on average: between two small samples of rows."""
    dim, m = case["dim"], case["nnz"]
    most = m + m // 2
    cdf, place = _cdf(dim - most, case["zipf"]), np.arange(most)
    counts = []
    for which in (0, 1):
        r = np.random.RandomState(which)
        d = np.searchsorted(cdf, r.rand(n, most)).clip(max=dim - most - 1)
        keep = place < _lens(n, m, which)[:, None]
        d = np.sort(np.where(keep, d, dim), 1) - place
        d = np.maximum.accumulate(d, 1) + place
        counts.append(np.bincount(d[keep], minlength=dim))
    return float((counts[0] * counts[1]).sum()) / n / n


def prepare(case, seed):
    g, dt = _gen(seed), _DTYPES[case["dtype"]]
    s = dict(case)
    if case["kind"] == "beam":
        rows = case["groups"] * case["beams"]
        s["x"] = _scores(g, rows, case["cols"], case).to(dt)
        b = torch.randn(rows, generator=g, device=_DEV) * 0.05
        b[torch.rand(rows, generator=g, device=_DEV) < 0.1] = -math.inf  # beams that have ended
        s["beam_scores"] = b
        s["tokens"] = torch.randint(0, case["cols"], (rows, 37), generator=g, device=_DEV,
                                    dtype=torch.int32)
        s["hidden"] = torch.randn(rows, case["state"], generator=g, device=_DEV)
    elif case["kind"] == "select":
        half = case["cols"] // 2
        s["chunks"] = [_scores(g, case["rows"], half, case).to(dt) for _ in range(2)]
    elif case["kind"] in ("distill", "stream"):
        n, cols, k, tau = case["rows"], case["cols"], case["k"], case["tau"]
        k = s["k"] = min(k, cols // 2)
        x = _scores(g, n, cols, case)
        # a teacher's list: k distinct columns, most of which the student scores high too
        start = torch.randint(0, cols, (n, 1), generator=g, device=_DEV)
        step = torch.randint(1, cols // k + 1, (n, 1), generator=g, device=_DEV)
        ids = (start + step * torch.arange(k, device=_DEV)) % cols
        t = (torch.randn(n, k, generator=g, device=_DEV) * tau).sort(1, descending=True).values
        x.scatter_add_(1, ids, t.add(3 * tau))
        # lists of different lengths, some of them empty
        lens = torch.randint(max(1, k // 2), k + 1, (n, 1), generator=g, device=_DEV)
        lens[torch.rand(n, 1, generator=g, device=_DEV) < 0.01] = 0
        ids[torch.arange(k, device=_DEV) >= lens] = -1
        s["ids"], s["logits"] = ids.to(torch.int32), t
        s["lse"] = None
        if case["rest"]:  # the teacher's log sum over all columns: 5 to 50 % of its mass is outside
            out = torch.rand(n, generator=g, device=_DEV) * 0.45 + 0.05
            listed_mass = torch.where(ids >= 0, t / tau, -math.inf).logsumexp(1)
            s["lse"] = torch.where(lens[:, 0] > 0, listed_mass - torch.log1p(-out), torch.zeros_like(out))
        # a mean over the batch, scaled up where the gradient's type is narrow
        scale = 256.0 if case["dtype"] == "fp16" else 1.0 / n
        s["weights"] = torch.rand(n, generator=g, device=_DEV) * scale
        x = x.to(dt)
        if case["kind"] == "stream":
            s["chunks"] = [c.contiguous() for c in x.chunk(2, 1)]
        else:
            s["x"] = x
    else:
        s["q"] = _corpus(g, case["rows"], case, 0)
        s["i"] = _corpus(g, case["items"], case, 1)
        gm = torch.randn(case["rows"], case["items"], generator=g, device=_DEV)
        s["g"] = gm.to(dt)
    return s


# ---------------------------------------------------------------------------
# plain forms

def _best(keys, k):
    """Best k of every row of 32-bit keys, ties to the lowest place: (keys, places), -inf and -1
    where a row has fewer candidates. The order of a key and its place is that of one integer."""
    n, m = keys.shape
    bits = (keys + 0.0).view(torch.int32)  # + 0: one zero
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)
    order = (order << 32) | (0xFFFFFFFF - torch.arange(m, device=keys.device))
    order.masked_fill_(~(keys > -math.inf), torch.iinfo(torch.int64).min)
    top = order.topk(min(k, m), dim=1).values
    place = 0xFFFFFFFF - (top & 0xFFFFFFFF)
    there = top > torch.iinfo(torch.int64).min
    place = torch.where(there, place, -1)
    value = torch.where(there, keys.gather(1, place.clamp(min=0)), -math.inf)
    pad = (0, k - min(k, m))
    return (torch.nn.functional.pad(value, pad, value=-math.inf),
            torch.nn.functional.pad(place, pad, value=-1))


def _plain_beam(s):
    g, b, n, k = s["groups"], s["beams"], s["cols"], s["k"]
    keys = s["x"].float() + s["beam_scores"][:, None]
    value, place = _best(keys.view(g, b * n), k)
    there = place >= 0
    first = torch.arange(g, device=place.device)[:, None] * b
    parents = torch.where(there, first + place // n, -1)
    cols = torch.where(there, place % n, -1)
    # a place that stayed empty has a state of zeros
    src, live = parents.clamp(min=0).view(-1), there.view(-1, 1)
    return dict(scores=value, parents=parents.to(torch.int32), cols=cols.to(torch.int32),
                tokens=s["tokens"][src] * live, hidden=s["hidden"][src] * live)


def _plain_select(s):
    value, place = _best(torch.cat([c.float() for c in s["chunks"]], 1), s["k"])
    return dict(scores=value, cols=place.to(torch.int32))


def _plain_distill(x, s):
    tau = s["tau"]
    z = x.float() / tau
    ids = s["ids"].long()
    valid = ids >= 0
    t = torch.where(valid, s["logits"] / tau, -math.inf)
    at = ids.clamp(min=0)
    has = valid.any(1)
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1)
    lse = m[:, 0] + torch.log(total)
    zk = torch.where(valid, z.gather(1, at), 0.0)
    if s["lse"] is None:
        p = torch.exp(t - torch.where(has, t.amax(1), 0.0)[:, None])
        p = torch.where(has[:, None], p / p.sum(1, keepdim=True), 0.0)
    else:
        p = torch.exp(t - s["lse"][:, None])
    entropy = torch.where(p > 0, p * torch.log(p), 0.0).sum(1)
    mass = p.sum(1)
    loss = entropy - torch.where(p > 0, p * zk, 0.0).sum(1)
    q = e / total[:, None]
    if s["lse"] is None:
        loss = loss + mass * lse
        grad = q * mass[:, None]
    else:
        rest = (1 - mass).clamp(min=0)
        listed_e = torch.where(valid, e.gather(1, at), 0.0)
        # the columns outside the list, summed without those inside it
        outside = e.scatter_add(1, at, -listed_e)
        z_rest = outside.sum(1)
        loss = loss + rest * (torch.log(rest) - torch.log(z_rest) - m[:, 0]) + (mass + rest) * lse
        grad = q * (mass + rest)[:, None] - outside * (rest / z_rest)[:, None]
    grad = grad.scatter_add(1, at, -p)
    grad = grad * (s["weights"] / tau)[:, None]
    return torch.where(has, loss, 0.0), torch.where(has[:, None], grad, 0.0).to(x.dtype)


def _unit(m):
    count = (m["indptr"][1:] - m["indptr"][:-1]).long()
    row = torch.repeat_interleave(torch.arange(m["n"], device=count.device), count)
    norm = torch.zeros(m["n"], device=count.device).index_add_(0, row, m["values"].square()).sqrt()
    return row, norm, m["values"] / norm[row]


def _through_norm(du, u, row, norm):
    along = torch.zeros_like(norm).index_add_(0, row, u * du)
    return (du - u * along[row]) / norm[row]


def _plain_grad(s):
    q, i, g = s["q"], s["i"], s["g"].float()
    (rq, nq, u), (ri, ni, w) = _unit(q), _unit(i)
    # dense rows over the dims that the queries hold: no other dim is shared
    dims, dq = torch.unique(q["indices"], return_inverse=True)
    di = torch.searchsorted(dims, i["indices"]).clamp(max=dims.numel() - 1)
    shared = dims[di] == i["indices"]
    dense_i = torch.zeros(i["n"], dims.numel(), device=w.device)
    dense_i[ri[shared], di[shared]] = w[shared]
    du = (g @ dense_i)[rq, dq]
    dense_q = torch.zeros(q["n"], dims.numel(), device=w.device)
    dense_q[rq, dq] = u
    dw = torch.where(shared, (g.t() @ dense_q)[ri, di], 0.0)
    return dict(queries=_through_norm(du, u, rq, nq), items=_through_norm(dw, w, ri, ni))


# ---------------------------------------------------------------------------
# the framework's calls

def _own_beam(s):
    import sparse_embedding_exact_amd as sps
    step = sps.beam_select(s["x"], s["beam_scores"], s["beams"], s["k"])
    tokens, hidden = sps.reorder_states([s["tokens"], s["hidden"]], step.parents)
    return dict(scores=step.scores, parents=step.parents, cols=step.cols, tokens=tokens,
                hidden=hidden)


def _own_select(s):
    import sparse_embedding_exact_amd as sps
    a, b = s["chunks"]
    top = sps.top_rows(a.shape[0], s["k"], a.device)
    sps.select_chunk(a, top, 0, first=True)
    sps.select_chunk(b, top, a.shape[1])
    return dict(scores=top.scores, cols=top.cols)


def _own_distill(s):
    import sparse_embedding_exact_amd as sps
    return sps.distill(s["x"], s["ids"], s["logits"], temperature=s["tau"], teacher_lse=s["lse"],
                       row_weights=s["weights"])


def _own_stream(s):
    import sparse_embedding_exact_amd as sps
    a, b = s["chunks"]
    n = a.shape[1]
    d = sps.distill_prepare(s["ids"], s["logits"], 2 * n, temperature=s["tau"], teacher_lse=s["lse"])
    sps.distill_chunk(d, a, 0, first=True)
    sps.distill_chunk(d, b, n)
    loss = sps.distill_loss(d)
    return loss, (sps.distill_chunk_grad(d, a, 0, s["weights"]),
                  sps.distill_chunk_grad(d, b, n, s["weights"]))


def _own_grad(s):
    import sparse_embedding_exact_amd as sps
    q, i = (sps.CSR(m["indptr"], m["indices"], m["values"], m["n"], m["dim"])
            for m in (s["q"], s["i"]))
    gq, gi = sps.cosine_grad(q, i, s["g"])
    return dict(queries=gq, items=gi)


def run(s):
    kind = s["kind"]
    if own:
        return {"beam": _own_beam, "select": _own_select, "distill": _own_distill,
                "stream": _own_stream, "grad": _own_grad}[kind](s)
    if kind == "beam":
        return _plain_beam(s)
    if kind == "select":
        return _plain_select(s)
    if kind == "distill":
        return _plain_distill(s["x"], s)
    if kind == "stream":
        loss, grad = _plain_distill(torch.cat(s["chunks"], 1), s)
        a, b = grad.chunk(2, 1)
        return loss, (a.contiguous(), b.contiguous())
    return _plain_grad(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    size = _SIZE[case["dtype"]]
    if case["kind"] == "beam":
        rows, kept = case["groups"] * case["beams"], case["groups"] * case["k"]
        n = rows * case["cols"]
        state = 4 * (37 + case["state"])
        # a state's rows are read where a place took them: each parent once
        return dict(bytes=n * size + 4 * rows + 12 * kept + state * (min(rows, kept) + kept),
                    flops=2 * n)
    if case["kind"] == "select":
        n = case["rows"] * case["cols"]
        return dict(bytes=n * size + 8 * case["rows"] * case["k"], flops=n)
    if case["kind"] in ("distill", "stream"):
        n, rows, k = case["rows"] * case["cols"], case["rows"], min(case["k"], case["cols"] // 2)
        return dict(bytes=2 * n * size + rows * (8 * k + 12), flops=8 * n)
    n, m = case["rows"], case["items"]
    nnz = float(_lens(n, case["nnz"], 0).sum() + _lens(m, case["nnz"], 1).sum())
    return dict(bytes=n * m * size + 12 * nnz + 4 * (n + m), flops=4 * n * m * _shared(case))


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rows(keys64, keys32, k):
    """By sorting: 64-bit keys of the places that the 32-bit ones put first."""
    n, m = keys32.shape
    order = torch.sort(-torch.where(torch.isnan(keys32), -math.inf, keys32), dim=1, stable=True)
    place = order.indices[:, :k]
    there = order.values[:, :k] < math.inf
    value = torch.where(there, keys64.gather(1, place), -math.inf)
    place = torch.where(there, place, -1)
    if k > m:
        value = torch.cat([value, value.new_full((n, k - m), -math.inf)], 1)
        place = torch.cat([place, place.new_full((n, k - m), -1)], 1)
    return value, place


def _exact_beam(s):
    g, b, n = s["groups"], s["beams"], s["cols"]
    keys64 = s["x"].double() + s["beam_scores"].double()[:, None]
    keys32 = keys64.float()  # one sum of 32-bit terms, rounded once: the operator's own keys
    value, place = _exact_rows(keys64.view(g, -1), keys32.view(g, -1), s["k"])
    row = torch.div(place, n, rounding_mode="floor")
    parents = torch.where(place < 0, -1, row + b * torch.arange(g, device=place.device).view(-1, 1))
    flat = parents.view(-1)
    hidden = torch.zeros(flat.numel(), s["state"], dtype=torch.float64, device=flat.device)
    hidden[flat >= 0] = s["hidden"].double()[flat[flat >= 0]]
    return dict(scores=value, parents=parents.int(),
                cols=torch.where(place < 0, -1, place - row * n).int(), tokens=None, hidden=hidden)


def _exact_distill(x, s):
    n, cols = x.shape
    tau = float(s["tau"])
    z = x.double() / tau
    row, col = (s["ids"] >= 0).nonzero(as_tuple=True)
    at = s["ids"][row, col].long()
    t = s["logits"].double()[row, col] / tau
    new = lambda fill=0.0: torch.full((n,), fill, dtype=torch.float64, device=x.device)  # noqa: E731
    top = new(-math.inf).scatter_reduce_(0, row, t, "amax")
    if s["lse"] is None:
        p = torch.exp(t - top[row])
        p = p / new().index_add_(0, row, p)[row]
    else:
        p = torch.exp(t - s["lse"].double()[row])
    rest = (1 - new().index_add_(0, row, p)).clamp(min=0) if s["lse"] is not None else new()
    lse = torch.logsumexp(z, 1)
    loss = new().index_add_(0, row, p * (torch.log(p) - (z[row, at] - lse[row])))
    others = z.clone()
    others[row, at] = -math.inf
    lse_rest = torch.logsumexp(others, 1)
    if s["lse"] is not None:
        loss += rest * (torch.log(rest) - (lse_rest - lse))
    grad = torch.exp(z - lse[:, None])
    grad[row, at] -= p
    if s["lse"] is not None:
        grad -= rest[:, None] * torch.exp(others - lse_rest[:, None])
    has = (s["ids"] >= 0).any(1)
    grad *= (has * s["weights"].double() / tau)[:, None]
    return torch.where(has, loss, torch.zeros_like(loss)), grad


def _exact_grad(s):
    q, i, g = s["q"], s["i"], s["g"]

    def rows(m):
        r = torch.bucketize(torch.arange(m["indices"].numel(), device=_DEV),
                            m["indptr"].long(), right=True) - 1
        v = m["values"].double()
        nn = torch.zeros(m["n"], dtype=torch.float64, device=_DEV).index_add_(0, r, v * v).sqrt()
        return r, v / nn[r], nn

    (rq, u, nq), (ri, w, ni) = rows(q), rows(i)
    # every pair of a query's and an item's entry that share their dim, by the items' entries in
    # the order of their dims
    order = torch.argsort(i["indices"], stable=True)
    sorted_dims = i["indices"][order]
    lo = torch.searchsorted(sorted_dims, q["indices"])
    count = torch.searchsorted(sorted_dims, q["indices"], right=True) - lo
    eq = torch.repeat_interleave(torch.arange(count.numel(), device=_DEV), count)
    at = torch.arange(eq.numel(), device=_DEV) - (count.cumsum(0) - count)[eq] + lo[eq]
    ei = order[at]
    pair = g[rq[eq], ri[ei]].double()
    du = torch.zeros_like(u).index_add_(0, eq, pair * w[ei])
    dw = torch.zeros_like(w).index_add_(0, ei, pair * u[eq])

    def back(d, unit, r, nn):
        dot = torch.zeros_like(nn).index_add_(0, r, d * unit)
        return (d - dot[r] * unit) / nn[r]

    return dict(queries=back(du, u, rq, nq), items=back(dw, w, ri, ni))


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "beam":
        return _exact_beam(s)
    if case["kind"] == "select":
        x = torch.cat(s["chunks"], 1)
        value, place = _exact_rows(x.double(), x.float(), s["k"])
        return dict(scores=value, cols=place.int())
    if case["kind"] == "distill":
        return _exact_distill(s["x"], s)
    if case["kind"] == "stream":
        loss, grad = _exact_distill(torch.cat(s["chunks"], 1), s)
        a, b = grad.chunk(2, 1)
        return loss, (a.contiguous(), b.contiguous())
    return _exact_grad(s)
