"""Float64 oracles of the operators on dense rows, and how far float32 work may be off.

u = 2^-24 is half a step of float32. Every bound below counts roundings: a sum of d products in
float32 is off by at most 2 d u times the sum of their magnitudes (a matrix instruction may round
twice an addition), e^x of an argument that is off by E by a factor of about 1 + E.
"""
import numpy as np

U = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}  # half a step
TINY = {"float32": 2.0 ** -126, "float16": 2.0 ** -14, "bfloat16": 2.0 ** -126}
STEP = {"float32": 2.0 ** -149, "float16": 2.0 ** -24, "bfloat16": 2.0 ** -133}  # least subnormal


def quantize(x):
    """(integers, float32 scales) of rows given in float64: nearest of 127 x / a, ties to even,
    by exact comparisons (x has at most 24 significant bits)."""
    x = np.asarray(x, np.float64)
    q = np.zeros(x.shape, np.int64)
    s = np.zeros(len(x), np.float32)
    for r, row in enumerate(x):
        if not np.isfinite(row).all():
            s[r] = np.nan
            continue
        a = np.abs(row).max() if row.size else 0.0
        if a == 0:
            continue
        s[r] = np.float32(np.float32(a) / np.float32(127))
        h = np.floor(127 * np.abs(row) / a)
        # the quotient itself may have been rounded onto the next integer
        h -= 127 * np.abs(row) < h * a
        d = 254 * np.abs(row) - (2 * h + 1) * a
        q[r] = (h + ((d > 0) | ((d == 0) & (h % 2 == 1)))) * np.sign(row)
    return q, s


def rounding(v, dtype):
    """What one rounding to the type may add."""
    return np.abs(v) * HALF[dtype] + STEP[dtype] / 2


# float32 rows are multiplied as lead + rest in fp16: a value is off by half a step of the rest,
# 2^-11 2^-11 of it, in both factors, and the product of both rests, as much again, is left out
PLANES = 3 * 2.0 ** -22
# and below 2^-14 2^-15 of the largest by an absolute half of fp16's least step, 2^-25 of 2^15
FLOOR = 2.0 ** -40


def cross_entropy(x, w, t, tau, bias=None, weights=None, dtype="float32"):
    """loss, grad of x, grad of w in float64 and the bars of each for rows of `dtype` (given as
    float64 values): a function of the type, since only then is G rounded."""
    n, m = len(x), len(w)
    d = x.shape[1]
    takes = (t >= 0) & (t < m)
    b = np.zeros(m) if bias is None else np.asarray(bias, np.float64)
    struck = np.isneginf(b)
    weight = np.ones(n) if weights is None else np.asarray(weights, np.float64)
    live = takes & (weight != 0)
    wl = np.where(struck[:, None], 0.0, w)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        z = x @ wl.T / tau + np.where(struck, 0.0, b)
        z[:, struck] = -np.inf
        top = z.max(1) if m else np.full(n, -np.inf)
        none = np.isneginf(top)
        base = np.where(none, 0.0, top)
        e = np.exp(z - base[:, None])
        total = e.sum(1)
        lse = base + np.log(total)
        at = np.where(takes, t, 0)
        zt = z[np.arange(n), at] if m else np.full(n, -np.inf)
        loss = np.where(takes & ~none, lse - zt, 0.0)
        p = e / total[:, None]
        g = p.copy()
        # an item that is struck out has no part in the gradient, be it the target
        g[np.arange(n), at] -= ~struck[at] if m else 0
        live = live & ~none
        g = np.where(live[:, None], g, 0.0)
    xl, ww = np.where(live[:, None], x, 0.0), np.where(live, weight, 0.0)
    G = g * (ww / tau)[:, None]
    # logits: products, the factor of base two, the bias; in units of z
    a = np.abs(x) @ np.abs(wl).T / tau
    wide = dtype == "float32"
    with np.errstate(invalid="ignore"):
        if wide:  # both rows' values have that floor
            top = np.abs(x).max(1, initial=0)[:, None], np.abs(wl).max(1, initial=0)[None, :]
            floor = FLOOR / tau * (top[0] * np.abs(wl).sum(1)[None, :] + top[1] * np.abs(x).sum(1)[:, None])
        else:
            floor = 0.0
        ez = ((2 * d + 8) * U + PLANES * wide) * a + floor + 4 * U * np.where(struck, 0.0, np.abs(b)) + 4 * U * np.abs(
            np.where(np.isfinite(z), z, 0.0))
    big = (ez.max(1) if m else np.zeros(n)) + 8 * U * np.abs(base)
    # sums of a block in float32 (128 columns), exponentials, logarithm
    e_loss = 2 * big + 160 * U + 4 * U * np.abs(np.where(np.isfinite(loss), loss, 0.0))

    def bars(out):
        fine = np.where(live, big, 0.0)
        rel = 4 * fine + 200 * U + (0.0 if dtype == "float32" else 2.0 ** -13)
        pm = np.where(live[:, None], p, 0.0)
        eg = pm * rel[:, None]
        # 1 - p of the target comes from the loss
        r = np.arange(n)
        eg[r, at] = np.where(live, (1 - pm[r, at]) * 4 * U + np.where(np.isfinite(e_loss), e_loss, 0.0),
                             0.0)
        eg = eg + (2.0 ** -22 if wide else HALF[dtype]) * (np.abs(g) + eg)
        ww_abs = np.abs(ww)[:, None]
        if dtype != "float32":  # codes below 2^-14 of their block's maximum
            eg = eg + 2.0 ** -27 * live[:, None]
        eG = eg * ww_abs / tau
        if dtype != "bfloat16":  # G stands 2^14 to 2^15 over the largest weight
            eG = eG + 2.0 ** -25 * 2.0 ** -14 * ww_abs.max(initial=0) / tau
        else:
            eG = eG + STEP["bfloat16"] / tau
        sums = 4 * U + PLANES * wide
        xa, wa = np.abs(xl), np.abs(wl)
        Ga = np.abs(G)
        bq = eG @ wa + (Ga @ wa) * (2 * (m + 8) * U + sums)
        bi = eG.T @ xa + (Ga.T @ xa) * (2 * (n + 8) * U + sums)
        if wide:
            bq += FLOOR * wa.max(initial=0) * Ga.sum(1)[:, None]
            bi += FLOOR * xa.max(initial=0) * Ga.sum(0)[:, None]
        gq, gi = G @ wl, G.T @ xl
        return bq + rounding(np.abs(gq) + bq, out), bi + rounding(np.abs(gi) + bi, out)

    return loss, e_loss, G @ wl, G.T @ xl, bars
