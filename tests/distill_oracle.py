"""Distillation from a teacher's top list in float64 numpy, row by row, from its
definition, with the bounds that float32 work on it stays inside."""
import numpy as np

U = 2.0 ** -24  # half a step of float32, relative


def entries(ids, logits, n_cols):
    """(columns, logits) of the entries that take part."""
    cols, vals = [], []
    for i, t in zip(ids, logits):
        if 0 <= i < n_cols and t != -np.inf and i not in cols:
            cols.append(int(i))
            vals.append(float(t))
    return np.array(cols, dtype=np.int64), np.array(vals)


def row(x, ids, logits, tau, lse=None):
    """(loss, gradient, bound of the loss, bound of each gradient) of one row of float64
    scores; the bounds are those of float32 sums and of a final rounding left out."""
    n = len(x)
    zero = (0.0, np.zeros(n), 0.0, np.zeros(n))
    c, t = entries(ids, logits, n)
    live = ~np.isnan(x) & (x > -np.inf)
    if len(c) == 0 or not (live.any() or np.isnan(x).any()):
        return zero
    with np.errstate(all="ignore"):
        if lse is None:
            p = np.exp(t / tau - (t / tau).max())
            p, rest = p / p.sum(), 0.0
        else:
            p = np.exp(t / tau - lse)
            rest = max(0.0, 1 - p.sum()) if not np.isnan(p.sum()) else np.nan
        mass = p.sum() + rest
        m = x[~np.isnan(x)].max() if (~np.isnan(x)).any() else 0.0
        m = 0.0 if m == -np.inf else m
        d = (x - m) / tau                  # natural units, <= 0
        e = np.exp(d)
        z = e.sum()
        q = e / z
        out = np.ones(n, bool)
        out[c] = False
        z_rest = e[out].sum()
        logq = d[c] - np.log(z)
        loss = sum(pi * (np.log(pi) - lq) for pi, lq in zip(p, logq) if pi != 0)
        if rest != 0:
            loss += rest * (np.log(rest) - np.log(z_rest / z))
        g = mass * q
        if rest != 0 and z_rest != 0:
            g[out] -= rest * e[out] / z_rest
        g[c] -= p
        g /= tau
        # an exponential: its argument is one difference, one product and one rounded constant
        # (3 U relative of |d|), the function one step (2 U); a sum of 32 of them in float32 adds
        # 31 U, its factor and product 3 U, the masses' own rounding 1 U
        ad = np.where(np.isfinite(d), np.abs(d), 0.0)
        off = 3 * ad + 40
        g_bound = U * off * q * (mass + (rest * z / z_rest if rest != 0 and z_rest != 0 else 0))
        # errors of the two sums, as relative ones of both factors
        dz = U * float((q * off).sum())
        dr = U * float((e[out] * off[out]).sum() / z_rest) if z_rest != 0 else 0.0
        g_bound = g_bound + q * mass * dz
        if rest != 0 and z_rest != 0:
            g_bound[out] += (rest * e / z_rest)[out] * dr
        g_bound[c] += U * 2 * p
        g_bound /= tau
        k = p != 0
        fin = np.isfinite(logq)
        l_bound = mass * dz + rest * (dr + dz) + U * (
            abs(loss) + float((p * np.abs(logq))[k & fin].sum()) + 3 * float((p * ad[c])[k].sum())
            + float(np.abs(p[k] * np.log(p[k])).sum()) + 4 * mass)
    return float(loss), g, float(l_bound), g_bound


def batch(x, ids, logits, tau, lse=None):
    r = [row(x[i], ids[i], logits[i], tau, None if lse is None else float(lse[i]))
         for i in range(len(x))]
    return (np.array([v[0] for v in r]), np.array([v[1] for v in r]).reshape(x.shape),
            np.array([v[2] for v in r]), np.array([v[3] for v in r]).reshape(x.shape))
