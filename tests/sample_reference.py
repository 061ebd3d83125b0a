"""Sampling from logits by its definition, in 64 bits (test-side only)."""
import numpy as np


def clean(l):
    """fp32 / bf16 logits in 64 bits, NaN as -infinity, -0 as 0."""
    l = np.asarray(l, np.float64) + 0.0
    return np.where(np.isnan(l), -np.inf, l)


def kept(l, temperature=1.0, k=0, p=1.0, m=0.0):
    """(weights left [V], candidates' order, how many of it are left, how near the decisions were: the least
    distance of a weight or running sum from its border, relative to the sum or the largest weight)."""
    l = clean(l)
    V = len(l)
    order = np.argsort(-l, kind="stable")
    top = l[order[0]]
    if top == -np.inf:
        return np.zeros(V), order, 0, np.inf
    if np.isnan(temperature) or temperature <= 0:
        n, margin, w = 1, np.inf, np.where(np.arange(V) == order[0], 1.0, 0.0)
        return w, order, n, margin
    if top == np.inf:
        w = np.where(l == np.inf, 1.0, 0.0)
    else:
        with np.errstate(invalid="ignore"):
            w = np.where(l == -np.inf, 0.0, np.exp((l - top) / temperature))
    s = w[order]
    n, margin = V, np.inf
    if 0 < k < V:
        n = k
    if p <= 0:
        n = 1
    elif p < 1:
        sums = s[:n].cumsum()
        gap = (sums - s[:n]) - p * sums[-1]
        n = max(1, int((gap < 0).sum()))
        margin = np.abs(gap).min() / sums[-1]
    if m > 0:
        unsure = s[:n][s[:n] != 1.0]  # the largest logit's own weight is exact
        margin = min(margin, np.abs(unsure - m).min()) if len(unsure) else margin
        n = max(1, int((s[:n] >= m).sum()))
    if ((s == 0) | (s == 1)).all():
        margin = np.inf  # whole numbers of equal weights: every sum is exact, a border is where it is
    out = np.zeros(V)
    out[order[:n]] = s[:n]
    return out, order, n, margin


def draw(w, r):
    """(token, distance of r sum(w) from the nearest running sum, relative to the sum)."""
    c = w.cumsum()
    if c[-1] <= 0:
        return -1, np.inf
    token = int((c <= r * c[-1]).sum())
    edges = np.concatenate([[0.0], c])
    inner = edges[(edges > 0) & (edges < c[-1])]  # r = 0 and the end are no borders that rounding could move
    return min(token, int(np.nonzero(w > 0)[0][-1])), (np.abs(inner - r * c[-1]).min() / c[-1] if len(inner) else np.inf)
