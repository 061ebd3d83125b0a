"""Bounds of the tree attention's output that shrink with it, as more keys share a row's weight (test-side
only).

What is rounded: the output to bf16 (half a step, 2^-8 relative), each probability to bf16 before the
product with its value (2^-8), and each score by at most e = 576 * 2^-22 * S (fp32 sums of 576
products, each addition off by at most 2^-22 of the magnitudes' sum S), which moves its
probability by at most a factor 1 + 2 e.  So the error of a row O = sum_t p_t v_t is
  d + sum_t p_t r_t v_t,  |d| <= 2^-8 |O| entry by entry,  |r_t| <= h = 2^-8 + 2 e,
and 2^-20 sum_t p_t |v_t| for the exponentials and the division.  The values of different keys are drawn
independently, 512 entries each, so they are orthogonal but for a few percent, and the norm of
the middle term stays below h sqrt(sum_t p_t^2 |v_t|^2) (reached only if every rounding were half a step: for
roundings spread evenly over a step it is about 1 / sqrt(3) of that, which leaves room for the
few percent)."""
import numpy as np

STEP = 2.0 ** -8


def scores(q, rows, seen, ctx, scale):
    """Per node of q [n, H, 576]: the visible rows' indexes, their probabilities [H, m] and S [H]."""
    for i in range(q.shape[0]):
        see = np.concatenate([np.arange(ctx), ctx + np.nonzero(seen[i])[0]])
        s = scale * (q[i] @ rows[see].T)
        p = np.exp(s - s.max(1, keepdims=True))
        yield i, see, p / p.sum(1, keepdims=True), (scale * (np.abs(q[i]) @ np.abs(rows[see]).T)).max(1)


def row_errors(o, q, rows, seen, ctx, scale):
    """Norm of each (node, head) row's error as a part of its bound, [n, H]."""
    out = np.zeros(q.shape[:2])
    for i, see, p, S in scores(q, rows, seen, ctx, scale):
        v = rows[see, :512]
        O, A = p @ v, p @ np.abs(v)
        h = STEP + 2 * 576 * 2.0 ** -22 * S
        spread = np.sqrt((p * p) @ (v * v).sum(1))
        bound = STEP * np.linalg.norm(O, axis=1) + h * spread + 2.0 ** -20 * np.linalg.norm(A, axis=1)
        out[i] = np.linalg.norm(o[i] - O, axis=1) / bound
    return out
