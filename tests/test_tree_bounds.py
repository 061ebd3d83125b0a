"""The bounds of tree_bounds on the CPU: a result rounded as the kernel rounds it stays inside, and results
with a planted mistake (some keys left out, a page's values in another's place) do not."""
import numpy as np
import pytest

import spec_reference as ref
import tree_bounds

SCALE = 1.0 / np.sqrt(192.0)


def bf16(x):
    """To the nearest bf16 (ties to even), in 64 bits."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + (b >> 16 & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def case(ctx, n, H, signed, seed=0):
    rng = np.random.default_rng(seed)
    rows = bf16(rng.standard_normal((ctx + n, 576)))
    if not signed:  # each page has a column of its own
        rows[:, :512] = np.arange(512) == (np.arange(ctx + n) // 64 % 512)[:, None]
    return bf16(rng.standard_normal((n, H, 576)) / np.sqrt(192.0)), rows, np.tril(np.ones((n, n), bool))


def rounded(q, rows, seen, ctx, keep=None, values=None):
    """The output with bf16 probabilities, relative to the maximum, and a bf16 result; `keep` masks keys out
    of the product alone, `values` replaces the rows there."""
    n, H = q.shape[:2]
    o = np.zeros((n, H, 512))
    for i in range(n):
        see = np.concatenate([np.arange(ctx), ctx + np.nonzero(seen[i])[0]])
        s = SCALE * (q[i] @ rows[see].T)
        p = np.exp(s - s.max(1, keepdims=True))
        w = bf16(p) if keep is None else bf16(p) * keep[see]
        o[i] = bf16(w @ (rows if values is None else values)[see, :512] / p.sum(1)[:, None])
    return o


def by_entry(o, q, rows, seen, ctx):
    """The largest error of an entry as a part of the entry-wise bound, which holds for any values."""
    O, _, A, S = ref.tree_attention(q, rows, seen, ctx, SCALE)
    e = 576 * 2.0 ** -22 * S
    return (np.abs(o - O) / (tree_bounds.STEP * np.abs(O) + (tree_bounds.STEP + 2 * e[..., None] + 2.0 ** -20) * A + 1e-30)).max()


@pytest.mark.parametrize("ctx,n", [(3, 1), (64, 2), (1000, 3), (20000, 1)])
def test_bounds_of_rows(ctx, n):
    q, rows, seen = case(ctx, n, 2, True)
    good = tree_bounds.row_errors(rounded(q, rows, seen, ctx), q, rows, seen, ctx, SCALE)
    assert good.max() <= 1.0
    if ctx < 1000:
        return
    t = np.arange(len(rows))
    piece = tree_bounds.row_errors(rounded(q, rows, seen, ctx, keep=t // 704 != 1), q, rows, seen, ctx, SCALE)
    other = rows.copy()
    other[640:704] = rows[:64]
    page = tree_bounds.row_errors(rounded(q, rows, seen, ctx, values=other), q, rows, seen, ctx, SCALE)
    assert piece.min() > 2.0 and page.min() > 2.0


@pytest.mark.parametrize("ctx", [1000, 50000])
def test_bounds_of_pages(ctx):
    """With a column for each page the entry-wise bound reads off each page's weight."""
    q, rows, seen = case(ctx, 1, 2, False)
    assert by_entry(rounded(q, rows, seen, ctx), q, rows, seen, ctx) <= 1.0
    t = np.arange(len(rows))
    if ctx <= 32768:  # a column of one page: even one of its keys is missed
        assert by_entry(rounded(q, rows, seen, ctx, keep=t != 700), q, rows, seen, ctx) > 1.0
    assert by_entry(rounded(q, rows, seen, ctx, keep=t // 64 != 11), q, rows, seen, ctx) > 20.0
    other = rows.copy()
    other[640:704] = rows[:64]
    assert by_entry(rounded(q, rows, seen, ctx, values=other), q, rows, seen, ctx) > 20.0
