"""The sampling kernel's distance of a logit from the row's maximum and its bin, restated in numpy's fp32 (test-side only)."""
import numpy as np

BINS, OCTAVES = 1024, np.float32(43.9)
SCALE = np.float32(np.float32(BINS - 1) / OCTAVES)
f32, f64 = np.float32, np.float64


def scale_of(T):
    """(h, log2(e) / (h T)) of a temperature."""
    T = f32(T)
    h = f32(2.0 ** -24) if T > f32(2.0 ** 100) else f32(2.0 ** 24) if T < f32(2.0 ** -100) else f32(1)
    return h, f32(f32(1) / f32(h * T)) * f32(1.4426950408889634)


def octaves(l, m, T):
    with np.errstate(all="ignore"):
        h, ch = scale_of(T)
        l, m = np.asarray(l, f32), f32(m)
        d = (l.astype(f64) * f64(h) + f64(-h * m)).astype(f32)  # one rounding: the product is exact in 64 bits
        return np.where(l == m, f32(0), -np.abs(d) * ch)


def octaves_with_a_sign(l, m, T):
    """A mistake: the difference as it comes, which is +infinity once h m overflows below zero."""
    with np.errstate(all="ignore"):
        h, ch = scale_of(T)
        l, m = np.asarray(l, f32), f32(m)
        d = (l.astype(f64) * f64(h) + f64(-h * m)).astype(f32)
        return np.where(l == m, f32(0), d * ch)


def bin_of(t):
    """The bin, before anything clamps it from below."""
    with np.errstate(all="ignore"):
        x = -t * SCALE
        whole = np.where(np.abs(x) < 2.0 ** 31, np.trunc(x), np.where(x > 0, 2.0 ** 31 - 1, -2.0 ** 31))
        return np.where(t > -OCTAVES, np.minimum(BINS - 2, whole), BINS - 1)


def fine_of(t, b, fused=False):
    """The part of bin b in which t lies; fused: product and difference in one rounding."""
    t = np.asarray(t, f32)
    x = (-t.astype(f64) * f64(SCALE) - f64(b)).astype(f32) if fused else (-t * SCALE).astype(f32) - f32(b)
    return np.clip(np.trunc(x * f32(BINS)), 0, BINS - 1).astype(int)


def logits_of_a_bin(b, n, rng, T=1.0):
    """n logits, whose largest is 0 elsewhere, that lie in bin b; those whose part of it depends on the fusing first."""
    h, ch = scale_of(T)
    l = -((b + rng.random(8 * n)) / f64(SCALE) / f64(ch)).astype(f32)
    t = octaves(l, 0.0, T)
    l, t = l[bin_of(t) == b], t[bin_of(t) == b]
    differ = fine_of(t, b) != fine_of(t, b, fused=True)
    return np.concatenate([l[differ], l[~differ]])[:n], int(differ.sum())
