"""Plain models of the 8-bit cache's rows and of the position rotation (test-side only)."""
import numpy as np

# e4m3 by its definition: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN
_mag = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7) for e in range(16) for m in range(8)])
_mag[127] = np.nan
E4M3 = np.concatenate([_mag, -_mag])


def nearest_code(x):
    """Codes of finite values: to the nearest, ties to the even code, at most 448 in magnitude."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.minimum(np.searchsorted(_mag[:127], a), 126)  # first magnitude >= a
    lo = np.maximum(hi - 1, 0)
    up, down = _mag[hi] - a, a - _mag[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def encode(c):
    """Rows c [n, 512] (64 bits) -> codes [n, 512] uint8, scales [n, 4]: the smallest power of two that fits 448."""
    g = c.reshape(-1, 4, 128)
    codes, scales = np.zeros(g.shape, np.uint8), np.full(g.shape[:2], np.nan)
    for i in range(g.shape[0]):
        for k in range(4):
            most = np.abs(g[i, k]).max()
            if not np.isfinite(most):
                continue
            e = 0
            if most > 0:
                e = -126
                while e < 7 and most > 448.0 * 2.0 ** e:
                    e += 1
            scales[i, k] = 2.0 ** e
            codes[i, k] = nearest_code(g[i, k] / scales[i, k])
    return codes.reshape(-1, 512), scales


def decode(raw):
    """Bytes [n, 656] -> rows [n, 576] in 64 bits."""
    raw = np.ascontiguousarray(raw).reshape(-1, 656)
    scale = np.ascontiguousarray(raw[:, 512:528]).view(np.float32).astype(np.float64)
    k_r = (np.ascontiguousarray(raw[:, 528:]).view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return np.concatenate([E4M3[raw[:, :512]] * np.repeat(scale, 128, 1), k_r], 1)


def rotate(x, position, inv_freq=None, interleaved=False, factor=1.0):
    """x [..., 64] turned by its positions [...], pair j by position * theta_j."""
    f = 10000.0 ** (-2.0 * np.arange(32) / 64.0) if inv_freq is None else np.asarray(inv_freq, np.float64)
    a = np.asarray(position, np.float64)[..., None] * f
    c, s = factor * np.cos(a), factor * np.sin(a)
    out = np.empty(np.broadcast_shapes(x.shape, a.shape[:-1] + (64,)))
    u, v = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    out[..., u] = x[..., u] * c - x[..., v] * s
    out[..., v] = x[..., u] * s + x[..., v] * c
    return out
