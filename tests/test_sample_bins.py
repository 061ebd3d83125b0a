"""Every logit has a bin of the histogram, at every temperature (on the CPU: a bin outside it would be a write
outside the kernel's array)."""
import numpy as np
import pytest

import sample_bins as sb

TEMPERATURES = [1.4e-45, 1e-45 * 700, 1e-38, 2.0 ** -101, 2.0 ** -100, 1e-10, 0.5, 1.0, 3.0, 1e10, 2.0 ** 100, 2.0 ** 101, 1e30, 2e38, 3.4e38, np.inf]


def rows():
    rng = np.random.default_rng(0)
    for std in (1e-45, 1e-38, 1e-30, 1.0, 1e10, 1e30, 1e31, 1e38):
        with np.errstate(over="ignore"):
            x = np.clip(rng.standard_normal(2000) * std, -3.4e38, 3.4e38).astype(np.float32)
        for part in (x, -np.abs(x), np.abs(x), np.append(-np.abs(x), -np.inf)):
            yield part
    yield np.array([-2e38, -3e38, -np.inf, -2.5e38], np.float32)
    yield np.array([np.inf, 3e38, 0.0, -3e38, -np.inf], np.float32)


@pytest.mark.parametrize("T", TEMPERATURES)
def test_bins_are_in_range(T):
    for l in rows():
        t = sb.octaves(l, l.max(), T)
        b = sb.bin_of(t)
        assert ((b >= 0) & (b < sb.BINS)).all()
        assert (t[l == l.max()] == 0).all() and not (t > 0).any()
        assert (b[l == -np.inf] == sb.BINS - 1).all() or l.max() == -np.inf


@pytest.mark.parametrize("T", [1e-38, 1e-45])
def test_a_distance_with_a_sign_is_noticed(T):
    l = np.array([-2e38, -3e38], np.float32)
    assert sb.bin_of(sb.octaves_with_a_sign(l, l.max(), T)).min() < 0


@pytest.mark.parametrize("T", [1e-38, 2.0 ** -101])
def test_far_logits_have_no_weight_at_low_temperatures(T):
    l = np.array([-2e38, -3e38, -1e32], np.float32)
    assert list(sb.bin_of(sb.octaves(l, l.max(), T))) == [sb.BINS - 1, sb.BINS - 1, 0]


@pytest.mark.parametrize("b", [520, 800, 1000])
def test_there_are_logits_whose_part_of_a_bin_depends_on_fusing(b):
    l, differ = sb.logits_of_a_bin(b, 40000, np.random.default_rng(b))
    assert len(l) == 40000 and differ > 1000
    t = sb.octaves(l, 0.0, 1.0)
    assert (sb.bin_of(t) == b).all() and np.abs(sb.fine_of(t, b) - sb.fine_of(t, b, fused=True)).max() == 1
