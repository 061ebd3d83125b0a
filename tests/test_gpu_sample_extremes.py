"""Sampling at the ends of what fp32 holds, against 64 bits (as in test_gpu_sample)."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
import sample_bins as sb
from test_gpu_sample import check, f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


@pytest.mark.parametrize("temperature", [1.4e-45, 1e-40, 1e-38, 2.0 ** -101, 2.0 ** -100, 1e-20])
@pytest.mark.parametrize("V", [2, 40, 3000, 102400])
def test_low_temperatures_of_far_negative_rows(temperature, V):
    """Rows whose every logit is below -2^104: differences that a low temperature takes out of fp32's range leave
    the largest logit (and its equals) alone."""
    rng = np.random.default_rng(V)
    l = -(10.0 ** rng.uniform(31.5, 38.3, (6, V))).astype(np.float32)
    l[1, V // 2:] = l[1, 0]
    l[2] = np.where(rng.random(V) < 0.5, -2e38, -3e38)
    l[3, 1:] = np.nextafter(l[3, 0], np.float32(-np.inf))
    l[4, V // 2] = -np.inf
    l[5] = l[5, 0]
    r = rng.random(6, np.float32)
    for dtype in (torch.float32, torch.bfloat16):
        x = f32(l).to(dtype)
        for s in (dict(), dict(k=2), dict(k=V // 2 + 1), dict(p=0.5), dict(p=0.9, m=0.1), dict(k=V, p=0.3)):
            check(x, r, temperature=np.full(6, temperature), **{n: np.full(6, v) for n, v in s.items()})


@pytest.mark.parametrize("b", [520, 800, 1000])
@pytest.mark.parametrize("n", [3000, 40000])
def test_a_full_bin_is_parted_alike_by_every_pass(b, n):
    """Many logits of one bin of the histogram, which are looked at again by its 1024 parts: of those at a part's
    border each pass has to think the same (whether it rounds the product before the difference or not)."""
    rng = np.random.default_rng(b + n)
    T = 10
    l = np.full((T, n + 1), -np.inf, np.float32)
    for t in range(T):
        l[t, 1:] = rng.permutation(sb.logits_of_a_bin(b, n, rng)[0])
    l[:, 0] = 0.0
    r = rng.random(T, np.float32)
    x = f32(l)
    check(x, r, k=rng.integers(2, n, T))
    check(x, r, k=n // 10 + np.arange(T))
    # b = 800: p leaves out 2^-24, and the bin's weights, of 2^-34.3 each, have more together (2^-22.7 or more), so the cut is
    # among them, where running sums lie 2^-34.3 apart: nearer than the 2^-32 within which check() does not decide
    if b != 800:
        check(x, r, k=np.full(T, n - 100), p=np.full(T, 1.0 - 2.0 ** -24))
    if b == 520 and n == 40000:  # a weight of 2^-22.3 each: together 2^-7
        check(x, r, p=1.0 - np.arange(1, T + 1) * 2.0 ** -11)


HIGH = [1e30, 2.0 ** 101, 1e37, 1.5e38, 1.75e38, 2e38, 3e38, 3.4028235e38]


@pytest.mark.parametrize("temperature", HIGH)
def test_high_temperatures(temperature):
    """Logits up to the ends of fp32 over temperatures up to there, whose reciprocals would be denormal."""
    T, V = 24, 1 << 16
    rng = np.random.default_rng(3)
    l = (rng.uniform(-1.0, 1.0, (T, V)) * min(3.4e38, 4.0 * temperature)).astype(np.float32)
    r = rng.random(T, np.float32)
    for s in (dict(), dict(p=0.7)):
        check(f32(l), r, temperature=np.full(T, temperature), **{n: np.full(T, v) for n, v in s.items()})


@pytest.mark.parametrize("temperature", HIGH)
def test_min_p_between_neighbours_at_high_temperatures(temperature):
    """Neighbouring fp32 logits around the one whose weight is min_p: each is on its side of it."""
    T, V = 20, 4000
    rng = np.random.default_rng(5)
    m = rng.uniform(0.45, 0.9, T).astype(np.float32)  # nearer to 1 / e neighbours would be closer than check() decides
    temperature = np.float32(temperature)
    top = np.float32(min(3.4e38, float(temperature)))
    l = np.empty((T, V), np.float32)
    for t in range(T):
        at = np.float32(float(top) + float(temperature) * np.log(float(m[t])))
        key = lambda f: int(f.view(np.int32)) if f >= 0 else -(int(f.view(np.int32)) & 0x7fffffff)  # noqa: E731
        keys = key(at) + np.arange(V) - V // 2
        l[t] = np.where(keys >= 0, keys, -keys | -2 ** 31).astype(np.int64).astype(np.int32).view(np.float32)
        l[t, 0] = top
    check(f32(l), rng.random(T, np.float32), temperature=np.full(T, temperature), m=m)
