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
