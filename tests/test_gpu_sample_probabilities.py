"""Probabilities of the sampling against 64 bits, to what their arithmetic allows.

p = w / sum: the exponential of two-part exponents, ex2.approx to 2^-22 of itself; its correction's fma, the sum's
rounding to fp32, the division and the product, 2^-24 each: 2^-22 + 4 x 2^-24 = 2^-21 in all.  What the exponent
loses in two parts (44 octaves x 2^-46), the correction's second order (44 x 2^-24, squared) and the exact weights
that are summed (2^-33) are below 2^-32 together."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
import sample_reference as ref
from test_gpu_sample import f32, i32, normal

pytestmark = pytest.mark.gpu
BOUND = 2.0 ** -21 + 2.0 ** -32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


def compare(l, temperature, k=0, p=1.0):
    T, V = l.shape
    temperature, p = np.float32(temperature), np.float32(p)
    probs = torch.full((T, V), 7.0, device="cuda")
    irm.irm_sample(l, None, f32(np.full(T, temperature)), i32(np.full(T, k)), f32(np.full(T, p)), probs=probs)
    got, x = probs.double().cpu().numpy(), l.double().cpu().numpy()
    decided = 0
    for t in range(T):
        w, _, _, margin = ref.kept(x[t], float(temperature), k, float(p))
        if margin <= 2.0 ** -31 + V * 2.0 ** -43:
            continue
        decided += 1
        want = w / w.sum()
        some = want * w.sum() > 2.0 ** -42  # of the largest weight: below that it may be zero
        assert (got[t][want == 0] == 0).all()
        err = np.abs(got[t] - want)[some] / want[some]
        assert err.max() <= BOUND, f"row {t}: {err.max() / BOUND} of the bound"
    assert decided >= T - 1


@pytest.mark.parametrize("temperature", [0.05, 0.3, 0.7, 0.8, 1.0, 1.3, 3.0, 20.0])
@pytest.mark.parametrize("shift", [0.0, 1000.0])
def test_wide_rows(temperature, shift):
    l, _ = normal(6, 20000, seed=11, std=14.0)
    compare(l + shift, temperature)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2, 300, 5001, 102400, 600000])
@pytest.mark.parametrize("k,p", [(0, 1.0), (20, 1.0), (900, 1.0), (0, 0.9), (60, 0.8), (3000, 0.95)])
def test_each_way_to_the_probabilities(dtype, V, k, p):
    """Whole rows, those of at most 128 entries left, and those of a list."""
    l, _ = normal(3, V, seed=V + k, std=4.0, dtype=dtype)
    compare(l, 0.9, k, p)


@pytest.mark.parametrize("temperature", [1e-39, 1e-30, 1e-5, 1e5, 1e31, 2e38])
def test_far_temperatures(temperature):
    rng = np.random.default_rng(1)
    l = np.clip(rng.standard_normal((4, 9000)) * 4.0 * temperature, -3.4e38, 3.4e38).astype(np.float32)
    compare(f32(l), temperature)
