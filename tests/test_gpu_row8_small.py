"""The 8-bit cache's rows of the smallest magnitudes: groups of 128 columns whose scale is near 2^-126, the least.

Products down to 2^-133, bf16's smallest step, are exact.  What the append writes has no smaller ones: its values are
bf16, whole multiples of 2^-133, and rounding one to a code (whose steps double with its magnitude) leaves a multiple.
Codes from elsewhere may: such a product is rounded to that step."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
import row8_reference as ref8
from test_gpu_tree import call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


def alone(n):
    """A batch of n rows, each seen by one node alone with weight 1 (the queries are zero): O is the row."""
    c = make([0], [n], 1, seed=0, mask="none", kv_std=0.0)
    c["mask"] = torch.from_numpy(np.packbits(np.eye(n, dtype=bool), axis=1, bitorder="little").view(np.int32).reshape(n, -1)).cuda()
    return dict(c, q_lat=torch.zeros_like(c["q_lat"]), q_rope=torch.zeros_like(c["q_rope"]))


def to_bf16(x):
    """Nearest bf16 of 64-bit values, ties to even, its steps of 2^-133 at the small end."""
    step = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -140))) - 7, -133)
    return np.round(x / step) * step


def attended(c, raw):
    """The rows as attention reads them, over the 8-bit cache and over a bf16 cache of the same values."""
    n = raw.shape[0]
    pages = c["table"][0, : -(-n // 64)].long()
    kv = torch.zeros((c["kv"].shape[0], 64, 656), dtype=torch.uint8, device="cuda")
    kv[pages] = torch.from_numpy(raw).cuda().reshape(-1, 64, 656)
    out, _, ws = call(dict(c, kv=kv))
    irm.device_status(ws)
    wide = torch.zeros((c["kv"].shape[0], 64, 576), dtype=torch.bfloat16, device="cuda")
    wide[pages] = torch.from_numpy(to_bf16(ref8.decode(raw))).to(torch.bfloat16).cuda().reshape(-1, 64, 576)
    out16, _, ws = call(dict(c, kv=wide))
    irm.device_status(ws)
    return out[:, 0].double().cpu().numpy(), out16[:, 0].double().cpu().numpy()


def test_small_scales():
    n = 128
    rng = np.random.default_rng(4)
    finite = np.array([x for x in range(256) if x & 127 != 127], np.uint8)
    raw = np.zeros((n, 656), np.uint8)
    raw[:, :512] = rng.choice(finite, (n, 512))
    raw[:, :254] = finite
    scale = 2.0 ** rng.integers(-126, -114, (n, 4)).astype(np.float64)
    scale[0], scale[1], scale[2] = [2.0 ** -126] * 4, [2.0 ** -125] * 4, [2.0 ** -124] * 4
    raw[:, 512:528] = scale.astype(np.float32).view(np.uint8)
    got, got16 = attended(alone(n), raw)
    assert np.array_equal(got, got16)
    assert np.array_equal(got, to_bf16(ref8.decode(raw)[:, :512]))


@pytest.mark.parametrize("most", [1, 3, 100, 255, 57344, 57345, 65535])
def test_appended_rows_are_exact(most):
    """Values of up to `most` steps of 2^-133: the codes' products are in bf16 what they are."""
    n = 64
    rng = np.random.default_rng(most)
    steps = rng.integers(-most, most + 1, (n, 512))
    steps[:, ::128] = most
    c = torch.from_numpy(to_bf16(steps * 2.0 ** -133)).to(torch.bfloat16).cuda()
    k = torch.zeros((n, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((1, 64, 656), dtype=torch.uint8, device="cuda")
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    row = torch.arange(n, dtype=torch.int32, device="cuda")
    ws = irm.irm_pages_append(c, k, kv, table, row, torch.zeros_like(row), encoded=True)
    irm.device_status(ws)
    raw = kv[0].cpu().numpy()
    codes, scales = ref8.encode(c.double().cpu().numpy())
    assert np.array_equal(raw[:, :512], codes)
    assert np.array_equal(np.ascontiguousarray(raw[:, 512:528]).view(np.float32), scales.astype(np.float32))
    value = ref8.decode(raw)[:, :512]
    assert np.array_equal(value, to_bf16(value))
    got, _ = attended(alone(n), raw)
    assert np.array_equal(got, value)
