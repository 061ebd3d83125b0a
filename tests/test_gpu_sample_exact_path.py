"""Sampling where the sum that top-p takes its part of is known exactly before the row is finished from a short
list: after a top-k cut, in rows that do not stay in shared memory, and where bounds of the sum do not decide.  The
list's weights, and the sums of the warps, are then read and written again within one block, so results are
compared with 64 bits (as in test_gpu_sample) and with themselves over many calls."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
from test_gpu_sample import check, f32, i32, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


def again(l, r, times, **kw):
    """The same call many times: every result is the first one's."""
    T = l.shape[0]
    args = dict(top_k=i32(np.full(T, kw["k"])) if "k" in kw else None, top_p=f32(np.zeros(T) + kw["p"]))
    first = irm.irm_sample(l, f32(r), probs=torch.empty(l.shape, device="cuda"), **args)
    for _ in range(times):
        token, probs, _ = irm.irm_sample(l, f32(r), probs=torch.empty(l.shape, device="cuda"), **args)
        assert torch.equal(token, first[0]) and torch.equal(probs, first[1])


@pytest.mark.parametrize("T,V", [(64, 4000), (40, 32000), (300, 9000)])
@pytest.mark.parametrize("k,p", [(300, 0.3), (300, 0.5), (1000, 0.4), (2000, 0.05)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_top_p_behind_a_top_k_cut(T, V, k, p, dtype):
    """A cut of several hundreds, and few of them up to the top-p guess."""
    l, r = normal(T, V, seed=k, dtype=dtype)
    check(l, r, k=np.full(T, k), p=np.full(T, p))
    again(l, r, 20, k=k, p=p)


@pytest.mark.parametrize("dtype,V", [(torch.float32, 600000), (torch.bfloat16, 700001)])
@pytest.mark.parametrize("p", [0.2, 0.5])
def test_rows_that_do_not_stay_in_shared_memory(dtype, V, p):
    l, r = normal(4, V, seed=V, std=6.0, dtype=dtype)
    check(l, r, p=np.full(4, p))
    again(l, r, 10, p=p)


@pytest.mark.parametrize("std", [3.0, 8.0, 14.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_top_p_next_to_a_running_sum(std, dtype):
    """top_p as near to a running sum as fp32 comes, which bounds from fp32 sums cannot tell from it."""
    T, V = 60, 6000
    l, r = normal(T, V, seed=int(std), std=std, dtype=dtype)
    x = np.sort(l.double().cpu().numpy(), axis=1)[:, ::-1]
    w = np.exp(x - x[:, :1])
    part = w.cumsum(1) / w.sum(1, keepdims=True)
    for first in (0, 3, 20):
        p = np.minimum(part[np.arange(T), first + np.arange(T) % 40], 1.0 - 2.0 ** -20).astype(np.float32)
        check(l, r, p=p)
        again(l, r, 5, p=p)
