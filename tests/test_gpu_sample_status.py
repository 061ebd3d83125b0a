"""What sampling records in its workspace: uniform numbers outside [0, 1)."""
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


@pytest.mark.parametrize("bad", [np.nan, -1e-30, -1.0, 1.0, 1.5, np.inf, -np.inf])
@pytest.mark.parametrize("at", [0, 6])
@pytest.mark.parametrize("V", [50, 30000, 600000])
def test_uniforms_outside_are_recorded(bad, at, V):
    """The row's token is that of 0, or the last one left; the other rows' are as ever."""
    l, r = normal(7, V, seed=V)
    l[3] = -float("inf")
    want = irm.irm_sample(l, f32(r), top_k=i32(np.full(7, 20)))[0].clone()
    x = r.copy()
    x[at] = bad
    token, _, ws = irm.irm_sample(l, f32(x), top_k=i32(np.full(7, 20)))
    with pytest.raises(irm.IrmError) as e:
        irm.device_status(ws)
    assert e.value.status == -7
    irm.device_status(ws)  # read and cleared
    left = l[at].topk(20).indices
    want[at] = left.max() if bad >= 1 else left.min()
    assert torch.equal(token, want)


def test_nothing_is_recorded_of_others():
    l, _ = normal(4, 3000)
    for r in (np.zeros(4), np.full(4, -0.0), np.full(4, 1.0 - 2.0 ** -24), np.full(4, 1e-45)):
        token, _, ws = irm.irm_sample(l, f32(r))
        irm.device_status(ws)


def test_uniforms_are_not_read_without_a_token():
    l, _ = normal(3, 400)
    _, probs, ws = irm.irm_sample(l, None, probs=torch.empty_like(l))
    irm.device_status(ws)
    assert probs.sum() > 2.99


def test_a_workspace_that_is_kept_collects():
    """One bad number among several calls on the same workspace is seen at the end."""
    l, r = normal(5, 2000)
    ws = irm.new_workspace(irm.WORKSPACE_HEADER)
    for i in range(4):
        x = r.copy()
        if i == 1:
            x[2] = 2.0
        irm.irm_sample(l, f32(x), workspace=ws)
    with pytest.raises(irm.IrmError):
        irm.device_status(ws)
    check(l, r, workspace=ws)
