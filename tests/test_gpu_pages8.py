"""The page operations that move rows, on an 8-bit cache: every byte against the list model."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
import spec_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def random_cache(layers, n_pages, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 256, (layers, n_pages, 64, 656), generator=g, device="cuda", dtype=torch.uint8)


@pytest.mark.parametrize("layers", [1, 3])
@pytest.mark.parametrize("lengths", [(1, 63), (64, 65), (130, 200)])
def test_fork(layers, lengths):
    kv = random_cache(layers, 40)
    want, m = kv.cpu().clone(), ref.Pages(6, 4, 40)
    seq, table, count = i32(np.zeros(6)), i32(np.full((6, 4), -1)), i32(np.zeros(40))
    ws = irm.new_workspace(irm.pages_workspace_size(6))
    new = [*lengths, 0, 0, 0, 0]
    irm.irm_pages_resize(i32(new), seq, table, count, workspace=ws)
    m.resize(new)
    irm.irm_pages_fork([0, 1, 1], [2, 3, 5], kv, seq, table, count, workspace=ws)
    for a, b, n in m.fork([0, 1, 1], [2, 3, 5]):
        want[:, b, :n] = want[:, a, :n]
    irm.device_status(ws)
    assert seq.tolist() == m.seq and table.tolist() == m.table and count.tolist() == m.ref
    assert torch.equal(kv.cpu(), want)


@pytest.mark.parametrize("layers", [1, 4, 5])
def test_compact(layers):
    rng = np.random.default_rng(layers)
    S, kv = 3, random_cache(layers, 30)
    table = rng.permutation(30)[:12].reshape(S, 4)
    base, want = rng.integers(0, 150, S), kv.cpu().clone()
    path, depth = np.full((S, 9), -1), np.array([9, 1, 5])
    for s in range(S):
        path[s, :depth[s]] = np.concatenate([[0], np.sort(rng.choice(np.arange(1, 60), depth[s] - 1, replace=False))])
        for k in range(depth[s]):
            a, b = base[s] + path[s, k], base[s] + k
            want[:, table[s, b // 64], b % 64] = want[:, table[s, a // 64], a % 64].clone()
    ws = irm.irm_pages_compact(kv, i32(table), i32(base), i32(path), i32(depth))
    irm.device_status(ws)
    assert torch.equal(kv.cpu(), want)


@pytest.mark.parametrize("n,layers", [(1, 1), (3, 5), (100, 2), (700, 1)])
def test_copy(n, layers):
    kv = random_cache(layers, 2 * n + 1)
    order = np.random.default_rng(n).permutation(2 * n + 1)
    want = kv.cpu().clone()
    want[:, order[n:2 * n]] = want[:, order[:n]]
    irm.irm_pages_copy(kv, order[:n], order[n:2 * n])
    assert torch.equal(kv.cpu(), want)
    one = kv[0].clone()
    irm.irm_pages_copy(one, order[n:2 * n], order[:n])
    assert torch.equal(one[order[:n]], one[order[n:2 * n]])


def test_rows_of_other_widths_are_refused():
    with pytest.raises(ValueError, match="656"):
        irm.irm_pages_copy(torch.zeros((4, 64, 576), dtype=torch.uint8, device="cuda"), [0], [1])
    with pytest.raises(ValueError, match="576"):
        irm.irm_pages_copy(torch.zeros((4, 64, 656), dtype=torch.bfloat16, device="cuda"), [0], [1])
