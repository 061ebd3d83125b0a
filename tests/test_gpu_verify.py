"""Verification of drafted trees: whole numbers, equal to the 64-bit walk of spec_reference.verify."""
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


def softmax_rows(rng, T, V, sharp):
    z = rng.standard_normal((T, V)) * sharp
    p = np.exp(z - z.max(1, keepdims=True))
    return (p / p.sum(1, keepdims=True)).astype(np.float32)


def batch(nodes, V, draft, seed=0, sharp=3.0, par="tree"):
    """Trees whose tokens are the target's likeliest (or drawn from the draft model), so that walks run deep."""
    rng = np.random.default_rng(seed)
    T = int(np.sum(nodes))
    indptr = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    target = softmax_rows(rng, T, V, sharp)
    dp = softmax_rows(rng, T, V, sharp * 0.3) * 0.5 + target * 0.5 if draft else None
    dp = dp.astype(np.float32) if draft else None
    parents, tokens = np.full(T, -1, np.int32), np.zeros(T, np.int32)
    for b in range(len(nodes)):
        lo, n = indptr[b], nodes[b]
        order = {}
        for i in range(1, n):
            u = i - 1 if par == "chain" else int(rng.integers(max(0, i - 4), i)) if par == "tree" else 0
            parents[lo + i] = u
            if draft:
                tokens[lo + i] = rng.choice(V, p=dp[lo + u].astype(np.float64) / dp[lo + u].astype(np.float64).sum())
            else:
                k = order.get(u, 0)
                order[u] = k + 1
                tokens[lo + i] = np.argsort(-target[lo + u], kind="stable")[min(k, V - 1)]
    return dict(indptr=indptr, target=target, draft=dp, tokens=tokens, parents=parents,
                r=rng.random(T).astype(np.float32))


def call(c, max_path=None, **kw):
    dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    return irm.irm_tree_verify(dev(c["target"]), dev(c["tokens"]), dev(c["parents"]), dev(c["r"]), c["indptr"],
                               draft_probs=dev(c["draft"]), max_path=max_path, **kw)


def check(c, n_accept, path, token, max_path=None, requests=None):
    n_accept, path, token = (x.cpu().numpy() for x in (n_accept, path, token))
    depth = []
    for b in range(len(c["indptr"]) - 1) if requests is None else requests:
        lo, hi = c["indptr"][b], c["indptr"][b + 1]
        want = ref.verify(c["target"][lo:hi], None if c["draft"] is None else c["draft"][lo:hi], c["tokens"][lo:hi],
                          c["parents"][lo:hi], c["r"][lo:hi], path.shape[1])
        got = (int(n_accept[b]), path[b, :n_accept[b]].tolist(), int(token[b]))
        assert got == want, f"request {b}: {got} instead of {want}"
        assert (path[b, n_accept[b]:] == -1).all()
        depth.append(want[0])
    return depth


def run_and_check(c, max_path=None):
    n, path, token, ws = call(c, max_path)
    irm.device_status(ws)
    return check(c, n, path, token, max_path)


@pytest.mark.parametrize("V", [1, 2, 3, 4, 63, 1000, 4096, 5001, 102400])
@pytest.mark.parametrize("draft", [False, True])
def test_vocabularies(V, draft):
    depth = run_and_check(batch([8, 5, 1], V, draft, seed=V))
    assert len(depth) == 3


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("par", ["chain", "tree", "star"])
def test_tree_shapes(draft, par):
    depth = run_and_check(batch([40, 33, 32, 31, 64, 2], 300, draft, seed=3, par=par, sharp=4.0))
    assert max(depth) > 1 or draft


@pytest.mark.parametrize("B", [1, 39, 77, 160, 400])
@pytest.mark.parametrize("draft", [False, True])
def test_batch_sizes(B, draft):
    """A request's row spread over 8, 4, 2 and 1 blocks."""
    run_and_check(batch([5] * B, 1200, draft, seed=B))


@pytest.mark.parametrize("B", [1, 50])
def test_largest_vocabulary(B):
    """2^20 entries: a flat row, where every entry counts, with borders next to the uniform numbers."""
    V, rng = 1 << 20, np.random.default_rng(B)
    target = torch.rand((B, V), device="cuda") + 0.5
    target /= target.sum(1, keepdim=True)
    c = dict(indptr=np.arange(B + 1, dtype=np.int32), target=target.cpu().numpy(), draft=None, tokens=np.zeros(B, np.int32),
             parents=np.full(B, -1, np.int32), r=rng.random(B).astype(np.float32))
    if B == 1:
        c["r"][0] = np.nextafter(np.float32(1), np.float32(0))
    n, path, token, ws = call(c)
    irm.device_status(ws)
    check(c, n, path, token)


def test_largest_tree():
    run_and_check(batch([1024], 50, False, seed=5))


def test_ragged_batch_with_empty_trees():
    run_and_check(batch([0, 3, 1, 0, 17, 0], 200, False, seed=6))


def test_many_requests():
    """More requests than one launch's parameters carry; checked in full."""
    rng = np.random.default_rng(7)
    run_and_check(batch(rng.integers(0, 6, 2500).tolist(), 33, False, seed=7))


@pytest.mark.parametrize("draft", [False, True])
def test_duplicate_siblings(draft):
    c = batch([9], 6, draft, seed=8, par="star")
    c["tokens"][1:] = [2, 2, 5, 2, 5, 1, 1, 0]
    for seed in range(20):
        c["r"] = np.random.default_rng(seed).random(9).astype(np.float32)
        run_and_check(c)


def test_exact_borders():
    """Probabilities in eighths: uniform numbers exactly on the borders go to the higher token, and an exact
    tie of the acceptance test is a rejection."""
    p = np.array([[2, 0, 3, 0, 1, 2]], np.float32) / 8
    for r0, token in ((0.0, 0), (0.249, 0), (0.25, 2), (0.625, 4), (0.75, 5), (0.999, 5)):
        c = dict(indptr=np.array([0, 1], np.int32), target=p, draft=None, tokens=np.zeros(1, np.int32),
                 parents=np.full(1, -1, np.int32), r=np.array([r0], np.float32))
        _, _, t, _ = call(c)
        assert int(t[0]) == token, r0
    c = dict(indptr=np.array([0, 2], np.int32), target=np.repeat(p, 2, 0), draft=None, tokens=np.array([0, 0], np.int32),
             parents=np.array([-1, 0], np.int32), r=np.array([0.0, 0.25], np.float32))
    n, _, t, _ = call(c)
    assert int(n[0]) == 1 and int(t[0]) == 2  # 0.25 * 1 < 0.25 is false; token 0 has left the row
    c["r"][1] = np.nextafter(np.float32(0.25), np.float32(0))
    assert int(call(c)[0][0]) == 2


def test_greedy_target():
    """One-hot target rows (temperature 0): the drafts are accepted where they are the target's choice."""
    rng = np.random.default_rng(9)
    c = batch([12, 12], 40, False, seed=9, par="chain")
    best = rng.integers(0, 40, 24)
    c["target"] = np.eye(40, dtype=np.float32)[best]
    c["tokens"][1:6] = best[0:5]
    c["tokens"][6] = (best[5] + 1) % 40
    c["tokens"][13:24] = best[12:23]
    depth = run_and_check(c)
    assert depth == [6, 12]


def test_first_token_follows_the_target():
    """20000 requests with the same rows and random numbers of their own: the first emitted token's counts
    within 6 standard deviations of the target's probabilities, with and without draft probabilities."""
    rng = np.random.default_rng(10)
    B, V = 20000, 6
    p, q = rng.dirichlet(np.ones(V)).astype(np.float32), rng.dirichlet(np.ones(V)).astype(np.float32)
    for draft in (False, True):
        kids = rng.choice(V, (B, 3), p=q.astype(np.float64) / q.astype(np.float64).sum()) if draft else np.tile([1, 4, 2], (B, 1))
        tokens = np.concatenate([np.zeros((B, 1)), kids], 1).astype(np.int32).reshape(-1)
        c = dict(indptr=(np.arange(B + 1) * 4).astype(np.int32), target=np.tile(p, (4 * B, 1)),
                 draft=np.tile(q, (4 * B, 1)) if draft else None, tokens=tokens, parents=np.tile([-1, 0, 0, 0], B).astype(np.int32),
                 r=rng.random(4 * B).astype(np.float32))
        n, path, token, ws = call(c)
        irm.device_status(ws)
        check(c, n, path, token, requests=range(0, B, 97))
        n, path, token = n.cpu().numpy(), path.cpu().numpy(), token.cpu().numpy()
        first = np.where(n > 1, tokens.reshape(B, 4)[np.arange(B), np.maximum(path[:, 1], 0)], token)
        count, pd = np.bincount(first, minlength=V), p.astype(np.float64) / p.astype(np.float64).sum()
        assert (np.abs(count - B * pd) <= 6 * np.sqrt(B * pd * (1 - pd)) + 1).all()


@pytest.mark.parametrize("max_path", [1, 2, 5])
def test_path_limit(max_path):
    depth = run_and_check(batch([20, 20, 3], 50, False, seed=11, par="chain", sharp=6.0), max_path)
    assert max(depth) <= max_path


def test_strided_and_misaligned_rows():
    """Rows inside wider buffers, at starts that no vector load may use."""
    c = batch([6, 6], 1001, True, seed=12)
    want = [x.cpu() for x in call(c)[:3]]
    T = 12
    for off in (0, 1, 3):
        t, d = (torch.zeros((T, 1100), device="cuda") for _ in range(2))
        t[:, off:off + 1001] = torch.from_numpy(c["target"])
        d[:, off:off + 1001] = torch.from_numpy(c["draft"])
        dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
        got = irm.irm_tree_verify(t[:, off:off + 1001], dev(c["tokens"]), dev(c["parents"]), dev(c["r"]), c["indptr"],
                                  draft_probs=d[:, off:off + 1001])
        assert all(torch.equal(a, b.cpu()) for a, b in zip(want, got[:3]))


def test_odd_probabilities():
    """NaN, negative and infinite entries count as 0 or 1; a row without probability gives no token."""
    c = batch([2, 2, 1], 10, False, seed=13)
    c["target"][0, 3], c["target"][1, 2] = np.nan, -1.0
    c["target"][2] = 0.0
    c["target"][2, 7] = np.inf
    c["target"][4] = np.nan
    depth = run_and_check(c)
    assert int(call(c)[2][2]) == -1 and len(depth) == 3


def test_bad_tokens_and_parents_are_recorded():
    for what, value in (("tokens", 50), ("tokens", -1), ("tokens", 2 ** 31 - 1), ("parents", 5), ("parents", -1), ("parents", 2 ** 31 - 1)):
        c = batch([6, 6], 50, False, seed=14, par="chain")
        c[what][3] = value
        n, path, token, ws = call(c)
        with pytest.raises(irm.IrmError) as e:
            irm.device_status(ws)
        assert e.value.status == -7
        check(c, n, path, token)


def test_outputs_reused_and_replayed():
    c = batch([7, 5], 2000, True, seed=15)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    args = [dev(c[k]) for k in ("target", "tokens", "parents", "r")]
    d, ws = dev(c["draft"]), irm.new_workspace(256)
    out = tuple(torch.full(s, 9, dtype=torch.int32, device="cuda") for s in ((2,), (2, 7), (2,)))
    irm.irm_tree_verify(*args, c["indptr"], draft_probs=d, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        irm.irm_tree_verify(*args, c["indptr"], draft_probs=d, out=out, workspace=ws)
    for seed in range(3):
        c["r"] = np.random.default_rng(seed).random(12).astype(np.float32)
        args[3].copy_(torch.from_numpy(c["r"]))
        g.replay()
        irm.device_status(ws)
        check(c, *out)
