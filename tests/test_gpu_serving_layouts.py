"""Appending, attention over the 8-bit cache, rotation and sampling where memory and streams are not the plain ones:
far into caches and logits of more than 4 GiB, logits and probabilities in one buffer, two streams at once, two
captured graphs on one workspace.  Every result has to be, bit by bit, that of the same call on small tensors,
alone."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
from helpers import SCALE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def cache(n_pages, bits):
    if bits == 8:
        return torch.zeros((n_pages, 64, 656), dtype=torch.uint8, device="cuda")
    return torch.zeros((n_pages, 64, 576), dtype=torch.bfloat16, device="cuda")


def rows(T, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, 576), generator=g, device="cuda").to(torch.bfloat16)


class Step:
    """One token for each of B requests of n rows each: append, rotate, attend, sample."""

    def __init__(self, kv, pages, B=5, H=16, n=200, V=5000, seed=0):
        self.kv, self.B, self.n = kv, B, n
        self.table = i32(np.asarray(pages).reshape(B, -1))
        assert self.table.shape[1] * 64 >= n
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
        self.x = rows(B * n, seed)
        self.request, self.row = i32(np.repeat(np.arange(B), n)), i32(np.tile(np.arange(n), B))
        self.last = i32(np.full(B, n - 1))
        self.q, self.ql = r(B, H, 192).to(torch.bfloat16), r(B, H, 512).mul_(0.07).to(torch.bfloat16)
        self.ctx, self.indptr = np.full(B, n - 1, np.int32), np.arange(B + 1, dtype=np.int32)
        self.mask = i32(np.ones((B, 1)))
        self.logits, self.u = r(B, V) * 3, torch.rand(B, generator=g, device="cuda")
        self.p = torch.full((B,), 0.9, device="cuda")
        self.out, self.probs, self.token = torch.zeros((B, H, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, V), device="cuda"), i32(np.zeros(B))

    def __call__(self, ws, stream=None):
        irm.irm_pages_append(self.x[:, :512], self.x[:, 512:], self.kv, self.table, self.row, self.request, workspace=ws, stream=stream)
        qr = irm.irm_rope_apply(self.q[:, :, 128:], self.last, out=torch.empty_like(self.q[:, :, 128:]) if stream is None else self.qr, stream=stream)
        irm.irm_mla_attn_tree(self.ql, qr, self.ctx, self.indptr, self.kv, self.table, self.mask, SCALE, out=self.out, workspace=ws, stream=stream)
        irm.irm_sample(self.logits, self.u, top_p=self.p, probs=self.probs, token=self.token, workspace=ws, stream=stream)

    def results(self):
        return [self.kv[self.table.long()].clone(), self.out.clone(), self.probs.clone(), self.token.clone()]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [8, 16])
def test_far_into_a_large_cache(bits):
    """Pages whose bytes start beyond 4 GiB."""
    n_pages = 120000 if bits == 8 else 65000  # 5.0 and 4.8 GB
    order = np.arange(20)
    ws = irm.new_workspace(1 << 24)
    near = Step(cache(20, bits), order)
    near(ws)
    want = near.results()
    far = Step(cache(n_pages, bits), n_pages - 1 - order)
    far(ws)
    irm.device_status(ws)
    assert same(far.results(), want)
    used = torch.zeros(n_pages, dtype=torch.bool, device="cuda")
    used[far.table.long().reshape(-1)] = True
    assert not far.kv.view(torch.uint8).reshape(n_pages, -1)[~used].any()


def test_rows_of_logits_far_apart():
    """bf16 rows 2.5 GB apart, probabilities 5 GB apart."""
    V, ld = 5000, 1250000000
    g = torch.Generator(device="cuda").manual_seed(1)
    small = (torch.randn((2, V), generator=g, device="cuda") * 3).to(torch.bfloat16)
    u, p = torch.rand(2, generator=g, device="cuda"), torch.full((2,), 0.9, device="cuda")
    token, probs, _ = irm.irm_sample(small, u, top_p=p, probs=torch.empty((2, V), device="cuda"))
    wide = torch.empty(ld + V, dtype=torch.bfloat16, device="cuda").as_strided((2, V), (ld, 1))
    wide.copy_(small)
    far = torch.empty(ld + V, device="cuda").as_strided((2, V), (ld, 1))
    got, _, ws = irm.irm_sample(wide, u, top_p=p, probs=far)
    irm.device_status(ws)
    assert torch.equal(got, token) and torch.equal(far, probs)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_and_probabilities_in_one_buffer(dtype):
    """Columns of the same rows; each side keeps what it had."""
    V, T = 700, 6
    size = 4 if dtype == torch.float32 else 2
    buf = torch.full((T, 2000), 3.0, device="cuda")
    logits, probs = buf.view(dtype)[:, :V], buf[:, 900:900 + V]
    g = torch.Generator(device="cuda").manual_seed(2)
    logits.copy_(torch.randn((T, V), generator=g, device="cuda"))
    before = logits.clone()
    u, k = torch.rand(T, generator=g, device="cuda"), i32(np.full(T, 50))
    token, _, ws = irm.irm_sample(logits, u, top_k=k, probs=probs)
    irm.device_status(ws)
    want, wp, _ = irm.irm_sample(before, u, top_k=k, probs=torch.empty((T, V), device="cuda"))
    assert torch.equal(token, want) and torch.equal(probs, wp) and torch.equal(logits, before)
    assert (buf[:, 900 + V:] == 3.0).all() and (buf[:, -(-V * size // 4):900] == 3.0).all()


@pytest.mark.parametrize("bits", [8, 16])
def test_two_streams_at_once(bits):
    steps = [Step(cache(400, bits), np.random.default_rng(k).permutation(400).reshape(20, 20), B=20, n=1250, seed=k) for k in range(2)]
    need = 1 << 26
    spaces = [irm.new_workspace(need) for _ in steps]
    want = []
    for s, ws in zip(steps, spaces):
        s.qr = torch.empty_like(s.q[:, :, 128:])
        s(ws)
        torch.cuda.synchronize()
        want.append(s.results())
        for t in (s.kv, s.out, s.probs, s.token):
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(20):
        for s, ws, stream in zip(steps, spaces, streams):
            s(ws, stream)
    torch.cuda.synchronize()
    for s, ws, w in zip(steps, spaces, want):
        irm.device_status(ws)
        assert same(s.results(), w)


@pytest.mark.parametrize("bits", [8, 16])
def test_two_graphs_on_one_workspace(bits):
    """Replayed in turn: nothing of one call is left in the workspace for the next."""
    steps = [Step(cache(40, bits), np.arange(40)[::1 - 2 * k].reshape(2, 20), B=2, H=128, n=1250 - 100 * k, seed=5 + k) for k in range(2)]
    ws, want, graphs = irm.new_workspace(1 << 26), [], []
    for s in steps:
        s(ws)
        torch.cuda.synchronize()
        want.append(s.results())
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s(ws)
        graphs.append(g)
    for s in steps:
        for t in (s.kv, s.out, s.probs, s.token):
            t.zero_()
    for k in (0, 1, 1, 0):
        graphs[k].replay()
    torch.cuda.synchronize()
    irm.device_status(ws)
    for s, w in zip(steps, want):
        assert same(s.results(), w)
