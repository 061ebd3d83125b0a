"""Page operations against the list model of spec_reference.Pages; rows are compared bit for bit."""
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


CODES = {"bounds": -7, "pages": -9, "shared": -10}


class Cache:
    """The library's state and the model's, side by side."""

    def __init__(self, n_slots, max_pages, n_pages, layers=2, seed=0, one_layer=False):
        i32 = lambda *s, v=0: torch.full(s, v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.seq, self.table, self.ref = i32(n_slots), i32(n_slots, max_pages, v=-1), i32(n_pages)
        shape = (n_pages, 64, 576) if one_layer else (layers, n_pages, 64, 576)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kv = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        self.rows = self.kv.reshape(-1, n_pages, 64, 576).cpu().clone()
        self.model = ref.Pages(n_slots, max_pages, n_pages)
        self.ws = irm.new_workspace(irm.pages_workspace_size(n_slots))

    def resize(self, new):
        irm.irm_pages_resize(torch.tensor(new, dtype=torch.int32, device="cuda"), self.seq, self.table, self.ref, workspace=self.ws)
        self.model.resize(new)
        self.check()

    def fork(self, src, dst):
        irm.irm_pages_fork(src, dst, self.kv, self.seq, self.table, self.ref, workspace=self.ws)
        for a, b, n in self.model.fork(src, dst):
            self.rows[:, b, :n] = self.rows[:, a, :n]
        self.check()

    def check(self):
        m = self.model
        if m.status:
            with pytest.raises(irm.IrmError) as e:
                irm.device_status(self.ws)
            assert e.value.status in {CODES[s] for s in m.status}
            m.status.clear()
        irm.device_status(self.ws)
        assert self.seq.tolist() == m.seq
        assert self.table.tolist() == m.table
        assert self.ref.tolist() == m.ref
        assert torch.equal(self.kv.cpu().reshape(self.rows.shape).view(torch.int16), self.rows.view(torch.int16))


def test_grow_trim_free():
    c = Cache(4, 6, 20)
    c.resize([1, 64, 65, 0])
    c.resize([64, 65, 384, 10])
    c.resize([64, 63, 1, 0])
    c.resize([0, 0, 0, 0])
    c.resize([384, 384, 384, 0])
    c.resize([0, 384, 0, 384])  # releases come before allocations
    assert c.ref.sum() == 12


def test_too_few_pages_leave_every_request_that_grows():
    c = Cache(3, 8, 6)
    c.resize([100, 100, 0])
    c.resize([300, 10, 200])  # request 1 shrinks all the same; 3 + 4 pages are wanted, 3 are free
    c.resize([164, 10, 128])  # exactly the free ones
    assert (c.ref == 1).all()
    c.resize([165, 10, 129])
    c.resize([0, 0, 0])


def test_lengths_out_of_range():
    c = Cache(4, 3, 20)
    c.resize([100, 50, 0, 64])
    c.resize([193, 60, -1, 192])  # 3 pages hold 192 rows
    c.resize([2 ** 31 - 1, 0, -2 ** 31, 0])


def test_bad_state_is_recorded():
    """Page indices outside the cache, and a page released more often than held."""
    c = Cache(2, 3, 5)
    c.resize([100, 100])
    c.table[0, 1] = 5
    c.model.table[0][1] = 5
    c.resize([10, 100])
    c.ref[2] = 0
    c.model.ref[2] = 0
    c.resize([10, 10])
    c.table[1, 0] = -7
    c.model.table[1][0] = -7
    c.resize([10, 20])  # its last page cannot be looked up: it does not grow
    assert c.seq.tolist() == [10, 10]


def test_other_holders_are_kept():
    """Pages with a count of the caller's own are neither handed out nor freed."""
    c = Cache(2, 4, 10)
    c.ref[[0, 3, 4]] = torch.tensor([1, 2, 1], dtype=torch.int32, device="cuda")
    c.model.ref[0], c.model.ref[3], c.model.ref[4] = 1, 2, 1
    c.resize([200, 130])
    c.resize([0, 0])
    assert c.ref.tolist() == [1, 0, 0, 2, 1, 0, 0, 0, 0, 0]


@pytest.mark.parametrize("one_layer", [False, True])
def test_fork(one_layer):
    c = Cache(8, 4, 40, layers=1 if one_layer else 3, one_layer=one_layer)
    c.resize([130, 64, 5, 0, 0, 0, 0, 0])
    c.fork([0, 1, 2, 0], [3, 4, 5, 6])
    c.resize([192, 100, 64, 140, 64, 6, 130, 0])  # both sides of a fork may grow
    c.fork([3], [7])
    c.resize([0, 0, 0, 0, 0, 0, 0, 200])
    c.resize([0] * 8)
    assert (c.ref == 0).all()


def test_fork_of_an_empty_request_and_onto_a_full_one():
    c = Cache(5, 3, 12)
    c.resize([70, 0, 90, 0, 0])
    c.fork([1, 0], [3, 4])
    c.fork([0, 0], [2, 1])  # slot 2 holds rows: recorded, left alone; slot 1 is forked


def test_fork_without_pages_forks_none():
    c = Cache(5, 4, 5)
    c.resize([130, 70, 0, 0, 0])
    c.fork([0, 1], [2, 3])
    assert c.seq.tolist() == [130, 70, 0, 0, 0]
    c.resize([128, 64, 0, 0, 0])
    c.fork([0, 1], [2, 3])
    assert c.ref.tolist() == [2, 2, 0, 2, 0]


def test_growth_inside_a_shared_page():
    """A branch trimmed to the middle of a page that its origin still holds may not write there."""
    c = Cache(4, 4, 12)
    c.resize([200, 0, 0, 0])
    c.fork([0], [1])
    c.resize([200, 100, 0, 0])
    c.resize([201, 101, 0, 0])  # request 1 is refused, request 0 grows
    c.fork([1], [2])
    c.resize([201, 100, 110, 0])  # the fork has a copy of that page
    c.resize([0, 100, 110, 0])
    c.resize([0, 128, 110, 0])  # now the page is request 1's alone


def test_random_histories():
    rng = np.random.default_rng(3)
    c = Cache(12, 6, 50, layers=1)
    for _ in range(60):
        if rng.random() < 0.6:
            c.resize([int(x) if rng.random() < 0.5 else s for x, s in zip(rng.integers(-3, 400, 12), c.model.seq)])
        else:
            slots = rng.permutation(12)
            k = int(rng.integers(1, 5))
            c.fork(rng.choice(slots[k:], k).tolist(), slots[:k].tolist())


def test_many_slots_and_pages():
    """More requests than threads, and free pages behind many held ones; counts at an address that no
    vector load may use."""
    n = 3000
    seq, table = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.full((n, 3), -1, dtype=torch.int32, device="cuda")
    store = torch.zeros(40002, dtype=torch.int32, device="cuda")
    for refcount in (store[:40001], store[1:]):
        refcount[:] = 0
        refcount[:30000] = 1
        refcount[5], refcount[20000] = 0, 0
        rng = np.random.default_rng(2)
        m = ref.Pages(n, 3, len(refcount))
        m.ref = refcount.tolist()
        for k in range(3):
            new = rng.integers(0, 193, n).tolist()
            m.resize(new)
            ws = irm.irm_pages_resize(torch.tensor(new, dtype=torch.int32, device="cuda"), seq, table, refcount)
            irm.device_status(ws)
            assert seq.tolist() == m.seq and table.tolist() == m.table and refcount.tolist() == m.ref
        irm.irm_pages_resize(torch.zeros_like(seq), seq, table, refcount)


def test_slot_limit():
    seq, table = torch.zeros(8192, dtype=torch.int32, device="cuda"), torch.full((8192, 1), -1, dtype=torch.int32, device="cuda")
    refcount = torch.zeros(9000, dtype=torch.int32, device="cuda")
    ws = irm.irm_pages_resize(torch.full_like(seq, 3), seq, table, refcount)
    irm.device_status(ws)
    assert torch.equal(table[:, 0], torch.arange(8192, dtype=torch.int32, device="cuda")) and (seq == 3).all()


def test_many_forks():
    c = Cache(1025, 2, 1100, layers=1)
    c.resize([70] + [0] * 1024)
    c.fork([0] * 1024, list(range(1, 1025)))
    assert int(c.ref[0]) == 1025


# ----------------------------------------------------------------------------- compaction

def compact(kv, table, base, path, n_accept, ws=None):
    dev = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
    return irm.irm_pages_compact(kv, dev(table), dev(base), dev(path), dev(n_accept), workspace=ws)


def moved(rows, table, base, path, n_accept):
    """The rows that compaction leaves, from a copy of what was there."""
    was, flat = rows.clone().reshape(rows.shape[0], -1, 576), rows.clone().reshape(rows.shape[0], -1, 576)
    at = lambda s, t: int(table[s][t // 64]) * 64 + t % 64  # noqa: E731
    for s in range(len(base)):
        for k in range(n_accept[s]):
            flat[:, at(s, base[s] + k)] = was[:, at(s, base[s] + path[s][k])]
    return flat.reshape(rows.shape)


@pytest.mark.parametrize("layers", [1, 3, 4, 9])
def test_compact(layers):
    rng = np.random.default_rng(layers)
    S, P, W = 7, 30, 40
    kv = torch.randn((layers, P, 64, 576), device="cuda").to(torch.bfloat16)
    table = rng.permutation(P)[:S * 4].reshape(S, 4)
    base = [0, 1, 60, 63, 64, 100, 150]  # paths inside a page, over an edge, and from a page's start
    path = np.full((S, W), -1)
    n = [0, 1, 5, 40, 17, 2, 9]
    for s in range(S):
        k = np.sort(rng.choice(np.arange(1, 100), n[s] - 1, replace=False)) if n[s] > 1 else np.zeros(0, int)
        path[s, :n[s]] = np.concatenate([[0], k])[:n[s]]
    path[3, :40] = np.arange(40)  # nothing moves
    path[4, :17] = np.arange(1, 18)  # every row is a source and a destination
    want = moved(kv.cpu(), table, base, path, n)
    ws = compact(kv, table, base, path, n)
    irm.device_status(ws)
    assert torch.equal(kv.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("bad", ["order", "negative", "far", "page", "count", "base"])
def test_compact_refuses_bad_paths(bad):
    """A bad path is recorded and its request left as it was; the others are moved."""
    kv = torch.randn((2, 10, 64, 576), device="cuda").to(torch.bfloat16)
    table, base, n = np.arange(9).reshape(3, 3), [10, 20, 30], [3, 4, 2]
    path = np.array([[0, 2, 5, -1], [1, 3, 60, 70], [4, 5, -1, -1]])
    good = [0, 2]
    if bad == "order":
        path[1, 2] = 3
    elif bad == "negative":
        path[1, 0] = -1
    elif bad == "far":
        path[1, 3] = 172
    elif bad == "page":
        table[1, 1] = 10
    elif bad == "count":
        n[1] = 5
    else:
        base[1] = -1
    want = moved(kv.cpu(), table, [base[s] for s in range(3)], path, [n[s] if s in good else 0 for s in range(3)])
    ws = compact(kv, table, base, path, n)
    with pytest.raises(irm.IrmError) as e:
        irm.device_status(ws)
    assert e.value.status == -7
    assert torch.equal(kv.cpu().view(torch.int16), want.view(torch.int16))


def test_compact_looks_up_no_row_behind_the_table():
    """A path that is long and steps back, of the last request and near its table's end: step 39 is fine
    by itself (0 -> 1, row 190 of 192), while base + 39 would lie behind the table."""
    kv = torch.randn((2, 10, 64, 576), device="cuda").to(torch.bfloat16)
    table, base, n = np.arange(6).reshape(2, 3), [0, 189], [2, 40]
    path = np.full((2, 40), -1)
    path[0, :2] = [0, 5]
    path[1] = [2, 1] * 19 + [0, 1]
    want = moved(kv.cpu(), table, base, path, [2, 0])
    ws = compact(kv, table, base, path, n)
    with pytest.raises(irm.IrmError) as e:
        irm.device_status(ws)
    assert e.value.status == -7
    assert torch.equal(kv.cpu().view(torch.int16), want.view(torch.int16))


# ---------------------------------------------------------------------------------- copies

@pytest.mark.parametrize("n,layers", [(1, 1), (3, 5), (100, 2)])
def test_copy(n, layers):
    rng = np.random.default_rng(n)
    kv = torch.randn((layers, 2 * n + 3, 64, 576), device="cuda").to(torch.bfloat16)
    order = rng.permutation(2 * n + 3)
    src, dst = order[:n], order[n:2 * n]
    src[-1] = src[0]  # one page to two places
    want = kv.cpu().clone()
    want[:, dst] = want[:, src]
    irm.irm_pages_copy(kv, src, dst)
    assert torch.equal(kv.cpu().view(torch.int16), want.view(torch.int16))


def test_copy_more_pairs_than_a_launch_holds():
    n = 4100
    kv = torch.zeros((2 * n, 64, 576), dtype=torch.bfloat16, device="cuda")
    kv[:n] = torch.arange(n, device="cuda").to(torch.bfloat16)[:, None, None]
    order = np.random.default_rng(1).permutation(n)
    irm.irm_pages_copy(kv, order, n + np.arange(n))
    assert torch.equal(kv[n:], kv[torch.from_numpy(order).cuda()])


def test_a_call_on_another_stream_makes_its_workspace_there():
    # zeroed behind the current stream's work, the workspace would lose what the call recorded in it
    c = Cache(2, 4, 8)
    new = torch.tensor([300, 0], dtype=torch.int32, device="cuda")  # 4 pages hold 256 rows
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    ws = irm.irm_pages_resize(new, c.seq, c.table, c.ref, stream=side)
    torch.cuda.synchronize()
    with pytest.raises(irm.IrmError) as e:
        irm.device_status(ws)
    assert e.value.status == CODES["bounds"]


def test_replayed_graph():
    """A captured step (grow, compact, trim) advances the state at each replay."""
    c = Cache(2, 4, 9, layers=1)
    c.resize([70, 10])
    base, keep, grown = c.seq.clone(), torch.zeros_like(c.seq), torch.zeros_like(c.seq)
    path = torch.tensor([[0, 2, 3], [0, 1, -1]], dtype=torch.int32, device="cuda")
    n = torch.tensor([3, 2], dtype=torch.int32, device="cuda")

    def step():
        base.copy_(c.seq)
        torch.add(base, 5, out=grown)
        irm.irm_pages_resize(grown, c.seq, c.table, c.ref, workspace=c.ws)
        irm.irm_pages_compact(c.kv, c.table, base, path, n, workspace=c.ws)
        torch.add(base, n, out=keep)
        irm.irm_pages_resize(keep, c.seq, c.table, c.ref, workspace=c.ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            step()
    torch.cuda.synchronize()
    for _ in range(12):
        seq = c.model.seq[:]
        c.model.resize([x + 5 for x in seq])
        c.rows = moved(c.rows, c.model.table, seq, path.tolist(), n.tolist())
        c.model.resize([seq[0] + 3, seq[1] + 2])
        g.replay()
        torch.cuda.synchronize()
        c.check()
