"""Tree attention over the paged cache against its 64-bit formula.

Tolerances, element by element and before any run: the output is rounded to bf16 (half a step,
2^-8 |O|); the probabilities are rounded to bf16 before the product with the values (2^-8 each,
so at most 2^-8 A with A = sum p |v|); scores are sums of 576 products in fp32, each addition off
by at most 2^-22 of the sum of magnitudes S (tensor-core accumulation may truncate), e = 576 *
2^-22 S, which moves a probability by at most a factor 1 + 2 e; exponentials and the final
division add 2^-20 A.  lse is off by at most e plus 2^-20 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
import spec_reference as ref
import tree_bounds
from helpers import SCALE

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


def make(ctx, nodes, H, seed=0, q_std=1.0 / np.sqrt(192.0), mask="tree", spare=3, words=None, max_pages=None, kv_std=1.0):
    """A batch of trees over scattered pages; rows that nothing reads are NaN."""
    rng = np.random.default_rng(seed)
    B, T = len(ctx), int(np.sum(nodes))
    indptr = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    held = [-(-(c + n) // 64) for c, n in zip(ctx, nodes)]
    n_pages = sum(held) + spare
    order = rng.permutation(n_pages)
    table = np.full((B, max_pages or max(max(held), 1)), -1, np.int32)
    kv = np.full((n_pages, 64, 576), np.nan, np.float32)
    at, seen = 0, []
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
        rows = rng.standard_normal((ctx[b] + nodes[b], 576)).astype(np.float32) * kv_std
        for t in range(0, len(rows), 64):
            kv[table[b, t // 64], :len(rows[t:t + 64])] = rows[t:t + 64]
        n = nodes[b]
        if mask == "tree":
            par = np.array([-1] + [int(rng.integers(0, i)) for i in range(1, n)])
            seen.append(ref.ancestors(par) if n else np.zeros((0, 0), bool))
        elif mask == "chain":
            seen.append(np.tril(np.ones((n, n), bool)))
        elif mask == "none":
            seen.append(np.zeros((n, n), bool))
        else:
            seen.append(rng.random((n, n)) < 0.5)
    W = words or max(1, (max(nodes) + 31) // 32)
    bits = np.concatenate([ref.mask_words(s, W) for s in seen if len(s)] or [np.zeros((0, W), np.int32)])
    f = lambda *shape: torch.from_numpy((rng.standard_normal(shape) * q_std).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    return dict(ctx=np.array(ctx, np.int32), indptr=indptr, H=H, kv=torch.from_numpy(kv).to(torch.bfloat16).cuda(),
                table=torch.from_numpy(table).cuda(), mask=torch.from_numpy(bits.reshape(T, W)).cuda(), seen=seen,
                q_lat=f(T, H, 512), q_rope=f(T, H, 64))


def call(c, scale=SCALE, **kw):
    T, H = c["q_lat"].shape[:2]
    kw.setdefault("lse", torch.full((T, H), 7.0, dtype=torch.float32, device="cuda"))
    kw.setdefault("out", torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device="cuda"))
    return irm.irm_mla_attn_tree(c["q_lat"], c["q_rope"], c["ctx"], c["indptr"], c["kv"], c["table"], c["mask"], scale, **kw)


def request(c, b):
    """Request b's queries, rows and mask in 64 bits."""
    lo, hi = c["indptr"][b], c["indptr"][b + 1]
    rows = int(c["ctx"][b]) + hi - lo
    pages = c["table"][b, :-(-rows // 64)].long()
    kv = c["kv"][pages].reshape(-1, 576)[:rows].double().cpu().numpy()
    q = torch.cat([c["q_lat"][lo:hi], c["q_rope"][lo:hi]], 2).double().cpu().numpy()
    return q, kv


def check(c, out, lse, scale=SCALE, requests=None, heads=None):
    for b in range(len(c["ctx"])) if requests is None else requests:
        lo, hi = c["indptr"][b], c["indptr"][b + 1]
        if lo == hi:
            continue
        q, kv = request(c, b)
        hs = np.arange(c["H"]) if heads is None else np.asarray(heads)
        O, L, A, S = ref.tree_attention(q[:, hs], kv, c["seen"][b], int(c["ctx"][b]), scale)
        o = out[lo:hi].double().cpu().numpy()[:, hs]
        e = 576 * 2.0 ** -22 * S
        tol = STEP * np.abs(O) + (STEP + 2 * e[..., None] + 2.0 ** -20) * A + 1e-30
        assert np.isfinite(o).all(), f"request {b}: non-finite output"
        worst = (np.abs(o - O) / tol).max()
        assert worst <= 1.0, f"request {b}: {worst:.3f} of the tolerance"
        if lse is not None:
            g = lse[lo:hi].double().cpu().numpy()[:, hs]
            none = np.isneginf(L)
            assert np.array_equal(none, np.isneginf(g))
            d = np.abs(g[~none] - L[~none])
            assert (d <= e[~none] + 2.0 ** -20 * (1 + np.abs(L[~none]))).all(), f"request {b}: lse off by {d.max():.3e}"


def run_and_check(c, **kw):
    out, lse, ws = call(c)
    irm.device_status(ws)
    check(c, out, lse, **kw)


@pytest.mark.parametrize("ctx", [0, 1, 2, 31, 63, 64, 65, 127, 128, 200, 577])
@pytest.mark.parametrize("n", [1, 3, 64])
def test_lengths(ctx, n):
    run_and_check(make([ctx], [n], 16, seed=ctx + n))


@pytest.mark.parametrize("H", [1, 2, 3, 7, 8, 16, 24, 40, 64, 100, 127, 128])
def test_head_counts(H):
    run_and_check(make([150, 3], [5, 9], H, seed=H))


@pytest.mark.parametrize("n", [31, 32, 33, 65, 100, 300, 1024])
def test_tree_sizes(n):
    """Trees whose rows run over several pages and mask words."""
    run_and_check(make([70], [n], 3, seed=n), heads=[0, 2] if n > 100 else None)


@pytest.mark.parametrize("mask", ["chain", "random", "none"])
@pytest.mark.parametrize("ctx", [0, 40, 100])
def test_masks(mask, ctx):
    """Any mask: a chain, half of the bits at random (rows without themselves), nothing (with no committed
    rows either, every row is empty: zeros and -inf)."""
    run_and_check(make([ctx, ctx], [20, 37], 8, seed=ctx, mask=mask))


def test_mask_bits_beyond_the_tree_are_ignored():
    c = make([90, 10], [7, 30], 16, seed=2, words=3)
    out, lse, _ = call(c)
    c["mask"] = c["mask"].clone()
    c["mask"][:7, 0] |= -1 << 7
    c["mask"][7:, 0] |= -1 << 30
    c["mask"][:, 1:] = -1
    again, lse2, ws = call(c)
    irm.device_status(ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_ragged_batch_with_empty_trees():
    run_and_check(make([300, 0, 1000, 5, 64, 77], [4, 0, 1, 33, 12, 0], 16, seed=5))


def test_many_requests():
    """More requests than one launch's parameters carry."""
    rng = np.random.default_rng(8)
    ctx, n = rng.integers(0, 90, 1500).tolist(), rng.integers(0, 4, 1500).tolist()
    c = make(ctx, n, 2, seed=8)
    out, lse, ws = call(c)
    irm.device_status(ws)
    check(c, out, lse, requests=list(range(0, 1500, 37)) + [1022, 1023, 1024, 1025, 1499])


def test_split_contexts():
    """Contexts long enough to be shared by many clusters, beside a short one."""
    c = make([9000, 20, 4100], [3, 5, 17], 16, seed=9)
    out, lse, ws = call(c)
    irm.device_status(ws)
    check(c, out, lse, heads=[0, 7, 15])


def test_long_context_many_heads():
    c = make([20000], [9], 128, seed=10)
    out, lse, ws = call(c)
    irm.device_status(ws)
    check(c, out, lse, heads=[0, 64, 127])


@pytest.mark.parametrize("nodes", [1, 5])
def test_many_pieces(nodes):
    """One long context on the whole GPU: dozens of pieces of one row tile, each with a maximum of its own."""
    c = make([50000], [nodes], 2, seed=25, q_std=0.6)
    out, lse, ws = call(c)
    irm.device_status(ws)
    check(c, out, lse)


@pytest.mark.parametrize("q_std", [0.0, 1.0, 6.0])
def test_score_sizes(q_std):
    """Flat scores, and scores in the tens, where one row takes nearly all and the running maximum moves."""
    run_and_check(make([700, 130], [11, 2], 16, seed=11, q_std=q_std))


def test_growing_scores():
    """Every page's scores are far above those before: the running maximum moves at each page."""
    c = make([640], [4], 16, seed=12, q_std=0.2)
    kv = c["kv"].float()
    for i, p in enumerate(c["table"][0].tolist()):
        kv[p] *= 1.0 + 2.5 * i
    c["kv"] = kv.to(torch.bfloat16)
    run_and_check(c)


def test_masked_values_may_be_anything():
    """Rows behind the last draft (already NaN in every case here), and drafts that no node sees."""
    c = make([100], [12], 16, seed=13)
    seen = c["seen"][0].copy()
    seen[:, [4, 9]] = False
    c["seen"] = [seen]
    c["mask"] = torch.from_numpy(ref.mask_words(seen)).cuda()
    rows = c["kv"][c["table"][0].long()].reshape(-1, 576)
    rows[104], rows[109] = float("nan"), float("inf")
    c["kv"][c["table"][0].long()] = rows.reshape(-1, 64, 576)
    out, lse, ws = call(c)
    irm.device_status(ws)
    rows[104], rows[109] = 0.0, 0.0
    c["kv"][c["table"][0].long()] = rows.reshape(-1, 64, 576)
    check(c, out, lse)


@pytest.mark.parametrize("scale", [1e-3, 1.0])
def test_scale(scale):
    c = make([200], [5], 16, seed=14)
    out, lse, _ = call(c, scale)
    check(c, out, lse, scale)


def test_requests_may_share_pages():
    """A prefix's pages in two requests' tables, their drafts in pages of their own."""
    c = make([128, 128], [6, 6], 16, seed=15)
    c["table"][1, :2] = c["table"][0, :2]
    run_and_check(c)


def test_wider_page_table_and_no_lse():
    c = make([100, 30], [3, 4], 16, seed=16, max_pages=9)
    out, lse, ws = irm.irm_mla_attn_tree(c["q_lat"], c["q_rope"], c["ctx"], c["indptr"], c["kv"], c["table"], c["mask"], SCALE)
    irm.device_status(ws)
    assert lse is None
    check(c, out, None)


def test_bad_pages_are_recorded_not_read():
    c = make([200, 100], [3, 4], 16, seed=17)
    good, _, _ = call(c)
    for bad in (-1, c["kv"].shape[0], 2 ** 31 - 1, -2 ** 31):
        c["table"][0, 1] = bad
        out, lse, ws = call(c)
        with pytest.raises(irm.IrmError) as e:
            irm.device_status(ws)
        assert e.value.status == -7
        irm.device_status(ws)  # cleared
        assert torch.equal(out[3:], good[3:])  # the other request is whole


def test_nothing_outside_is_written():
    c = make([70, 200], [3, 2], 24, seed=18)
    big = torch.full((9, 24, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, 24), 5.0, dtype=torch.float32, device="cuda")
    kv = c["kv"].clone()
    call(c, out=big[2:7], lse=lse[2:7])
    torch.cuda.synchronize()
    assert (big[:2] == 5).all() and (big[7:] == 5).all() and (lse[:2] == 5).all() and (lse[7:] == 5).all()
    assert torch.equal(kv.view(torch.int16), c["kv"].view(torch.int16))
    check(c, big[2:7], lse[2:7])


def test_same_call_gives_the_same_bits():
    c = make([5000, 100, 900], [7, 30, 2], 32, seed=19)
    ws = irm.new_workspace(irm.tree_workspace_size(c["ctx"], c["indptr"], 32))
    a, la, _ = call(c, workspace=ws)
    for _ in range(3):
        b, lb, _ = call(c, workspace=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_one_workspace_for_calls_of_different_sizes():
    big, small = make([6000, 3000], [9, 9], 64, seed=20), make([40], [2], 16, seed=21)
    ws = irm.new_workspace(irm.tree_workspace_size(big["ctx"], big["indptr"], 64))
    for c in (big, small, big, small):
        out, lse, _ = call(c, workspace=ws)
        irm.device_status(ws)
        check(c, out, lse, heads=[0, 15])


def test_workspace_is_checked():
    c = make([9000, 4000], [3, 2], 16, seed=26)
    need = irm.tree_workspace_size(c["ctx"], c["indptr"], 16)
    assert need > 256  # the contexts are cut
    ws = irm.new_workspace(need)
    with pytest.raises(irm.IrmError) as e:
        call(c, workspace=ws[:need - 256])
    assert e.value.status == -8
    out, lse, _ = call(c, workspace=ws)
    irm.device_status(ws)
    check(c, out, lse, heads=[0, 15])


def test_two_streams_and_a_replayed_graph():
    a, b = make([3000, 50], [6, 5], 16, seed=22), make([700], [40], 128, seed=23)
    ref_a, ref_b = call(a)[0], call(b)[0]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        outs.append((call(a, stream=sa)[0], call(b, stream=sb)[0]))
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, ref_a) and torch.equal(y, ref_b)
    g = torch.cuda.CUDAGraph()
    ws = irm.new_workspace(irm.tree_workspace_size(a["ctx"], a["indptr"], 16))
    out = torch.zeros_like(ref_a)
    lse = torch.zeros(out.shape[:2], dtype=torch.float32, device="cuda")
    call(a, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(a, out=out, lse=lse, workspace=ws)
    a["ctx"][:] = 1  # the graph keeps the lengths it was captured with
    a["q_lat"].mul_(2.0)
    a["q_rope"].mul_(2.0)
    g.replay()
    a["ctx"][:] = [3000, 50]
    irm.device_status(ws)
    check(a, out, lse)


@pytest.mark.parametrize("ctx,nodes,H,q_std", [([4000, 4100, 900], [2, 1, 9], 128, 0.07), ([30000], [3], 16, 0.6), ([700] * 20, [13] * 20, 24, 0.3)])
def test_repeats_beside_other_work(ctx, nodes, H, q_std):
    """Hand-overs between the two halves of a pair, with their timing disturbed: the same bits each time."""
    c = make(ctx, nodes, H, seed=27, q_std=q_std)
    ws = irm.new_workspace(irm.tree_workspace_size(c["ctx"], c["indptr"], H))
    out, lse, _ = call(c, workspace=ws)
    check(c, out, lse, heads=[0, H - 1])
    side, junk = torch.cuda.Stream(), torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    for k in range(60):
        if k % 2:
            with torch.cuda.stream(side):
                junk.add_(1)
        again, lse2, _ = call(c, workspace=ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2), k
    irm.device_status(ws)
    torch.cuda.synchronize()


# ------------------------------------------------------------- values that are not finite

def lengths(cut):
    """A request that is cut into pieces or not, and a short one beside it."""
    return ([9000, 70], [3, 4]) if cut else ([150, 70], [3, 4])


def set_row(c, b, t, col, value):
    """Entry `col` of row t of request b's cache."""
    c["kv"][int(c["table"][b, t // 64]), t % 64, col] = value


def both(c):
    out, lse, ws = call(c)
    irm.device_status(ws)
    return out.clone(), lse.clone()


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("col", [3, 300, 530, 575])
@pytest.mark.parametrize("t", [0, 100, 149])
def test_a_nan_key_reaches_every_row_that_sees_it(cut, col, t):
    """One NaN entry of a committed row: its score is NaN, and so are the sums that it enters."""
    ctx, nodes = lengths(cut)
    c = make(ctx, nodes, 16, seed=30)
    assert (irm.tree_workspace_size(c["ctx"], c["indptr"], 16) > 256) == cut
    clean, clean_lse = both(c)
    set_row(c, 0, t, col, float("nan"))
    out, lse = both(c)
    assert torch.isnan(out[:3]).all() and torch.isnan(lse[:3]).all()
    assert torch.equal(out[3:], clean[3:]) and torch.equal(lse[3:], clean_lse[3:])


@pytest.mark.parametrize("ctx", [0, 64, 9000])
def test_a_nan_draft_reaches_the_nodes_that_see_it(ctx):
    """Others may get NaN in O (0 times NaN), and have the sum of what they see in lse."""
    c = make([ctx], [12], 16, seed=31)
    sees = c["seen"][0][:, 5]
    assert sees.any() and not sees.all()
    set_row(c, 0, ctx + 5, 17, float("nan"))
    out, lse = both(c)
    q, kv = request(c, 0)
    kv[ctx + 5] = 0.0
    _, L, _, S = ref.tree_attention(q, kv, c["seen"][0], ctx, SCALE)
    lse, out = lse.double().cpu().numpy(), out.float().cpu().numpy()
    assert np.isnan(lse[sees]).all() and np.isnan(out[sees]).all()
    d = np.abs(lse[~sees] - L[~sees])
    assert (d <= 576 * 2.0 ** -22 * S[~sees] + 2.0 ** -20 * (1 + np.abs(L[~sees]))).all()


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("part", ["q_lat", "q_rope"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_is_its_own_rows_alone(cut, part, value):
    """Among many keys some score is infinite or NaN: no weights are defined, and NaN comes out."""
    ctx, nodes = lengths(cut)
    c = make(ctx, nodes, 16, seed=32)
    clean, clean_lse = both(c)
    c[part][1, 6, 40] = value
    c[part][4, 0, 2] = value
    out, lse = both(c)
    hit = torch.zeros((7, 16), dtype=torch.bool, device="cuda")
    hit[1, 6], hit[4, 0] = True, True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


@pytest.mark.parametrize("ctx", [40, 9000])
def test_an_infinite_key(ctx):
    """k_r alone infinite: a score of -inf weighs nothing, one of +inf (or 0 times infinity) gives NaN."""
    c = make([ctx], [3], 16, seed=33)
    set_row(c, 0, 20, 540, float("inf"))
    q = c["q_rope"][:, :, 540 - 512].double().cpu().numpy()
    out, lse = both(c)
    low = q < 0
    assert low.any() and not low.all()
    g = lse.double().cpu().numpy()
    assert np.isnan(g[~low]).all() and np.isnan(out.float().cpu().numpy()[~low]).all()
    qq, kv = request(c, 0)
    kv[20, 540] = 0.0
    seen = np.delete(kv, 20, 0)  # the definition without that row
    O, L, A, S = ref.tree_attention(qq, seen, c["seen"][0], ctx - 1, SCALE)
    e = 576 * 2.0 ** -22 * S
    o = out.double().cpu().numpy()
    tol = STEP * np.abs(O) + (STEP + 2 * e[..., None] + 2.0 ** -20) * A + 1e-30
    assert (np.abs(o - O) <= tol)[low].all()
    assert (np.abs(g - L) <= e + 2.0 ** -20 * (1 + np.abs(L)))[low].all()


def test_a_row_whose_every_score_is_minus_infinity():
    """counts as one that sees nothing."""
    c = make([1, 5], [1, 2], 2, seed=34, mask="none")
    c["q_rope"][0, :, 0] = torch.tensor([-1.0, 1.0], device="cuda").to(torch.bfloat16)
    set_row(c, 0, 0, 512, float("inf"))
    out, lse = both(c)
    assert (out[0, 0] == 0).all() and lse[0, 0] == -float("inf")
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    check(c, out, lse, requests=[1])


@pytest.mark.parametrize("power", [20, 28, 40, 60])
@pytest.mark.parametrize("cut", [False, True])
def test_scores_of_great_size(power, cut):
    """Up to 2^30 the sums keep their meaning (lse to the error of a score); beyond, NaN may come out, and
    never the answer of a row that sees nothing."""
    ctx, nodes = lengths(cut)
    c = make(ctx, nodes, 16, seed=35, q_std=2.0 ** (power / 2), kv_std=2.0 ** (power / 2 - 4))
    out, lse = both(c)
    assert not torch.isinf(lse).any()
    for b in range(2):
        lo, hi = c["indptr"][b], c["indptr"][b + 1]
        q, kv = request(c, b)
        _, L, _, S = ref.tree_attention(q, kv, c["seen"][b], int(c["ctx"][b]), SCALE)
        g = lse[lo:hi].double().cpu().numpy()
        fine = np.abs(g - L) <= 576 * 2.0 ** -22 * S + 2.0 ** -20 * (1 + np.abs(L))
        if np.abs(S).max() * 1.4427 < 2.0 ** 30:
            assert fine.all() and torch.isfinite(out[lo:hi]).all()
        assert (fine | np.isnan(g)).all()
        some = (out[lo:hi].float().abs().amax(2) > 0) | torch.isnan(out[lo:hi]).any(2)
        assert some.all()


# ------------------------------------------------------------- every key of a long context

def pages_apart(c):
    """The values of each page of a request in a column of their own (page index mod 512): O holds the pages'
    weights, each to the rounding of its own size."""
    for b in range(len(c["ctx"])):
        rows = int(c["ctx"][b]) + int(c["indptr"][b + 1] - c["indptr"][b])
        for i, t in enumerate(range(0, rows, 64)):
            page = c["kv"][int(c["table"][b, i]), :rows - t]
            page[:, :512] = 0.0
            page[:, i % 512] = 1.0
    return c


LONG = [([200], [3], 16), ([50000], [1], 2), ([50000], [5], 2), ([20000], [9], 128), ([9000, 20, 4100], [3, 5, 17], 16), ([4095] * 3, [1] * 3, 16)]


@pytest.mark.parametrize("ctx,nodes,H", LONG)
def test_each_page_has_its_weight(ctx, nodes, H):
    run_and_check(pages_apart(make(ctx, nodes, H, seed=40)), heads=sorted({0, H // 2, H - 1}))


@pytest.mark.parametrize("ctx,nodes,H", LONG)
@pytest.mark.parametrize("q_std", [1.0 / np.sqrt(192.0), 1.0])
def test_rows_as_a_whole(ctx, nodes, H, q_std):
    """Each row's error against a bound that shrinks with the row, so that no page can be missed."""
    c = make(ctx, nodes, H, seed=41, q_std=q_std)
    out, lse, ws = call(c)
    irm.device_status(ws)
    hs = sorted({0, H // 2, H - 1})
    check(c, out, lse, heads=hs)
    for b in range(len(ctx)):
        q, kv = request(c, b)
        o = out[c["indptr"][b]:c["indptr"][b + 1]].double().cpu().numpy()
        assert tree_bounds.row_errors(o[:, hs], q[:, hs], kv, c["seen"][b], ctx[b], SCALE).max() <= 1.0


def test_cut_contexts_in_later_launches():
    """A launch takes 256 requests: long contexts at the edges and in the middle of the second and third, where
    the partials' buffer is used anew and the first node is not 0."""
    rng = np.random.default_rng(42)
    ctx, n = rng.integers(0, 90, 600), rng.integers(0, 4, 600)
    for b, rows in ((10, 6000), (255, 500), (256, 7000), (300, 9000), (511, 700), (512, 12000), (599, 5000)):
        ctx[b], n[b] = rows, 2
    n[[0, 254, 257, 510, 513, 598]] = 1, 3, 1, 2, 3, 1
    c = pages_apart(make(ctx.tolist(), n.tolist(), 16, seed=42))
    for lo in (0, 256, 512):  # each launch has a cut context
        hi = min(lo + 256, 600)
        assert irm.tree_workspace_size(c["ctx"][lo:hi], c["indptr"][lo:hi + 1] - c["indptr"][lo], 16) > 256
    out, lse, ws = call(c)
    irm.device_status(ws)
    check(c, out, lse, requests=sorted({0, 10, 254, 255, 256, 257, 300, 510, 511, 512, 513, 598, 599} | set(range(3, 600, 41))))
