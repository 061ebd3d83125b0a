"""Tree attention over the 8-bit cache: the 64-bit formula on the rows that the codes stand for (exact in bf16), with
the tolerances of the bf16 cache's tests."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
import row8_reference as ref8
import tree_bounds
from helpers import SCALE
from test_gpu_tree import call, check, make, request

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


def eight(c, scale_exponents=None):
    """The batch over an 8-bit cache, and the same with the bf16 rows that it stands for.  NaN rows become NaN scales."""
    kv = c["kv"]
    n = kv.shape[0] * 64
    g = kv.reshape(n, 576)[:, :512].float().reshape(n, 4, 128)
    bad = ~torch.isfinite(g).all(2)
    g = torch.where(bad[..., None], 0.0, g)
    most = g.abs().amax(2)
    e = torch.ceil(torch.log2(torch.clamp(most, min=1e-30) / 448.0)).clamp(-126, 7)
    s = torch.where(most > 0, torch.exp2(e), 1.0)
    if scale_exponents is not None:
        s = torch.exp2(scale_exponents.to(s.device))
    codes = (g / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    value = (codes.float() * s[..., None]).reshape(n, 512)
    value = torch.where(bad.repeat_interleave(128, 1), float("nan"), value)
    assert torch.equal(value.to(torch.bfloat16).float().nan_to_num(9.0), value.nan_to_num(9.0))  # exact in bf16
    s = torch.where(bad, float("nan"), s)
    raw = torch.empty((n, 656), dtype=torch.uint8, device=kv.device)
    raw[:, :512] = codes.reshape(n, 512).view(torch.uint8)
    raw[:, 512:528] = s.view(torch.uint8)
    raw[:, 528:] = kv.reshape(n, 576)[:, 512:].contiguous().view(torch.uint8)
    wide = torch.cat([value.to(torch.bfloat16), kv.reshape(n, 576)[:, 512:]], 1).reshape(kv.shape)
    return dict(c, kv=raw.reshape(kv.shape[0], 64, 656)), dict(c, kv=wide)


def run_and_check(c, scale=SCALE, **kw):
    c8, c16 = eight(c)
    out, lse, ws = call(c8, scale)
    irm.device_status(ws)
    check(c16, out, lse, scale, **kw)
    return out, lse, c16


@pytest.mark.parametrize("ctx", [0, 1, 2, 31, 63, 64, 65, 127, 128, 191, 192, 193, 256, 257, 577])
@pytest.mark.parametrize("n", [1, 3, 64])
def test_lengths(ctx, n):
    run_and_check(make([ctx], [n], 16, seed=ctx + n))


@pytest.mark.parametrize("H", [1, 2, 3, 7, 16, 24, 40, 64, 100, 127, 128])
def test_head_counts(H):
    run_and_check(make([150, 3], [5, 9], H, seed=H))


@pytest.mark.parametrize("n", [31, 33, 65, 300, 1024])
def test_tree_sizes(n):
    run_and_check(make([70], [n], 3, seed=n), heads=[0, 2] if n > 100 else None)


@pytest.mark.parametrize("mask", ["chain", "random", "none"])
@pytest.mark.parametrize("ctx", [0, 40, 100])
def test_masks(mask, ctx):
    run_and_check(make([ctx, ctx], [40, 7], 5, seed=ctx, mask=mask))


@pytest.mark.parametrize("B", [5, 80, 257, 300])
def test_batches(B):
    rng = np.random.default_rng(B)
    ctx, n = rng.integers(0, 200, B).tolist(), rng.integers(0, 4, B).tolist()
    n[-1] = 2
    run_and_check(make(ctx, n, 4, seed=B))


@pytest.mark.parametrize("ctx,n,H", [(20000, 1, 16), (9000, 3, 128), (70000, 2, 5)])
def test_long_contexts_are_cut_and_merged(ctx, n, H):
    c = make([ctx], [n], H, seed=H, q_std=0.03)
    run_and_check(c, heads=[0, H - 1])


def test_rows_shrink_with_their_bound():
    """Norms of whole rows against the bound that shrinks as keys share the weight."""
    c = make([3000, 700], [3, 5], 16, seed=1)
    c8, c16 = eight(c)
    out, _, ws = call(c8)
    irm.device_status(ws)
    for b in range(2):
        lo, hi = c["indptr"][b], c["indptr"][b + 1]
        q, rows = request(c16, b)
        part = tree_bounds.row_errors(out[lo:hi].double().cpu().numpy(), q, rows, c["seen"][b], int(c["ctx"][b]), SCALE)
        assert part.max() <= 1.0


@pytest.mark.parametrize("B,H,ctx,n", [(64, 128, 4096, 2), (152, 16, 3000, 1)])
def test_a_full_gpu_repeats_and_agrees_with_the_bf16_cache(B, H, ctx, n):
    """Every SM busy at once, many pages in turn: runs are equal bit for bit, and each row is the bf16 cache's up to the
    roundings that both make (the output's, 2^-8, once each; the scores' and probabilities' as in
    tree_bounds, where a row's spread over ctx independent keys is below an eighth of its norm's bound)."""
    g = torch.Generator(device="cuda").manual_seed(7)
    pages = B * (-(-(ctx + n) // 64))
    c = torch.randn((pages * 64, 4, 128), generator=g, device="cuda")
    s = torch.exp2(torch.ceil(torch.log2(c.abs().amax(2) / 448.0)))
    codes = (c / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    k_r = torch.randn((pages * 64, 64), generator=g, device="cuda").to(torch.bfloat16)
    raw = torch.cat([codes.reshape(-1, 512).view(torch.uint8), s.view(torch.uint8), k_r.view(torch.uint8)], 1).reshape(pages, 64, 656)
    wide = torch.cat([(codes.float() * s[..., None]).reshape(-1, 512).to(torch.bfloat16), k_r], 1).reshape(pages, 64, 576)
    table = torch.randperm(pages, generator=g, device="cuda").int().reshape(B, -1).contiguous()
    ql, qr = (torch.randn((B * n, H, w), generator=g, device="cuda").div(13.9).to(torch.bfloat16) for w in (512, 64))
    mask = torch.tensor([(1 << (i + 1)) - 1 for i in range(n)] * B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    args = (np.full(B, ctx), np.arange(B + 1) * n)
    ws = irm.new_workspace(irm.tree_workspace_size(*args, H))
    runs = []
    for _ in range(4):
        lse = torch.empty((B * n, H), device="cuda")
        out, _, _ = irm.irm_mla_attn_tree(ql, qr, *args, raw, table, mask, SCALE, lse=lse, workspace=ws)
        runs.append((out, lse))
    lse = torch.empty((B * n, H), device="cuda")
    want, _, _ = irm.irm_mla_attn_tree(ql, qr, *args, wide, table, mask, SCALE, lse=lse, workspace=ws)
    irm.device_status(ws)
    for o, l in runs:
        assert torch.equal(o, runs[0][0]) and torch.equal(l, runs[0][1])
    d = (runs[0][0].double() - want.double()).norm(dim=2) / want.double().norm(dim=2)
    assert float(d.max()) <= 2 * 2.0 ** -8
    assert float((runs[0][1] - lse).abs().max()) <= 2 * (576 * 2.0 ** -22 * 4 + 2.0 ** -16)


def test_every_code_and_scale():
    """Each of the codes reaches the output as its value: one row seen by itself has weight 1, so O is the row (exact
    in bf16); scales over their whole range."""
    n = 1024
    c = make([0], [n], 1, seed=0, mask="none", kv_std=0.0)
    W = c["mask"].shape[1]
    seen = np.eye(n, dtype=bool)
    bits = np.packbits(seen, axis=1, bitorder="little").view(np.int32).reshape(n, W)
    c["mask"], c["seen"] = torch.from_numpy(bits).cuda(), [seen]
    pages = c["table"][0, :n // 64].long()
    rng = np.random.default_rng(2)
    raw = np.zeros((n, 656), np.uint8)
    finite = np.array([x for x in range(256) if x & 127 != 127], np.uint8)
    raw[:, :512] = rng.choice(finite, (n, 512))
    raw[:, :254] = finite
    scale = 2.0 ** rng.integers(-100, 8, (n, 4)).astype(np.float32)
    scale[0], scale[1] = [2.0 ** -117] * 4, [128.0] * 4
    raw[:, 512:528] = scale.astype(np.float32).view(np.uint8)
    kv = torch.zeros((c["kv"].shape[0], 64, 656), dtype=torch.uint8, device="cuda")
    kv[pages] = torch.from_numpy(raw).cuda().reshape(-1, 64, 656)
    zero = torch.zeros_like  # zero queries: every score is 0, whatever the rows hold
    out, lse, ws = call(dict(c, kv=kv, q_lat=zero(c["q_lat"]), q_rope=zero(c["q_rope"])))
    irm.device_status(ws)
    assert np.array_equal(out[:, 0].double().cpu().numpy(), ref8.decode(raw)[:, :512])
    assert (lse == 0).all()


def test_scales_that_are_no_powers_of_two():
    """The upper 16 bits count, the product is rounded to bf16."""
    n = 64
    c = make([0], [n], 1, seed=0, mask="none", kv_std=0.0)
    seen = np.eye(n, dtype=bool)
    c["mask"] = torch.from_numpy(np.packbits(seen, axis=1, bitorder="little").view(np.int32).reshape(n, -1)).cuda()
    rng = np.random.default_rng(2)
    raw = np.zeros((n, 656), np.uint8)
    raw[:, :512] = rng.choice(np.array([x for x in range(256) if x & 127 != 127], np.uint8), (n, 512))
    scale = rng.uniform(0.01, 200.0, (n, 4)).astype(np.float32)
    raw[:, 512:528] = scale.view(np.uint8)
    kv = torch.zeros((c["kv"].shape[0], 64, 656), dtype=torch.uint8, device="cuda")
    kv[c["table"][0, 0].item()] = torch.from_numpy(raw).cuda()
    out, _, ws = call(dict(c, kv=kv, q_lat=torch.zeros_like(c["q_lat"]), q_rope=torch.zeros_like(c["q_rope"])))
    irm.device_status(ws)
    cut = (scale.view(np.uint32) & 0xffff0000).view(np.float32)
    want = torch.from_numpy((ref8.E4M3[raw[:, :512]] * np.repeat(cut.astype(np.float64), 128, 1)).astype(np.float32)).to(torch.bfloat16)
    assert torch.equal(out[:, 0].cpu(), want)


def test_nan_scale_reaches_who_sees_it():
    c8, c16 = eight(make([100], [2], 4, seed=5))
    page = int(c8["table"][0, 0])
    c8["kv"][page, 7, 512:516] = torch.tensor([0, 0, 0xc0, 0x7f], dtype=torch.uint8)
    out, lse, ws = call(c8)
    irm.device_status(ws)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_bad_page_is_recorded_and_reads_as_zeros():
    c8, c16 = eight(make([200, 90], [2, 3], 6, seed=7))
    for bad in (c8["kv"].shape[0], -1, 2**31 - 1):
        table = c8["table"].clone()
        table[0, 1] = bad
        out, lse, ws = call(dict(c8, table=table))
        with pytest.raises(irm.IrmError) as e:
            irm.device_status(ws)
        assert e.value.status == -7
        kv = torch.cat([c16["kv"], torch.zeros_like(c16["kv"][:1])])
        table[0, 1] = kv.shape[0] - 1
        check(dict(c16, kv=kv, table=table), out, lse)


def test_other_stream_workspace_and_graph():
    c8, c16 = eight(make([700, 5000], [3, 2], 16, seed=4))
    want, wlse, _ = call(c8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, lse, ws = call(c8, stream=s, out=None)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    ws = irm.new_workspace(irm.tree_workspace_size(c8["ctx"], c8["indptr"], 16))
    o, l = torch.zeros_like(want), torch.zeros_like(wlse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c8, out=o, lse=l, workspace=ws)
    for _ in range(3):
        o.zero_(), l.zero_()
        g.replay()
        assert torch.equal(o, want) and torch.equal(l, wlse)
    irm.device_status(ws)


def test_repeats_are_equal():
    c8, _ = eight(make([3000], [7], 100, seed=6))
    a = call(c8)
    for _ in range(5):
        b = call(c8)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
