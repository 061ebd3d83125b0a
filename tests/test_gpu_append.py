"""Rows appended to the paged cache and rotated queries, against plain models.

Tolerances, before any run: a rotated entry is rounded to bf16 (2^-8 of itself); the angle is an fp32
number in [-pi, pi] (off by at most 2^-23) whose sine and cosine come from the fast functions (absolute
error 2^-21.4 there), so with the products' roundings it is off by at most 2^-20 times |x| + |y|, times the
factor.  cKV bytes, codes and scales are exact."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
import row8_reference as ref
from helpers import rope_tables

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def near(got, x, position, **kw):
    """Rotated entries within their bound."""
    want = ref.rotate(x, position, **kw)
    mag = np.abs(x)
    u, v = (slice(0, None, 2), slice(1, None, 2)) if kw.get("interleaved") else (slice(0, 32), slice(32, 64))
    both = np.empty_like(want)
    both[..., u] = both[..., v] = mag[..., u] + mag[..., v]
    tol = STEP * np.abs(want) + 2.0 ** -20 * abs(kw.get("factor", 1.0)) * both + 1e-38
    assert np.isfinite(got).all()
    worst = (np.abs(got - want) / tol).max() if got.size else 0.0
    assert worst <= 1.0, f"{worst:.3f} of the tolerance"


def setup(T, slots, bits, seed=0, longest=300, spare=4, layout="projection"):
    """Tokens of random requests behind random lengths, over scattered pages filled with a pattern."""
    rng = np.random.default_rng(seed)
    request = np.sort(rng.integers(0, slots, T))
    base = rng.integers(0, longest, slots)
    row = base[request] + np.arange(T) - np.searchsorted(request, request)
    mix = rng.permutation(T)
    request, row = request[mix], row[mix]
    wide = (longest + T) // 64 + 1
    need = np.zeros((slots, wide), bool)
    need[request, row // 64] = True
    order = rng.permutation(int(need.sum()) + spare)
    table = np.full((slots, wide), -1, np.int32)
    table[need] = order[:int(need.sum())]
    n_pages = int(need.sum()) + spare
    kv = torch.full((n_pages, 64, 656), 0x55, dtype=torch.uint8) if bits == 8 else torch.full((n_pages, 64, 576), 7.0, dtype=torch.bfloat16)
    x = torch.from_numpy(rng.standard_normal((T, 576)).astype(np.float32)).to(torch.bfloat16).cuda()
    if layout == "projection":
        c, k = x[:, :512], x[:, 512:]
    elif layout == "apart":
        c, k = x[:, :512].contiguous(), x[:, 512:].contiguous()
    else:  # wider rows of each
        w = torch.zeros((T, 1024), dtype=torch.bfloat16, device="cuda")
        w[:, 8:520], w[:, 600:664] = x[:, :512], x[:, 512:]
        c, k = w[:, 8:520], w[:, 600:664]
    return dict(c=c, k=k, kv=kv.cuda(), table=i32(table), row=i32(row), request=i32(request), n_pages=n_pages,
                np_row=row, np_request=request, np_table=table)


def check(d, position=None, skip=None, encoded=False, **kw):
    """The written rows, and every other byte as it was."""
    kv, T = d["kv"].cpu(), len(d["np_row"])
    keep = np.ones(T, bool) if skip is None else ~skip
    page = d["np_table"][d["np_request"], d["np_row"] // 64]
    at = page * 64 + d["np_row"] % 64
    c, k = d["c"].double().cpu().numpy(), d["k"].double().cpu().numpy()
    pos = d["np_row"] if position is None else position
    if kv.dtype == torch.uint8:
        flat = kv.numpy().reshape(-1, 656)
        codes, scales = ref.encode(c[keep])
        assert np.array_equal(flat[at[keep], :512], codes)
        got = np.ascontiguousarray(flat[at[keep], 512:528]).view(np.float32)
        assert np.array_equal(got.astype(np.float64), scales, equal_nan=True)
        k_r = ref.decode(flat[at[keep]])[:, 512:]
        rest = np.delete(flat, at[keep], 0)
        assert (rest == 0x55).all()
    else:
        flat = kv.reshape(-1, 576)
        assert torch.equal(flat[at[keep], :512].view(torch.int16), d["c"].cpu()[keep].view(torch.int16))
        k_r = flat[at[keep], 512:].double().numpy()
        rest = np.delete(flat.float().numpy(), at[keep], 0)
        assert (rest == 7.0).all()
    if encoded:
        assert np.array_equal(k_r, k[keep])
    else:
        near(k_r, k[keep], np.asarray(pos)[keep], **kw)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("T,slots", [(1, 1), (7, 3), (8, 8), (9, 1), (64, 64), (513, 5), (2000, 40)])
def test_rows(bits, T, slots):
    d = setup(T, slots, bits, seed=T)
    ws = irm.irm_pages_append(d["c"], d["k"], d["kv"], d["table"], d["row"], d["request"])
    irm.device_status(ws)
    check(d)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("layout", ["apart", "wide"])
def test_input_strides(bits, layout):
    d = setup(37, 4, bits, seed=3, layout=layout)
    irm.device_status(irm.irm_pages_append(d["c"], d["k"], d["kv"], d["table"], d["row"], d["request"]))
    check(d)


@pytest.mark.parametrize("table", ["base10k", "base500k", "yarn"])
@pytest.mark.parametrize("pairing", [irm.ROPE_NEOX, irm.ROPE_INTERLEAVED])
@pytest.mark.parametrize("factor", [1.0, 1.2772588])
def test_variants_and_far_positions(table, pairing, factor):
    freq = rope_tables()[table]
    rope = irm.Rope.make(freq, pairing)
    for bits in (8, 16):
        d = setup(130, 7, bits, seed=11)
        pos = np.random.default_rng(5).integers(-2**31, 2**31, 130)
        pos[:6] = [0, 1, -1, 2**31 - 1, -2**31, 131072]
        ws = irm.irm_pages_append(d["c"], d["k"], d["kv"], d["table"], d["row"], d["request"], i32(pos), rope, factor)
        irm.device_status(ws)
        near_kw = dict(inv_freq=freq, interleaved=pairing == irm.ROPE_INTERLEAVED, factor=np.float64(np.float32(factor)))
        # 64-bit angles of the reference are good to |p| theta 2^-53 < 2^-22 here
        check(d, position=pos, **near_kw)


@pytest.mark.parametrize("bits", [8, 16])
def test_no_requests_given_and_padding(bits):
    """Token t belongs to request t; negative rows are left out."""
    d = setup(50, 50, bits, seed=2)
    # one token a slot: requests 0 .. 49 in order
    order = np.arange(50)
    base = np.random.default_rng(1).integers(0, 300, 50)
    table = np.full((50, 6), -1, np.int32)
    pages = np.random.default_rng(3).permutation(50)
    table[order, base // 64] = pages
    d.update(np_request=order, np_row=base, np_table=table, table=i32(table), n_pages=50,
             kv=(torch.full((50, 64, 656), 0x55, dtype=torch.uint8) if bits == 8 else torch.full((50, 64, 576), 7.0, dtype=torch.bfloat16)).cuda())
    skip = np.random.default_rng(4).random(50) < 0.3
    irm.device_status(irm.irm_pages_append(d["c"], d["k"], d["kv"], d["table"], i32(np.where(skip, -1, base))))
    check(d, skip=skip)


@pytest.mark.parametrize("bits", [8, 16])
def test_encoded_rows_are_copied(bits):
    d = setup(20, 3, bits, seed=8)
    irm.device_status(irm.irm_pages_append(d["c"], d["k"], d["kv"], d["table"], d["row"], d["request"], encoded=True))
    check(d, encoded=True)


def test_no_tokens():
    d = setup(4, 2, 8)
    before = d["kv"].clone()
    irm.irm_pages_append(d["c"][:0], d["k"][:0], d["kv"], d["table"], d["row"][:0], d["request"][:0])
    assert torch.equal(before, d["kv"])


def values(case, rng):
    """Groups of 128 columns whose largest value sits where the exponent changes, denormals, zeros, huge values."""
    c = rng.standard_normal((8, 512))
    if case == "borders":
        for i, m in enumerate([448.0, 450.0, 224.0, 446.0, 1.75, 1.7578125, 3.5, 3.515625]):
            c[i] = np.clip(c[i], -1, 1)
            c[i, ::128] = m * (-1) ** i
    elif case == "zeros":
        c[::2] = 0.0
        c[1, :128] = -0.0
    elif case == "small":
        c *= 2.0 ** np.array([-130, -126, -127, -120, -133, -100, -110, -118])[:, None]
    elif case == "large":
        c *= 2.0 ** np.array([10, 14, 15, 16, 17, 20, 100, 120])[:, None]
    elif case == "ties":  # every code's midpoint to the next
        mid = (ref.E4M3[:126] + ref.E4M3[1:127]) / 2
        c = np.resize(np.concatenate([mid, -mid, [448.0]]), (8, 512))
        c[:, ::128] = 448.0
    return torch.from_numpy(c.astype(np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("case", ["borders", "zeros", "small", "large", "ties"])
def test_codes_at_the_edges(case):
    rng = np.random.default_rng(0)
    d = setup(8, 2, 8, seed=1)
    d["c"] = values(case, rng).cuda()
    irm.device_status(irm.irm_pages_append(d["c"], d["k"], d["kv"], d["table"], d["row"], d["request"]))
    check(d)


def test_nan_and_infinity_mark_their_group():
    d = setup(4, 1, 8, seed=6)
    c = d["c"].clone()
    c[0, 5], c[1, 200], c[2, 511], c[3, 128] = float("nan"), float("inf"), -float("inf"), float("nan")
    d["c"] = c
    irm.device_status(irm.irm_pages_append(c, d["k"], d["kv"], d["table"], d["row"], d["request"]))
    at = d["np_table"][0, d["np_row"] // 64] * 64 + d["np_row"] % 64
    rows = ref.decode(d["kv"].cpu().numpy().reshape(-1, 656)[at])
    bad = np.isnan(rows[:, :512]).reshape(4, 4, 128)
    want = np.zeros((4, 4), bool)
    want[0, 0] = want[1, 1] = want[2, 3] = want[3, 1] = True
    assert np.array_equal(bad.all(2), want) and np.array_equal(bad.any(2), want)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("what", ["request", "negative request", "row", "page", "negative page"])
def test_bad_places_are_recorded(bits, what):
    d = setup(9, 3, bits, seed=4)
    row, request, table = d["np_row"].copy(), d["np_request"].copy(), d["np_table"].copy()
    if what == "request":
        request[4] = 3
    elif what == "negative request":
        request[4] = -1
    elif what == "row":
        row[4] = table.shape[1] * 64
    else:
        table[request[4], row[4] // 64] = d["n_pages"] if what == "page" else -1
    hit = np.arange(9) == 4
    if "page" in what:
        hit = (request == request[4]) & (row // 64 == row[4] // 64)
    ws = irm.irm_pages_append(d["c"], d["k"], d["kv"], i32(table), i32(row), i32(request))
    with pytest.raises(irm.IrmError) as e:
        irm.device_status(ws)
    assert e.value.status == -7
    check(d, skip=hit)


def test_stream_and_graph():
    """On a stream of its own, and captured: a replay writes the rows that the arrays name by then."""
    d = setup(30, 4, 8, seed=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = irm.irm_pages_append(d["c"], d["k"], d["kv"], d["table"], d["row"], d["request"], stream=s)
    irm.device_status(ws, s)
    check(d)
    row, kv = d["row"].clone(), torch.full_like(d["kv"], 0x55)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        irm.irm_pages_append(d["c"], d["k"], kv, d["table"], row, d["request"], workspace=ws)
    row.copy_(torch.where(torch.arange(30, device="cuda") % 2 == 0, d["row"], -1))
    g.replay()
    irm.device_status(ws)
    check(dict(d, kv=kv), skip=np.arange(30) % 2 == 1)


# ------------------------------------------------------------------ queries

@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (3, 7), (33, 1), (64, 16), (5, 100), (2, 255), (2, 256), (3, 257), (1, 700), (100, 24)])
@pytest.mark.parametrize("pairing", [irm.ROPE_NEOX, irm.ROPE_INTERLEAVED])
def test_queries(T, H, pairing):
    rng = np.random.default_rng(T * H)
    q = torch.from_numpy(rng.standard_normal((T, H, 192)).astype(np.float32)).to(torch.bfloat16).cuda()
    pos = rng.integers(0, 200000, T)
    rope = irm.Rope.make(rope_tables()["yarn"], pairing)
    kw = dict(inv_freq=rope_tables()["yarn"], interleaved=pairing == irm.ROPE_INTERLEAVED, factor=1.5)
    x = q[:, :, 128:].double().cpu().numpy()
    where = np.broadcast_to(pos[:, None], (T, H))
    out = irm.irm_rope_apply(q[:, :, 128:], i32(pos), rope, 1.5)
    assert out.is_contiguous()
    near(out.double().cpu().numpy(), x, where, **kw)
    # in place, in the middle of the head: the rest of it stays
    rest = q[:, :, :128].clone()
    got = irm.irm_rope_apply(q[:, :, 128:], i32(pos), rope, 1.5, out=q[:, :, 128:])
    assert torch.equal(got, out) and torch.equal(q[:, :, 128:], out) and torch.equal(q[:, :, :128], rest)


def test_query_layouts_agree():
    """Heads before tokens, broadcast heads, an output of other strides."""
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((12, 5, 64)).astype(np.float32)).to(torch.bfloat16).cuda()
    pos = i32(rng.integers(0, 5000, 12))
    want = irm.irm_rope_apply(x, pos)
    heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(irm.irm_rope_apply(heads_first, pos), want)
    out = torch.zeros((5, 12, 80), dtype=torch.bfloat16, device="cuda").transpose(0, 1)[:, :, 8:72]
    assert torch.equal(irm.irm_rope_apply(x, pos, out=out), want)
    one = x[:, :1].expand(12, 5, 64)
    assert torch.equal(irm.irm_rope_apply(one, pos), irm.irm_rope_apply(one.contiguous(), pos))


def test_turning_back_and_gradient():
    """A negative position undoes a rotation; with the same factor it is the rotation's gradient: the transposed
    map, against the reference's 64-bit rotation as a linear map and against differences of it."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 2, 64))
    g = torch.from_numpy(rng.standard_normal((6, 2, 64)).astype(np.float32)).to(torch.bfloat16)
    pos = rng.integers(0, 100000, 6)
    where = np.broadcast_to(pos[:, None], (6, 2))
    back = irm.irm_rope_apply(g.cuda(), i32(-pos), factor=1.25).double().cpu().numpy()
    near(back, g.double().numpy(), -where, factor=1.25)
    gn = g.double().numpy()
    f = lambda z: (ref.rotate(z, where, factor=1.25) * gn).sum()  # noqa: E731
    for _ in range(20):
        i = tuple(rng.integers(0, s) for s in x.shape)
        e = np.zeros_like(x)
        e[i] = 1.0  # the map is linear: a difference of any size is exact up to 64-bit rounding
        slope = f(x + e) - f(x)
        pair = np.abs(gn[i[:2]]).max() * 2
        assert abs(slope - back[i]) <= STEP * abs(slope) + 2.0 ** -20 * 1.25 * pair + 1e-9


def test_query_stream_graph_and_no_tokens():
    x = torch.randn((9, 4, 64), device="cuda").to(torch.bfloat16)
    pos = i32(np.arange(9))
    want = irm.irm_rope_apply(x, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = irm.irm_rope_apply(x, pos, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out, p = torch.zeros_like(x), pos.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        irm.irm_rope_apply(x, p, out=out)
    p.add_(100)
    g.replay()
    assert torch.equal(out, irm.irm_rope_apply(x, pos + 100))
    assert irm.irm_rope_apply(x[:0], pos[:0]).shape == (0, 4, 64)
