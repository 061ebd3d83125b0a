"""Refusals of the speculative-decoding entry points on the host (no GPU: every check comes before
any copy or launch; the device pointers below are never dereferenced), and the 64-bit
references' own checks."""
import ctypes

import numpy as np
import pytest

import spec_reference as ref

FAKE, WS = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)


@pytest.fixture(scope="module")
def irm():
    from mla_position_independent_gb300 import build
    build.build()
    import mla_position_independent_gb300 as m
    m.lib()
    return m


def i32(*x):
    return np.array(x, np.int32)


def tree_args(ctx=(100, 7), indptr=(0, 3, 5), H=16, q_lat=FAKE, kv=FAKE, n_pages=10, max_pages=2, words=1, scale=0.1,
              ws=WS, ws_bytes=1 << 30, table=FAKE, mask=FAKE, lse=None):
    c, p = i32(*ctx), i32(*indptr)
    keep = (c, p)
    return keep, (q_lat, FAKE, len(ctx), H, c.ctypes.data, p.ctypes.data, kv, n_pages, table, max_pages, mask, words,
                  ctypes.c_float(scale), FAKE, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(H=0), -4), (dict(H=129), -4), (dict(ctx=(-1, 7)), -1), (dict(indptr=(1, 3, 5)), -1),
    (dict(indptr=(0, 3, 2)), -1), (dict(indptr=(0, 1025, 1026), max_pages=100, words=40), -4),
    (dict(max_pages=1), -1), (dict(words=0), -1), (dict(indptr=(0, 33, 40), words=1), -1),
    (dict(n_pages=0), -4), (dict(n_pages=1 << 25), -4), (dict(scale=float("nan")), -1), (dict(scale=0.0), -1), (dict(scale=3e38), -1),
    (dict(q_lat=ctypes.c_void_p((1 << 20) + 8)), -1), (dict(kv=None), -1), (dict(table=ctypes.c_void_p((1 << 20) + 2)), -1),
    (dict(lse=ctypes.c_void_p((1 << 20) + 2)), -1), (dict(ws=None), -8), (dict(ws_bytes=255), -8),
    (dict(ws=ctypes.c_void_p((1 << 21) + 128)), -8), (dict(ctx=(2**31 - 10, 7), max_pages=2**25), -4),
])
def test_tree_attention_refusals(irm, change, code):
    keep, args = tree_args(**change)
    L = irm.lib()
    assert L.irm_mla_attn_tree(*args) == code, L.irm_last_error()
    assert L.irm_last_error()


def test_tree_attention_null_tables(irm):
    L, n = irm.lib(), ctypes.c_size_t(0)
    p = i32(0, 3)
    assert L.irm_mla_attn_tree_workspace_size(None, p.ctypes.data, 1, 16, ctypes.byref(n)) == -1
    assert L.irm_mla_attn_tree_workspace_size(p.ctypes.data, None, 1, 16, ctypes.byref(n)) == -1
    assert L.irm_mla_attn_tree_workspace_size(p.ctypes.data, p.ctypes.data, 0, 16, ctypes.byref(n)) == -1
    assert L.irm_mla_attn_tree_workspace_size(p.ctypes.data, p.ctypes.data, 1, 16, None) == -1
    assert irm.tree_workspace_size(i32(100), p, 16) >= 256


@pytest.mark.parametrize("B,ctx,nodes", [(256, 20_000_000, 1024), (256, 2_000_000_000, 1024), (300, 2_000_000_000, 1),
                                         (1, 2_000_000_000, 1024), (1, 2_000_000_000, 1)])
def test_tree_attention_workspace_of_the_largest_batches(irm, B, ctx, nodes):
    # at most 8192 partials of 128 rows of 512 + 1 fp32, however many pieces and row tiles there are
    size = irm.tree_workspace_size(np.full(B, ctx), np.arange(B + 1) * nodes, 128)
    assert 256 <= size <= 256 + 8192 * 128 * 513 * 4 + 512


def test_tree_attention_no_nodes_is_no_launch(irm):
    keep, args = tree_args(indptr=(0, 0, 0))
    assert irm.lib().irm_mla_attn_tree(*args) == 0


@pytest.mark.parametrize("change,code", [
    (dict(vocab=0), -4), (dict(vocab=(1 << 20) + 1, stride=1 << 21), -4), (dict(stride=99), -1), (dict(max_path=0), -1),
    (dict(indptr=(0, 1025)), -4), (dict(indptr=(0, -1)), -1), (dict(target=None), -1), (dict(out=None), -1),
    (dict(target=ctypes.c_void_p((1 << 20) + 2)), -1), (dict(ws=None), -8), (dict(ws_bytes=100), -8),
])
def test_verify_refusals(irm, change, code):
    d = dict(vocab=100, stride=100, max_path=4, indptr=(0, 5), target=FAKE, out=FAKE, ws=WS, ws_bytes=256)
    d.update(change)
    p = i32(*d["indptr"])
    st = irm.lib().irm_tree_verify(d["target"], None, d["stride"], d["vocab"], FAKE, FAKE, FAKE, p.ctypes.data, len(p) - 1,
                                   d["max_path"], d["out"], FAKE, FAKE, d["ws"], d["ws_bytes"], None)
    assert st == code, irm.lib().irm_last_error()


@pytest.mark.parametrize("change,code", [
    (dict(n_slots=0), -4), (dict(n_slots=8193), -4), (dict(max_pages=0), -1), (dict(n_pages=0), -4), (dict(seq=None), -1),
    (dict(seq=ctypes.c_void_p((1 << 20) + 1)), -1), (dict(ws=None), -8), (dict(ws_bytes=256), -8),
    (dict(n_slots=8192, max_pages=(1 << 17) + 1), -4),
])
def test_resize_refusals(irm, change, code):
    d = dict(n_slots=4, max_pages=4, n_pages=100, seq=FAKE, ws=WS, ws_bytes=1 << 20)
    d.update(change)
    st = irm.lib().irm_pages_resize(FAKE, d["seq"], d["n_slots"], FAKE, d["max_pages"], FAKE, d["n_pages"], d["ws"],
                                    d["ws_bytes"], None)
    assert st == code, irm.lib().irm_last_error()


@pytest.mark.parametrize("src,dst,code", [
    ((0, 1), (2, 2), -1), ((0, 1), (2, 0), -1), ((0, 4), (2, 3), -1), ((0, -1), (2, 3), -1), ((0,), (4,), -1),
    (tuple([0] * 1025), tuple(range(1, 1026)), -4),
])
def test_fork_refusals(irm, src, dst, code):
    s, t = i32(*src), i32(*dst)
    n_slots = 4 if len(src) < 100 else 2000
    st = irm.lib().irm_pages_fork(s.ctypes.data, t.ctypes.data, len(s), FAKE, 1, FAKE, n_slots, FAKE, 4, FAKE, 100, WS,
                                  1 << 20, None)
    assert st == code, irm.lib().irm_last_error()
    # the check leaves no marks behind: the same slots are fine in the next call, up to the workspace
    s, t = i32(0, 0), i32(2, 3)
    assert irm.lib().irm_pages_fork(s.ctypes.data, t.ctypes.data, 2, FAKE, 1, FAKE, 4, FAKE, 4, FAKE, 100, None, 0, None) == -8


def test_fork_of_nothing_is_no_launch(irm):
    assert irm.lib().irm_pages_fork(None, None, 0, FAKE, 1, FAKE, 4, FAKE, 4, FAKE, 100, WS, 1 << 20, None) == 0


@pytest.mark.parametrize("change,code", [
    (dict(kv=None), -1), (dict(kv=ctypes.c_void_p((1 << 20) + 8)), -1), (dict(layers=0), -4), (dict(layers=65536), -4),
    (dict(max_path=0), -1), (dict(base=None), -1), (dict(ws=None), -8),
])
def test_compact_refusals(irm, change, code):
    d = dict(kv=FAKE, layers=2, max_path=4, base=FAKE, ws=WS)
    d.update(change)
    st = irm.lib().irm_pages_compact(d["kv"], d["layers"], 100, FAKE, 4, 3, d["base"], FAKE, d["max_path"], FAKE, d["ws"],
                                     256, None)
    assert st == code, irm.lib().irm_last_error()


@pytest.mark.parametrize("src,dst", [((0, 1), (2, 2)), ((0, 1), (2, 1)), ((0, 10), (2, 3)), ((0, 1), (2, -3))])
def test_copy_refusals(irm, src, dst):
    s, t = i32(*src), i32(*dst)
    assert irm.lib().irm_pages_copy(FAKE, 1, 10, s.ctypes.data, t.ctypes.data, 2, None) == -1
    assert irm.lib().irm_pages_copy(FAKE, 1, 10, None, None, 0, None) == 0


def test_status_strings(irm):
    assert irm.lib().irm_status_string(-9) == b"too few free pages"
    assert irm.lib().irm_status_string(-10) == b"growth inside a shared page"


def test_binding_refuses_wrong_tensors(irm):
    """Shapes, types, devices and host arrays, before anything reaches the library."""
    import torch
    cpu = torch.zeros((3, 16, 512), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        irm.irm_mla_attn_tree(cpu, cpu, [10], [0, 3], cpu, cpu, cpu)
    with pytest.raises(ValueError, match="one entry more"):
        irm.irm_mla_attn_tree(cpu, cpu, [10, 3], [0, 3], cpu, cpu, cpu)
    with pytest.raises(ValueError, match="int32"):
        irm.tree_workspace_size(np.array([2**31]), [0, 1], 16)
    with pytest.raises(ValueError, match="integer"):
        irm.tree_workspace_size(np.array([1.5]), [0, 1], 16)
    with pytest.raises(ValueError, match="same length"):
        irm.irm_pages_copy(cpu, [1, 2], [3])
    with pytest.raises(irm.IrmError) as e:
        irm.pages_workspace_size(0)
    assert e.value.status == -4


# ------------------------------------------------------------------ the references themselves

def test_reference_attention_closed_forms():
    rng = np.random.default_rng(0)
    rows = rng.standard_normal((5, 576))
    q = np.zeros((2, 1, 576))
    seen = np.array([[False, False], [False, True]])
    O, L, _, _ = ref.tree_attention(q, rows, seen, 3, 0.5)  # zero queries: plain means
    assert np.allclose(O[0, 0], rows[:3, :512].mean(0)) and np.isclose(L[0, 0], np.log(3))
    assert np.allclose(O[1, 0], rows[[0, 1, 2, 4], :512].mean(0)) and np.isclose(L[1, 0], np.log(4))
    O, L, _, _ = ref.tree_attention(q, rows[3:], seen, 0, 0.5)  # nothing visible
    assert (O[0] == 0).all() and L[0, 0] == -np.inf and np.allclose(O[1, 0], rows[4, :512])


@pytest.mark.parametrize("draft", [False, True])
def test_reference_verification_keeps_the_targets_distribution(draft):
    """The first emitted token's exact distribution, by integration over the uniform numbers: each child's
    acceptance probability is the measure of its uniforms, so the walk's outcome tree sums up."""
    rng = np.random.default_rng(4)
    V = 5
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    got = np.zeros(V)

    def outcomes(w, S, kids, weight):
        """kids: tokens left to test, None = drawn from q now."""
        if not kids:
            got[:] += weight * w / w.sum()
            return
        for x, px in (enumerate(q) if draft else [(kids[0], 1.0)]):
            qx = q[x] if draft else 1.0
            a = min(1.0, w[x] / (qx * S))
            got[x] += weight * px * a
            if a < 1.0:
                rest = np.maximum(w - q * S, 0.0) if draft else np.where(np.arange(V) == x, 0.0, w)
                outcomes(rest, rest.sum() if draft else S - w[x], kids[1:], weight * px * (1 - a))

    outcomes(p.copy(), 1.0, [None, None] if draft else [3, 1, 0], 1.0)
    assert np.allclose(got, p, atol=1e-12)


def test_reference_pages_model():
    m = ref.Pages(3, 4, 6)
    m.resize([100, 64, 0])
    assert m.table[0][:2] == [0, 1] and m.table[1][0] == 2 and m.ref == [1, 1, 1, 0, 0, 0]
    assert m.fork([0], [2]) == [(1, 3, 36)] and m.ref == [2, 1, 1, 1, 0, 0] and m.table[2][:2] == [0, 3]
    m.resize([64, 64, 100])  # slot 0 now ends at a page's end
    m.resize([30, 64, 100])
    m.resize([31, 64, 100])  # page 0 is slot 2's as well
    assert m.status == {"shared"} and m.seq[0] == 30
    m.resize([30, 64 * 4, 64 * 4])
    assert m.status == {"shared", "pages"} and m.seq == [30, 64, 100]
