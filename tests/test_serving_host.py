"""Refusals of appending, rotation, sampling and the 8-bit cache's calls on the host (no GPU: every check comes
before any launch; the device pointers below are never dereferenced), and the references' own checks."""
import ctypes

import numpy as np
import pytest
import torch

import row8_reference as ref8
import sample_reference as refs

FAKE, WS = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 2)
EIGHT = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def irm():
    from mla_position_independent_gb300 import build
    build.build()
    import mla_position_independent_gb300 as m
    m.lib()
    return m


def rope(irm, **kw):
    r = irm.Rope.make(10000.0 ** (-np.arange(32) / 32.0))
    for k, v in kw.items():
        if k == "freq":
            r.inv_freq[3] = v
        else:
            setattr(r, k, v)
    return ctypes.cast(ctypes.pointer(r), ctypes.c_void_p), r


@pytest.mark.parametrize("suffix", ["", "8"])
@pytest.mark.parametrize("change,code", [
    (dict(c=None), -1), (dict(k=None), -1), (dict(kv=None), -1), (dict(table=None), -1), (dict(row=None), -1),
    (dict(c=EIGHT), -1), (dict(c_ld=577), -1), (dict(k=EIGHT), -1), (dict(k_ld=66), -1), (dict(c_ld=504), -1), (dict(k_ld=56), -1),
    (dict(kv=EIGHT), -1), (dict(table=ODD), -1), (dict(row=ODD), -1), (dict(request=ODD), -1), (dict(position=ODD), -1),
    (dict(T=-1), -1), (dict(T=1 << 31), -1), (dict(n_slots=0), -1), (dict(max_pages=0), -1), (dict(max_pages=1 << 30), -1), (dict(n_pages=0), -4),
    (dict(n_pages=1 << 25), -4), (dict(request=None, T=5), -1), (dict(encoded=2), -1), (dict(factor=float("inf")), -1),
    (dict(factor=float("nan")), -1), (dict(rope=dict(pairing=2)), -1), (dict(rope=dict(reserved=1)), -1), (dict(rope=dict(freq=float("nan"))), -1),
    (dict(ws=None), -8), (dict(ws_bytes=255), -8), (dict(ws=ctypes.c_void_p((1 << 21) + 128)), -8),
])
def test_append_refusals(irm, suffix, change, code):
    d = dict(c=FAKE, c_ld=576, k=FAKE, k_ld=576, T=4, kv=FAKE, n_pages=10, table=FAKE, n_slots=4, max_pages=3, row=FAKE, request=FAKE,
             position=None, rope=None, factor=1.0, encoded=0, ws=WS, ws_bytes=256)
    d.update(change)
    ptr, keep = rope(irm, **d["rope"]) if d["rope"] else (None, None)
    st = getattr(irm.lib(), "irm_pages_append" + suffix)(
        d["c"], d["c_ld"], d["k"], d["k_ld"], d["T"], d["kv"], d["n_pages"], d["table"], d["n_slots"], d["max_pages"], d["row"],
        d["request"], d["position"], ptr, d["factor"], d["encoded"], d["ws"], d["ws_bytes"], None)
    assert st == code, irm.lib().irm_last_error()
    assert irm.lib().irm_last_error()


@pytest.mark.parametrize("suffix", ["", "8"])
def test_append_of_nothing_is_no_launch(irm, suffix):
    assert getattr(irm.lib(), "irm_pages_append" + suffix)(FAKE, 576, FAKE, 576, 0, FAKE, 10, FAKE, 4, 3, FAKE, FAKE, None, None, 1.0, 0, WS,
                                                           256, None) == 0


@pytest.mark.parametrize("change,code", [
    (dict(x=None), -1), (dict(out=None), -1), (dict(position=None), -1), (dict(x=EIGHT), -1), (dict(out=EIGHT), -1), (dict(xt=196), -1),
    (dict(xh=63), -1), (dict(ot=12), -1), (dict(oh=68), -1), (dict(ot=56), -1), (dict(oh=0), -1), (dict(position=ODD), -1), (dict(T=-1), -1),
    (dict(H=0), -4), (dict(H=65536), -4), (dict(factor=float("nan")), -1), (dict(rope=dict(pairing=-1)), -1), (dict(rope=dict(freq=float("inf"))), -1),
])
def test_rotation_refusals(irm, change, code):
    d = dict(x=FAKE, xt=4096, xh=192, T=4, H=16, position=FAKE, rope=None, factor=1.0, out=FAKE, ot=1024, oh=64)
    d.update(change)
    ptr, keep = rope(irm, **d["rope"]) if d["rope"] else (None, None)
    st = irm.lib().irm_rope_apply(d["x"], d["xt"], d["xh"], d["T"], d["H"], d["position"], ptr, d["factor"], d["out"], d["ot"], d["oh"], None)
    assert st == code, irm.lib().irm_last_error()


def test_rotation_of_nothing_is_no_launch(irm):
    assert irm.lib().irm_rope_apply(FAKE, 1024, 64, 0, 16, FAKE, None, 1.0, FAKE, 1024, 64, None) == 0


@pytest.mark.parametrize("change,code", [
    (dict(type=2), -4), (dict(type=-1), -4), (dict(vocab=0), -4), (dict(vocab=(1 << 20) + 1, ld=1 << 21, pld=1 << 21), -4), (dict(ld=99), -1),
    (dict(pld=99), -1), (dict(token=None, probs=None), -1), (dict(logits=None), -1), (dict(uniforms=None), -1), (dict(logits=ODD), -1),
    (dict(logits=ctypes.c_void_p((1 << 20) + 1), type=1), -1), (dict(temperature=ODD), -1), (dict(k=ODD), -1), (dict(p=ODD), -1), (dict(m=ODD), -1),
    (dict(uniforms=ODD), -1), (dict(token=ODD), -1), (dict(probs=ODD), -1), (dict(T=-1), -1), (dict(T=1 << 28), -1), (dict(ws=None), -8),
    (dict(ws_bytes=255), -8),
])
def test_sampling_refusals(irm, change, code):
    d = dict(logits=FAKE, type=0, ld=100, T=3, vocab=100, temperature=None, k=None, p=None, m=None, uniforms=FAKE, token=FAKE, probs=FAKE, pld=100,
             ws=WS, ws_bytes=256)
    d.update(change)
    st = irm.lib().irm_sample(d["logits"], d["type"], d["ld"], d["T"], d["vocab"], d["temperature"], d["k"], d["p"], d["m"], d["uniforms"],
                              d["token"], d["probs"], d["pld"], d["ws"], d["ws_bytes"], None)
    assert st == code, irm.lib().irm_last_error()


def test_sampling_of_nothing_is_no_launch(irm):
    assert irm.lib().irm_sample(None, 0, 100, 0, 100, None, None, None, None, None, FAKE, None, 0, WS, 256, None) == 0


@pytest.mark.parametrize("off,type,ld,pld,T", [
    (0, 0, 100, 100, 3), (0, 0, 100, 100, 1), (4 * 299, 0, 100, 100, 3), (-4, 0, 100, 100, 1), (4 * 100, 0, 100, 120, 3), (4 * 50, 0, 250, 250, 3),
    (4 * 160, 0, 250, 250, 3), (-4 * 100, 0, 199, 199, 3), (2 * 98, 1, 400, 200, 3), (2 * 99, 1, 400, 200, 3), (2 * 2 * 150, 1, 402, 201, 3),
])
def test_probabilities_over_logits_are_refused(irm, off, type, ld, pld, T):
    probs = ctypes.c_void_p(FAKE.value + off)
    assert irm.lib().irm_sample(FAKE, type, ld, T, 100, None, None, None, None, FAKE, FAKE, probs, pld, WS, 256, None) == -1
    assert (b"overlap" if off % 4 == 0 else b"misaligned") in irm.lib().irm_last_error()


@pytest.mark.parametrize("T,H,ot,oh", [(4, 16, 960, 64), (4, 16, 64, 64), (4, 16, 64, 128), (4, 16, 192, 64), (4, 2, 96, 64), (2, 2, 64, 64)])
def test_rotated_rows_that_meet_are_refused(irm, T, H, ot, oh):
    assert irm.lib().irm_rope_apply(FAKE, 1024, 64, T, H, FAKE, None, 1.0, FAKE, ot, oh, None) == -1
    assert b"overlap" in irm.lib().irm_last_error()


def test_calls_over_the_8_bit_cache_refuse_as_the_others(irm):
    L, i32 = irm.lib(), lambda *x: np.array(x, np.int32)  # noqa: E731
    c, p = i32(100), i32(0, 3)
    args = [FAKE, FAKE, 1, 16, c.ctypes.data, p.ctypes.data, FAKE, 10, FAKE, 2, FAKE, 1, ctypes.c_float(0.1), FAKE, None, WS, 1 << 30, None]
    for at, value, code in ((3, 0, -4), (3, 129, -4), (6, None, -1), (6, EIGHT, -1), (7, 0, -4), (9, 1, -1), (11, 0, -1), (12, ctypes.c_float(0), -1),
                            (13, None, -1), (15, None, -8), (16, 10, -8)):
        bad = list(args)
        bad[at] = value
        assert L.irm_mla_attn_tree8(*bad) == code, (at, value)
    s, t = i32(0, 1), i32(2, 2)
    assert L.irm_pages_copy8(FAKE, 1, 10, s.ctypes.data, t.ctypes.data, 2, None) == -1
    assert L.irm_pages_fork8(s.ctypes.data, t.ctypes.data, 2, FAKE, 1, FAKE, 4, FAKE, 4, FAKE, 100, WS, 1 << 20, None) == -1
    assert L.irm_pages_compact8(FAKE, 0, 100, FAKE, 4, 3, FAKE, FAKE, 4, FAKE, WS, 256, None) == -4


def test_binding_refuses_wrong_tensors(irm):
    cpu = torch.zeros((3, 512), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="one layer"):
        irm.irm_pages_append(cpu, cpu, cpu, cpu, cpu)
    with pytest.raises(ValueError, match="GPU"):
        irm.irm_pages_append(cpu, cpu, torch.zeros((2, 64, 576), dtype=torch.bfloat16), cpu, cpu)
    with pytest.raises(ValueError, match="GPU"):
        irm.irm_rope_apply(torch.zeros((2, 2, 64), dtype=torch.bfloat16), cpu)
    with pytest.raises(ValueError, match="GPU"):
        irm.irm_sample(torch.zeros((2, 10)), None)
    with pytest.raises(ValueError, match="GPU"):
        irm.irm_mla_attn_tree(cpu[None], cpu, [10], [0, 1], torch.zeros((2, 64, 656), dtype=torch.uint8), cpu, cpu)


# ------------------------------------------------------------------ the references themselves

def test_reference_codes_are_the_types_own():
    x = torch.from_numpy(np.random.default_rng(0).standard_normal(20000).astype(np.float32) * 30).clamp(-448, 448)
    assert np.array_equal(ref8.nearest_code(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(every, ref8.E4M3, equal_nan=True)


def test_reference_rows_come_back():
    rng = np.random.default_rng(1)
    c = rng.standard_normal((5, 512)) * np.repeat([1.0, 100.0, 1e-3, 1e4], 128)
    codes, scales = ref8.encode(c)
    back = ref8.E4M3[codes] * np.repeat(scales, 128, 1)
    assert (np.abs(back - c) <= 2.0 ** -4 * np.abs(c) + 2.0 ** -10 * np.repeat(scales, 128, 1)).all()
    most = np.abs(c).reshape(5, 4, 128).max(2)
    assert (most <= 448 * scales).all() and (most > 448 * scales / 2).all()


def test_reference_rotation_closed_forms():
    x = np.random.default_rng(2).standard_normal((4, 64))
    p = np.array([3, 500, -7, 100000])
    for il in (False, True):
        y = ref8.rotate(x, p, interleaved=il)
        assert np.allclose(np.linalg.norm(y, axis=1), np.linalg.norm(x, axis=1))
        assert np.allclose(ref8.rotate(y, -p, interleaved=il), x)
        assert np.allclose(ref8.rotate(ref8.rotate(x, p, interleaved=il), p, interleaved=il), ref8.rotate(x, 2 * p, interleaved=il))
    e = np.zeros(64)
    e[1] = 1.0
    assert np.isclose(ref8.rotate(e, np.array(1), interleaved=True)[0], -np.sin(1.0))


def test_reference_sampling_closed_forms():
    l = np.log([0.1, 0.4, 0.1, 0.4])
    w, order, n, _ = refs.kept(l)
    assert list(order) == [1, 3, 0, 2] and n == 4
    assert [refs.draw(w, r)[0] for r in (0.0, 0.05, 0.11, 0.55, 0.7)] == [0, 0, 1, 2, 3]
    assert refs.kept(l, k=3)[2] == 3 and refs.kept(l, p=0.79)[2] == 2 and refs.kept(l, p=0.81)[2] == 3 and refs.kept(l, m=0.5)[2] == 2
    assert refs.kept(l, k=3, p=0.88)[2] == 2 and refs.kept(l, k=3, p=0.9)[2] == 3  # of 0.9 that are left
    assert refs.draw(refs.kept(l, temperature=0.0)[0], 0.99)[0] == 1 and refs.kept([-np.inf] * 3)[2] == 0
