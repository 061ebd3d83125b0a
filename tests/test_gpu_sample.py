"""Sampling from logits against its definition in 64 bits.

A weight is off by at most 2^-34 of itself (the exponent's two parts: ln2 / 32 is good to 2^-45 and taken up to
1405 times, 2^-34.5; the squares in the polynomial 2^-38) and half a unit of 2^-43 of the largest, so a
running sum over the sum is off by at most e = 2^-33 + V 2^-44 / (sum over the largest).  Tokens and kept sets
have to be the reference's unless its own decision was nearer than 2 e to a border, which the inputs
(fixed seeds) hardly ever are: such a row's token must then be one that is left.  Probabilities are fp32 of
weights from fp32 exponentials (2^-22 of themselves, and up to 44 octaves x 2^-24) or better: 2^-18 of
themselves."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
import sample_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


def f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def check(logits, r, temperature=None, k=None, p=None, m=None, want_probs=True, **kw):
    T, V = logits.shape
    probs = torch.full((T, V), 7.0, dtype=torch.float32, device="cuda") if want_probs else None
    dev = lambda x, f: None if x is None else f(x)  # noqa: E731
    token, probs, ws = irm.irm_sample(logits, f32(r), dev(temperature, f32), dev(k, i32), dev(p, f32), dev(m, f32), probs=probs, **kw)
    irm.device_status(ws)
    got, pr = token.cpu().numpy(), None if probs is None else probs.double().cpu().numpy()
    l = logits.double().cpu().numpy()
    one = lambda x, t, d: d if x is None else float(np.asarray(x, np.float32)[t])  # noqa: E731
    near = 0
    for t in range(T):
        args = (one(temperature, t, 1.0), 0 if k is None else int(k[t]), one(p, t, 1.0), one(m, t, 0.0))
        w, order, n, margin = ref.kept(l[t], *args)
        token, gap = ref.draw(w, float(np.float32(r[t])))
        e = 2.0 ** -33 + V * 2.0 ** -44 / max(1.0, w.sum())
        if margin <= 2 * e:
            near += 1
            continue
        if gap <= 2 * e:
            near += 1
            assert got[t] >= 0 and w[got[t]] > 0
        else:
            assert got[t] == token, f"row {t}: {got[t]}, not {token} (settings {args})"
        if pr is not None:
            if n == 0:
                assert (pr[t] == 0).all()
                continue
            want = w / w.sum()
            tiny = want < 2.0 ** -42  # below a unit of the largest weight: zero or what it is
            assert ((pr[t] == 0) | (want > 0)).all() and (pr[t][(want > 0) & ~tiny] > 0).all()
            assert (np.abs(pr[t] - want)[~tiny] <= 2.0 ** -18 * want[~tiny]).all() and (pr[t][tiny] <= 2.0 ** -41).all()
    assert near <= max(1, T // 20)
    return token, probs


def normal(T, V, seed=0, std=3.0, dtype=torch.float32):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.standard_normal((T, V)) * std).astype(np.float32)).to(dtype).cuda(), rng.random(T, np.float32)


SETTINGS = [dict(), dict(temperature=0.7), dict(k=5), dict(k=1), dict(k=600), dict(p=0.9), dict(p=0.999), dict(p=0.02), dict(m=0.05),
            dict(k=50, p=0.9), dict(k=2000, p=0.95, temperature=1.3), dict(p=0.8, m=0.1), dict(k=40, p=0.95, m=0.02, temperature=0.6),
            dict(temperature=0.0), dict(p=0.95, temperature=5.0), dict(k=1000, temperature=0.01)]


@pytest.mark.parametrize("V", [1, 2, 3, 31, 127, 1000, 1025, 5000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_vocabularies(V, dtype):
    for i, s in enumerate(SETTINGS):
        l, r = normal(9, V, seed=V + i, dtype=dtype)
        check(l, r, **{n: np.full(9, x) for n, x in s.items()})


@pytest.mark.parametrize("s", SETTINGS)
def test_large_vocabulary(s):
    for dtype, V in ((torch.float32, 102400), (torch.bfloat16, 102403)):
        l, r = normal(5, V, seed=len(s), dtype=dtype)
        check(l, r, **{n: np.full(5, x) for n, x in s.items()})


@pytest.mark.parametrize("T,V", [(1, 102400), (3, 262144), (2, 500000), (1, 1 << 20), (300, 4000), (40, 60000), (700, 300)])
def test_shapes(T, V):
    """One CTA a row up to clusters of eight; rows that do not stay in shared memory."""
    rng = np.random.default_rng(T)
    l, r = normal(T, V, seed=T)
    check(l, r, temperature=rng.choice([0.6, 1.0, 1.4], T), k=rng.choice([0, 0, 20, 3000], T), p=rng.choice([1.0, 0.9, 0.5], T),
          m=rng.choice([0.0, 0.03], T))


def test_settings_differ_by_row():
    rng = np.random.default_rng(1)
    l, r = normal(200, 3001, seed=3)
    check(l, r, temperature=rng.choice([0.0, 0.5, 1.0, 2.0], 200), k=rng.choice([-1, 0, 1, 3, 50, 5000], 200),
          p=rng.choice([0.0, 0.1, 0.9, 1.0, 1.5, -1.0], 200), m=rng.choice([0.0, -1.0, 0.1, 0.9, 1.0], 200))


@pytest.mark.parametrize("V", [40, 700, 3000, 102400])
@pytest.mark.parametrize("kind", ["constant", "two values", "few values", "steps", "one peak"])
def test_ties(V, kind):
    """Equal logits: the lowest index comes first, at every cut."""
    rng = np.random.default_rng(V)
    l = {"constant": np.full((6, V), 2.5), "two values": rng.choice([1.0, 1.0 + 2.0 ** -20], (6, V)), "few values": rng.integers(0, 3, (6, V)) / 4.0,
         "steps": np.broadcast_to(np.arange(V) // 600 * 2.0 ** -12, (6, V)), "one peak": np.where(np.arange(V) == V // 2, 30.0, 0.0) * np.ones((6, 1))}[kind]
    x = f32(l)
    r = rng.random(6, np.float32)
    for s in (dict(), dict(k=5), dict(k=V // 2 + 1), dict(k=V - 1), dict(p=0.31), dict(p=0.77), dict(k=V // 3 + 2, p=0.6), dict(m=0.99), dict(m=1.0)):
        check(x, r, **{n: np.full(6, v) for n, v in s.items()})


def test_special_values():
    V = 1500
    rng = np.random.default_rng(7)
    l = rng.standard_normal((12, V)).astype(np.float32) * 3
    l[0, ::2] = -np.inf
    l[1] = -np.inf
    l[2] = np.nan
    l[3, 100:] = np.nan
    l[4, [3, 700, 1499]] = np.inf
    l[5] = -np.inf
    l[5, 77] = -3.0e38
    l[6] = 3.0e38
    l[6, 5] = -3.0e38
    l[7] *= 1e-40  # denormal logits
    l[8] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    l[9] *= 1e30
    l[10, 1:] = -np.inf
    l[11] = -50.0 + l[11] * 1e-4
    r = rng.random(12, np.float32)
    for s in (dict(), dict(k=3), dict(p=0.5), dict(m=0.2), dict(temperature=0.0), dict(temperature=np.inf), dict(temperature=np.nan),
              dict(temperature=1e-38), dict(p=np.nan), dict(m=np.nan), dict(temperature=-1.0), dict(temperature=1e30)):
        check(f32(l), r, **{n: np.full(12, x) for n, x in s.items()})


@pytest.mark.parametrize("r", [0.0, 1.0 - 2.0 ** -24, 0.5])
def test_ends_of_the_uniforms(r):
    """0 draws the first entry left, the largest number below 1 the last one."""
    l, _ = normal(8, 5000, seed=2)
    for s in (dict(), dict(k=7), dict(p=0.9), dict(m=0.1)):
        check(l, np.full(8, r), **{n: np.full(8, x) for n, x in s.items()})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off,ld", [(0, 1003), (1, 1004), (3, 1010), (4, 1008), (0, 1200)])
def test_strides_and_alignment(dtype, off, ld):
    l, r = normal(5, ld, seed=off, dtype=dtype)
    V = 1000
    x = l[:, off:off + V]
    buf = torch.full((5, ld + 8), -5.0, device="cuda")
    probs = buf[:, off:off + V]
    k, p = i32(np.full(5, 100)), f32(np.full(5, 0.9))
    token, _, ws = irm.irm_sample(x, f32(r), None, k, p, probs=probs)
    irm.device_status(ws)
    want, wp = check(x.contiguous(), r, k=np.full(5, 100), p=np.full(5, 0.9))
    assert torch.equal(token, irm.irm_sample(x.contiguous(), f32(r), None, k, p)[0]) and torch.equal(probs, wp)
    rest = torch.cat([buf[:, :off], buf[:, off + V:]], 1)
    assert (rest == -5.0).all()


def test_outputs_are_optional_and_repeat():
    l, r = normal(20, 4000, seed=5)
    p = f32(np.full(20, 0.9))
    token, probs, _ = irm.irm_sample(l, f32(r), top_p=p, probs=torch.empty_like(l))
    alone, none, _ = irm.irm_sample(l, f32(r), top_p=p)
    assert none is None and torch.equal(alone, token)
    nothing, only, _ = irm.irm_sample(l, None, top_p=p, probs=torch.empty_like(l))
    assert nothing is None and torch.equal(only, probs)
    for _ in range(3):
        again = irm.irm_sample(l, f32(r), top_p=p, probs=torch.empty_like(l))
        assert torch.equal(again[0], token) and torch.equal(again[1], probs)
    assert irm.irm_sample(l[:0], f32(r[:0]))[0].shape == (0,)


def test_split_does_not_matter():
    """The same rows alone and in a batch (other clusters) give the same tokens and probabilities."""
    l, r = normal(320, 30000, seed=8)
    p, k = f32(np.full(320, 0.95)), i32(np.full(320, 900))
    tok, pr, _ = irm.irm_sample(l, f32(r), None, k, p, probs=torch.empty_like(l))
    for t in (0, 100, 319):
        a, b, _ = irm.irm_sample(l[t:t + 1], f32(r[t:t + 1]), None, k[:1], p[:1], probs=torch.empty_like(l[:1]))
        assert torch.equal(a, tok[t:t + 1]) and torch.equal(b, pr[t:t + 1])


def test_stream_and_graph():
    l, r = normal(6, 9000, seed=9)
    r, p = f32(r), f32(np.full(6, 0.8))
    want = irm.irm_sample(l, r, top_p=p)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = irm.irm_sample(l, r, top_p=p, stream=s)[0]
    s.synchronize()
    assert torch.equal(got, want)
    ws, tok, x = irm.new_workspace(irm.WORKSPACE_HEADER), torch.zeros(6, dtype=torch.int32, device="cuda"), l.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        irm.irm_sample(x, r, top_p=p, token=tok, workspace=ws)
    x.copy_(l.flip(0))
    g.replay()
    assert torch.equal(tok, irm.irm_sample(l.flip(0).contiguous(), r, top_p=p)[0])


def test_drawn_tokens_follow_the_probabilities():
    """Many draws of one row: counts against the probabilities, within five standard deviations."""
    V, n = 50, 20000
    l, _ = normal(1, V, seed=3, std=1.0)
    r = (np.arange(n) + 0.5) / n  # evenly spread: a token's count is off by at most one
    probs = torch.empty((n, V), device="cuda")
    token, probs, _ = irm.irm_sample(l.expand(n, V).contiguous(), f32(r), top_k=i32(np.full(n, 20)), probs=probs)
    got = np.bincount(token.cpu().numpy(), minlength=V)
    assert (np.abs(got - n * probs[0].double().cpu().numpy()) <= 1.1).all()


@pytest.mark.parametrize("V,std", [(600000, 3.0), (102400, 0.3), (400000, 0.02), (30000, 0.01)])
@pytest.mark.parametrize("s", [dict(p=0.95), dict(p=0.5), dict(k=1000), dict(k=20000, p=0.9)])
def test_many_equal_logits_at_the_cut(V, std, s):
    """bf16 logits, of which hundreds to thousands share a value; and beside them fp32 ones a few steps apart."""
    l, r = normal(3, V, seed=V, std=std, dtype=torch.bfloat16)
    full = {k: np.full(3, v) for k, v in s.items()}
    check(l, r, **full)
    near = (1.0 + torch.randint(0, 3, l.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 2.0 ** -20).float()
    check(near, r, **full)


@pytest.mark.parametrize("temperature", [0.3, 0.7, 0.8, 1.0, 1.3, 3.0, 20.0])
def test_small_probabilities(temperature):
    """Wide rows, whose probabilities go down to 2^-42 and are still good to 2^-18 of themselves."""
    l, r = normal(6, 20000, seed=11, std=14.0)
    check(l, r, temperature=np.full(6, temperature))
    check(l + 1000.0, r, temperature=np.full(6, temperature))
