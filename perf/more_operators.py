"""A serving step over the paged MLA cache: what is measured, in plain form and as the library's calls.

Four operators: appending a step's rows to the pages with the rotation on the way (bf16 or 8-bit
pages), the rotation of the queries, attention of drafted trees (or single tokens) over 8-bit
pages, and sampling from logits.  `own` chooses what run() does: False, elementary torch
operations; True, the calls of mla_position_independent_gb300.

A row of the 8-bit cache is 656 bytes: 512 e4m3 codes, 4 fp32 scales (powers of two, one for 128
columns), 64 bf16 of k_r.
"""
import math

import numpy as np
import torch

own = False

PAGE, D_LAT, D_ROPE, D_ROW, ROW8 = 64, 512, 64, 576, 656
SCALE = 1.0 / math.sqrt(192.0)
VOCAB = 102400


# --------------------------------------------------------------------------------- cases

def listed():
    return [
        # one short conversation, one token at a time: latency is everything
        dict(name="attn8_one_token", op="attn", B=1, H=16, ctx=512, nodes=1, ragged=False),
        # a small model's plain decode (16 heads, 8 x 8192): the cache's bytes
        dict(name="attn8_8x8192_16h", op="attn", B=8, H=16, ctx=8192, nodes=1, ragged=False),
        # a large model's batch (128 heads, 64 x 32768) with short trees: the tensor cores
        dict(name="attn8_64x32768_128h_2n", op="attn", B=64, H=128, ctx=32768, nodes=2, ragged=False),
        # mixed traffic: contexts from a few rows to thousands, odd tree sizes, a head count that divides nothing
        dict(name="attn8_ragged_23x5000_24h", op="attn", B=23, H=24, ctx=5000, nodes=13, ragged=True),
        # a decode step's rows, one a request, into 8-bit pages
        dict(name="append8_64", op="append", T=64, B=64, ctx=2000, bits=8, yarn=False, interleaved=False),
        # a chunk of prompts into 8-bit pages, positions scaled for long contexts
        dict(name="append8_8191", op="append", T=8191, B=5, ctx=60000, bits=8, yarn=True, interleaved=True),
        # a long prompt's chunk into bf16 pages
        dict(name="append_16384", op="append", T=16384, B=2, ctx=4000, bits=16, yarn=False, interleaved=False),
        # the queries of a decode step of 16 heads, rotated out of the projection's [T, H, 192]
        dict(name="rope_64x16h", op="rope", T=64, H=16, far=8192, yarn=False, interleaved=False),
        # the queries of a prompt's chunk, 128 heads, positions scaled for long contexts
        dict(name="rope_8192x128h", op="rope", T=8192, H=128, far=131072, yarn=True, interleaved=True),
        # one conversation's next token, top-k and top-p
        dict(name="sample_1", op="sample", T=1, vocab=VOCAB, bf16=False, k=50, p=0.9, m=0.0, mixed=False, probs=False),
        # a batch whose requests each bring their own settings (some greedy, some unrestricted)
        dict(name="sample_64_mixed", op="sample", T=64, vocab=VOCAB, bf16=False, k=0, p=1.0, m=0.0, mixed=True, probs=False),
        # every node of 16 trees of 24 drafts: the probabilities that the verification takes
        dict(name="sample_384_probs", op="sample", T=384, vocab=VOCAB, bf16=True, k=0, p=0.95, m=0.0, mixed=False, probs=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append", "rope", "sample", "sample"])
    if op == "attn":
        H = rng.choice([1, 7, 16, 16, 24, 32, 40, 64, 100, 128, 128])
        B, n = _log(rng, 1, 64), _log(rng, 1, 64)
        top = max(1, min(32768, int(1.1e12 / (B * n * H * 2176.0)), 2_000_000 // B))
        return dict(op="attn", B=B, H=H, ctx=_log(rng, 1, top), nodes=n, ragged=rng.random() < 0.6)
    if op == "append":
        T = _log(rng, 1, 16384)
        return dict(op="append", T=T, B=_log(rng, 1, min(T, 200)), ctx=_log(rng, 1, 100000), bits=rng.choice([8, 8, 16]),
                    yarn=rng.random() < 0.5, interleaved=rng.random() < 0.5)
    if op == "rope":
        H = rng.choice([1, 7, 16, 24, 40, 64, 100, 128])
        return dict(op="rope", T=_log(rng, 1, 1048576 // H if H > 64 else 8192), H=H, far=_log(rng, 1, 1000000), yarn=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5)
    return dict(op="sample", T=_log(rng, 1, 128), vocab=_log(rng, 2, VOCAB), bf16=rng.random() < 0.5, k=rng.choice([0, 0, 1, 20, 50, 1000]),
                p=rng.choice([1.0, 0.3, 0.9, 0.95]), m=rng.choice([0.0, 0.0, 0.02, 0.1]), mixed=rng.random() < 0.3, probs=rng.random() < 0.5)


# -------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _tree(rng, n):
    """Parents of n nodes (parent[0] = -1): a tree whose nodes hang on one of the last few."""
    par = np.full(n, -1, np.int32)
    for i in range(1, n):
        par[i] = int(rng.integers(max(0, (i - 1) // 4 - 1), (i - 1) // 2 + 1))
    return par


def _ancestors(par):
    """seen[i, k]: node k is i or one of its ancestors."""
    seen = np.eye(len(par), dtype=bool)
    for i in range(1, len(par)):
        seen[i] |= seen[par[i]]
    return seen


def _frequencies(yarn):
    """(angle per position of the 32 pairs, factor of the rotated vectors): base 10000, or that
    table stretched for 16 times 4096 positions (fast pairs kept, slow ones slowed by 16)."""
    f = 10000.0 ** (-2.0 * np.arange(32, dtype=np.float64) / 64.0)
    if not yarn:
        return f, 1.0
    at = lambda turns: 64.0 * math.log(4096.0 / (turns * 2.0 * math.pi)) / (2.0 * math.log(10000.0))  # noqa: E731
    lo, hi = max(0.0, math.floor(at(32.0))), min(63.0, math.ceil(at(1.0)))
    slow = np.clip((np.arange(32) - lo) / (hi - lo), 0.0, 1.0)
    return f * (1.0 - slow) + f / 16.0 * slow, 0.1 * math.log(16.0) + 1.0


def _quantized(c):
    """(codes, scales) of values [..., 512] fp32: the smallest power of two for which 128 columns fit e4m3."""
    x = c.reshape(*c.shape[:-1], 4, 128)
    m, e = torch.frexp(x.abs().amax(-1) / 448.0)  # 2^(e-1) <= amax / 448 < 2^e
    e = torch.where(m == 0.5, e - 1, e).clamp(-126, 7)
    e = torch.where(m == 0, 0, e)
    s = ((e + 127) << 23).int().view(torch.float32)  # 2^e
    codes = (x / s[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.reshape(c.shape), s


def _parts(kv):
    """Views of an 8-bit cache: codes [..., 512], scales [..., 4], k_r [..., 64]."""
    return kv[..., :512].view(torch.float8_e4m3fn), kv[..., 512:528].view(torch.float32), kv[..., 528:].view(torch.bfloat16)


def _sized(case):
    """Random numbers of a case's lengths: another seed gives other values, not other sizes."""
    return np.random.default_rng([case["B"], case["ctx"], case.get("nodes", 0)])


def _lengths(case):
    """Contexts and tree sizes of a batch: all alike, or spread over their range."""
    B, ctx, n = case["B"], case["ctx"], case["nodes"]
    rng = _sized(case)
    if not case["ragged"]:
        return np.full(B, ctx, np.int32), np.full(B, n, np.int32)
    c = np.exp(rng.uniform(0.0, math.log(ctx + 1.0), B)).astype(np.int32)
    c[0] = ctx
    k = rng.integers(1, n + 1, B).astype(np.int32)
    k[0] = n
    return np.clip(c, 0, ctx).astype(np.int32), k


def _table(rng, pages, spare):
    """Page table of requests that hold `pages` pages each, in a random order of all pages."""
    total = int(pages.sum()) + spare
    table = np.full((len(pages), max(1, int(pages.max()))), -1, np.int32)
    order, at = rng.permutation(total).astype(np.int32), 0
    for b in range(len(pages)):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
    return table, total


def prepare(case, seed):
    g, rng = _gen(seed), np.random.default_rng(int(seed) % (1 << 32))
    return {"attn": _prepare_attn, "append": _prepare_append, "rope": _prepare_rope, "sample": _prepare_sample}[case["op"]](case, g, rng)


def _prepare_attn(case, g, rng):
    ctx, n = _lengths(case)
    B, H = case["B"], case["H"]
    indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T, words = int(indptr[-1]), (int(n.max()) + 31) // 32
    mask = np.zeros((T, words * 32), bool)
    for b in range(B):
        mask[indptr[b]:indptr[b + 1], :n[b]] = _ancestors(_tree(rng, int(n[b])))
    bits = np.packbits(mask, axis=1, bitorder="little").view(np.int32)
    table, total = _table(rng, (ctx + n + PAGE - 1) // PAGE, 0)
    kv = torch.empty((total, PAGE, ROW8), dtype=torch.uint8, device="cuda")
    for p0 in range(0, total, 4096):  # rows as irm_pages_append leaves them
        part = kv[p0:p0 + 4096]
        codes, scales, k_r = _parts(part)
        c, s = _quantized(_normal(g, (*part.shape[:2], D_LAT), dtype=torch.float32))
        codes.copy_(c), scales.copy_(s), k_r.copy_(_normal(g, (*part.shape[:2], D_ROPE)))
    return dict(op="attn", H=H, ctx=ctx, indptr=indptr, kv=kv, table=_dev(table), mask=_dev(bits),
                q_lat=_normal(g, (T, H, D_LAT), 1.0 / math.sqrt(192.0)), q_rope=_normal(g, (T, H, D_ROPE), 1.0 / math.sqrt(192.0)))


def _prepare_append(case, g, rng):
    T, B = case["T"], case["B"]
    sizes = _sized(case)
    n = np.full(B, T // B, np.int64)  # new tokens of each request, behind what it holds
    n[:T % B] += 1
    base = sizes.integers(case["ctx"] // 2, case["ctx"] + 1, B)
    first = base // PAGE  # pages before it belong to no one here: only those that are written exist
    held = (base + n + PAGE - 1) // PAGE - first
    some, total = _table(rng, held, 8)
    table = np.full((B, int((first + held).max())), -1, np.int32)
    for b in range(B):
        table[b, first[b]:first[b] + held[b]] = some[b, :held[b]]
    request = np.repeat(np.arange(B), n)
    row = np.concatenate([np.arange(base[b], base[b] + n[b]) for b in range(B)])
    mix = rng.permutation(T)  # tokens of a batch come in any order
    request, row = request[mix].astype(np.int32), row[mix].astype(np.int32)
    shape = (total, PAGE, ROW8) if case["bits"] == 8 else (total, PAGE, D_ROW)
    kv = torch.zeros(shape, dtype=torch.uint8 if case["bits"] == 8 else torch.bfloat16, device="cuda")
    freq, factor = _frequencies(case["yarn"])
    return dict(op="append", kv=kv, table=_dev(table), request=_dev(request), row=_dev(row), freq=freq, factor=factor,
                interleaved=case["interleaved"], new=_normal(g, (T, D_ROW)))  # the projection's output, [cKV | k_r]


def _prepare_rope(case, g, rng):
    freq, factor = _frequencies(case["yarn"])
    return dict(op="rope", q=_normal(g, (case["T"], case["H"], 192)), position=_dev(rng.integers(0, case["far"] + 1, case["T"]).astype(np.int32)),
                freq=freq, factor=factor, interleaved=case["interleaved"])


def _prepare_sample(case, g, rng):
    T, V = case["T"], case["vocab"]
    logits = _normal(g, (T, V), 3.0, torch.bfloat16 if case["bf16"] else torch.float32)
    if case["mixed"]:
        pick = lambda *v: rng.choice(v, T)  # noqa: E731
        temp, k, p, m = pick(0.0, 0.6, 0.8, 1.0, 1.3), pick(0, 0, 20, 50, 400), pick(1.0, 0.5, 0.9, 0.95), pick(0.0, 0.0, 0.05)
    else:
        temp, k, p, m = np.full(T, 0.8), np.full(T, case["k"]), np.full(T, case["p"]), np.full(T, case["m"])
    return dict(op="sample", logits=logits, uniforms=torch.rand(T, generator=g, device="cuda"), temperature=_dev(temp.astype(np.float32)),
                k=_dev(k.astype(np.int32)), p=_dev(p.astype(np.float32)), m=_dev(m.astype(np.float32)), probs=case["probs"])


# ----------------------------------------------------------------------------------- run

def run(state):
    return {"attn": _run_attn, "append": _run_append, "rope": _run_rope, "sample": _run_sample}[state["op"]](state)


def _run_attn(s):
    if own:
        import mla_position_independent_gb300 as irm
        if "ws" not in s:
            s["ws"] = irm.new_workspace(irm.tree_workspace_size(s["ctx"], s["indptr"], s["H"]))
        lse = torch.empty(s["q_lat"].shape[:2], dtype=torch.float32, device="cuda")
        out, lse, _ = irm.irm_mla_attn_tree(s["q_lat"], s["q_rope"], s["ctx"], s["indptr"], s["kv"], s["table"], s["mask"],
                                            SCALE, lse=lse, workspace=s["ws"])
        return out, lse
    ctx, n = torch.from_numpy(s["ctx"]).cuda().long(), torch.from_numpy(np.diff(s["indptr"])).cuda().long()
    B, H, T = len(ctx), s["H"], s["q_lat"].shape[0]
    N, dev = int(np.diff(s["indptr"]).max()), s["kv"].device
    req = torch.repeat_interleave(torch.arange(B, device=dev), n, output_size=T)
    node = torch.arange(T, device=dev) - torch.from_numpy(s["indptr"][:-1]).cuda().long()[req]
    q = torch.zeros((B, N, H, D_ROW), device=dev)
    q[req, node] = torch.cat([s["q_lat"], s["q_rope"]], 2).float()
    codes, scales, k_r = _parts(s["kv"][s["table"].clamp(min=0).long()].reshape(B, -1, ROW8))
    S = codes.shape[1]
    kv = torch.cat([(codes.float().reshape(B, S, 4, 128) * scales[..., None]).reshape(B, S, D_LAT), k_r.float()], 2)
    t = torch.arange(S, device=dev)
    kv = torch.where((t < (ctx + n)[:, None])[..., None], kv, 0.0)  # pages hold anything past the last row
    drafted = (s["mask"][:, :, None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
    seen = torch.zeros((B, N, N), dtype=torch.bool, device=dev)
    seen[req, node] = drafted.reshape(T, -1)[:, :N].bool()
    slot = t - ctx[:, None]  # [B, S] draft slot of each row
    tail = torch.gather(seen, 2, slot.clamp(0, N - 1)[:, None, :].expand(B, N, S)) & (slot < n[:, None])[:, None, :]
    see = torch.where((slot < 0)[:, None, :], True, tail)  # [B, N, S]
    score = torch.matmul(q.reshape(B, N * H, D_ROW), kv.transpose(1, 2)).reshape(B, N, H, S).mul_(SCALE)
    score = score.masked_fill_(~see[:, :, None, :], -math.inf)
    top = score.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    score = score.sub_(top).exp_()
    total = score.sum(3, keepdim=True)
    out = torch.matmul(score.reshape(B, N * H, S), kv[..., :D_LAT]).reshape(B, N, H, D_LAT)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + total.log())[..., 0]
    return out[req, node].to(torch.bfloat16), lse[req, node]


def _rotated(x, position, freq, factor, interleaved):
    """x [T, ..., 64] turned by its positions; angles in 64 bits, since they are far."""
    a = position.double()[:, None] * torch.from_numpy(freq).to(x.device)
    c, s = ((f * factor).float().reshape(-1, *[1] * (x.dim() - 2), 32) for f in (a.cos(), a.sin()))
    x = x.float()
    if interleaved:
        u, v = x[..., 0::2], x[..., 1::2]
        return torch.stack([u * c - v * s, u * s + v * c], -1).flatten(-2).to(torch.bfloat16)
    u, v = x[..., :32], x[..., 32:]
    return torch.cat([u * c - v * s, u * s + v * c], -1).to(torch.bfloat16)


def _variant(s):
    import mla_position_independent_gb300 as irm
    if "rope" not in s:
        s["rope"] = irm.Rope.make(s["freq"], irm.ROPE_INTERLEAVED if s["interleaved"] else irm.ROPE_NEOX)
    return s["rope"]


def _run_append(s):
    kv, new = s["kv"], s["new"]
    if own:
        import mla_position_independent_gb300 as irm
        if "ws" not in s:
            s["ws"] = irm.new_workspace(irm.WORKSPACE_HEADER)
        irm.irm_pages_append(new[:, :D_LAT], new[:, D_LAT:], kv, s["table"], s["row"], s["request"], rope=_variant(s), factor=s["factor"],
                             workspace=s["ws"])
        return _parts(kv) if kv.dtype == torch.uint8 else kv
    row = s["row"].long()
    at = s["table"][s["request"].long(), row // PAGE].long(), row % PAGE
    k_r = _rotated(new[:, D_LAT:], s["row"], s["freq"], s["factor"], s["interleaved"])
    if kv.dtype != torch.uint8:
        kv[at] = torch.cat([new[:, :D_LAT], k_r], 1)
        return kv
    codes, scales = _quantized(new[:, :D_LAT].float())
    kv[at] = torch.cat([codes.view(torch.uint8), scales.view(torch.uint8), k_r.view(torch.uint8)], 1)
    return _parts(kv)


def _run_rope(s):
    if own:
        import mla_position_independent_gb300 as irm
        return irm.irm_rope_apply(s["q"][:, :, 128:], s["position"], rope=_variant(s), factor=s["factor"])
    return _rotated(s["q"][:, :, 128:], s["position"], s["freq"], s["factor"], s["interleaved"])


def _run_sample(s):
    if own:
        import mla_position_independent_gb300 as irm
        if "ws" not in s:
            s["ws"] = irm.new_workspace(irm.WORKSPACE_HEADER)
        probs = torch.empty(s["logits"].shape, dtype=torch.float32, device="cuda") if s["probs"] else None
        token, probs, _ = irm.irm_sample(s["logits"], s["uniforms"], s["temperature"], s["k"], s["p"], s["m"], probs=probs, workspace=s["ws"])
        return (token, probs) if s["probs"] else token
    l, V = s["logits"].double(), s["logits"].shape[1]
    t = s["temperature"].double()[:, None]
    best, index = l.sort(dim=1, descending=True, stable=True)  # ties: the lowest index first
    rank = torch.arange(V, device=l.device)
    k = torch.where(s["k"] > 0, s["k"], V)[:, None]
    k = torch.where(t > 0, k, 1)  # temperature 0: the best alone
    top = best[:, :1]
    best = torch.exp((best - top) / torch.where(t > 0, t, 1.0))
    best = torch.where(rank < k, best, 0.0)
    sums = best.cumsum(1)
    p = s["p"].double()[:, None]
    keep = (rank < k) & ((p >= 1) | (sums - best < p * sums[:, -1:])) & (best >= s["m"].double()[:, None])
    keep[:, 0] = True
    w = torch.zeros_like(l).scatter_(1, index, torch.where(keep, best, 0.0))
    sums = w.cumsum(1)
    token = (sums <= s["uniforms"].double()[:, None] * sums[:, -1:]).sum(1).clamp(max=V - 1).int()
    return (token, (w / sums[:, -1:]).float()) if s["probs"] else token


# ---------------------------------------------------------------------------------- work

def _sizes(case):
    """Mean lengths of a batch: ragged ones are spread over the logarithm of their range."""
    if not case["ragged"]:
        return float(case["ctx"]), float(case["nodes"])
    rest = case["ctx"] / math.log(case["ctx"] + 1.0)
    mean = lambda first, other: (first + (case["B"] - 1) * other) / case["B"]  # noqa: E731
    return mean(case["ctx"], rest), mean(case["nodes"], (case["nodes"] + 1) / 2.0)


def work(case):
    if case["op"] == "attn":
        ctx, n = _sizes(case)
        rows = case["B"] * n * case["H"]
        return {"bytes": case["B"] * (ctx + n) * ROW8 + rows * (2 * D_ROW + 2 * D_LAT + 4),
                "flops": rows * (ctx + n) * 2.0 * (D_ROW + D_LAT)}
    if case["op"] == "append":
        return {"bytes": case["T"] * (2.0 * D_ROW + (ROW8 if case["bits"] == 8 else 2 * D_ROW) + 12), "flops": case["T"] * D_LAT * 2.0}
    if case["op"] == "rope":
        return {"bytes": case["T"] * (case["H"] * 4.0 * D_ROPE + 4), "flops": case["T"] * case["H"] * 3.0 * D_ROPE}
    return {"bytes": case["T"] * case["vocab"] * ((2.0 if case["bf16"] else 4.0) + (4.0 if case["probs"] else 0.0)), "flops": case["T"] * case["vocab"] * 4.0}


# --------------------------------------------------------------------------------- exact

def exact(case, seed):
    """What run() returns, in 64 bits from the definitions (tokens are whole numbers: None)."""
    if case["op"] == "attn" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "rope": _exact_rope, "sample": _exact_sample}[case["op"]](s)


def _exact_attn(s):
    outs, lses = [], []
    for b in range(len(s["ctx"])):
        lo, hi, ctx = int(s["indptr"][b]), int(s["indptr"][b + 1]), int(s["ctx"][b])
        n, H = hi - lo, s["H"]
        raw = s["kv"][s["table"][b][: (ctx + n + PAGE - 1) // PAGE].long()].reshape(-1, ROW8)[: ctx + n]
        codes, scales, k_r = _parts(raw)
        lat, k_r = codes.double() * scales.double().repeat_interleave(128, 1), k_r.double()
        words = s["mask"][lo:hi].cpu().numpy().view(np.uint8)
        seen = torch.from_numpy(np.unpackbits(words, axis=1, bitorder="little")[:, :n].astype(bool)).cuda()
        for at in range(0, n, 8):  # a few nodes at a time
            ql, qr = (s[k][lo + at:min(hi, lo + at + 8)].double() for k in ("q_lat", "q_rope"))
            z = (ql.reshape(-1, D_LAT) @ lat.T + qr.reshape(-1, D_ROPE) @ k_r.T) / math.sqrt(192.0)
            z = z.reshape(ql.shape[0], H, -1)
            z[:, :, ctx:].masked_fill_(~seen[at:at + 8, None, :], -math.inf)
            lse = torch.logsumexp(z, 2)
            outs.append((torch.exp(z - lse[..., None]).reshape(-1, ctx + n) @ lat).reshape(-1, H, D_LAT))
            lses.append(lse)
    return torch.cat(outs), torch.cat(lses)


def _turned(x, position, s):
    """The pairs of x [..., 64] as complex numbers times factor e^(i position theta), in 64 bits."""
    turn = s["factor"] * torch.exp(1j * position.double()[..., None] * torch.from_numpy(s["freq"]).cuda())
    first, second = (slice(0, None, 2), slice(1, None, 2)) if s["interleaved"] else (slice(0, 32), slice(32, 64))
    z = torch.complex(x[..., first].double(), x[..., second].double()) * turn
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_append(s):
    """The rows, with the 8-bit cache's codes before they are rounded."""
    kv, new, row = s["kv"], s["new"].double(), s["row"].long()
    to = s["table"][s["request"].long(), row // PAGE].long() * PAGE + row % PAGE
    lat, k_r = new[:, :D_LAT], _turned(new[:, D_LAT:], s["row"], s)
    out = lambda v: torch.zeros((kv.shape[0] * PAGE, v.shape[1]), dtype=torch.float64, device="cuda").index_copy_(0, to, v).reshape(kv.shape[0], PAGE, -1)  # noqa: E731
    if kv.dtype != torch.uint8:
        return out(torch.cat([lat, k_r], 1))
    largest = lat.reshape(-1, 4, 128).abs().amax(2)
    scale = torch.where(largest > 0, torch.exp2(torch.ceil(torch.log2(largest / 448.0) - 1e-13)), 1.0)
    return out(lat / scale.repeat_interleave(128, 1)), out(scale), out(k_r)


def _exact_rope(s):
    return _turned(s["q"][:, :, 128:], s["position"][:, None], s)


def _exact_sample(s):
    """The probabilities, row by row: candidates in order of their logits, cut by each rule in turn."""
    if not s["probs"]:
        return None
    out = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    settings = [s[k].tolist() for k in ("temperature", "k", "p", "m")]
    for t, (temp, k, p, m) in enumerate(zip(*settings)):
        x = s["logits"][t].double()
        order = torch.argsort(-x, stable=True)
        if temp <= 0:
            out[t, order[0]] = 1.0
            continue
        left = order[:k] if k > 0 else order
        w = torch.softmax(x[left] / temp, 0)
        some = 1 + int((w.cumsum(0)[:-1] < p).sum()) if p < 1 else len(left)
        some = max(1, min(some, int((w >= m * w[0]).sum())))
        out[t, left[:some]] = w[:some] / w[:some].sum()
    return [None, out]
