"""Speculative decoding over the paged MLA cache: what is measured, in plain form and as the library's calls.

Three operators: attention of a tree of drafted tokens over 64-row pages, verification of the
drafted tokens against the target model's probabilities, and the page operations around them
(resize, fork, compact, copy).  `own` chooses what run() does: False, elementary torch
operations; True, the calls of mla_position_independent_gb300.
"""
import math

import numpy as np
import torch

own = False

PAGE, D_LAT, D_ROPE, D_ROW = 64, 512, 64, 576
SCALE = 1.0 / math.sqrt(192.0)
VOCAB = 102400


# --------------------------------------------------------------------------------- cases

def listed():
    return [
        # one short conversation, one token at a time: latency is everything
        dict(name="attn_one_token", op="attn", B=1, H=16, ctx=512, nodes=1, ragged=False),
        # a small model's batch (16 heads, 8 x 8192), trees of 16 drafts
        dict(name="attn_8x8192_16h_16n", op="attn", B=8, H=16, ctx=8192, nodes=16, ragged=False),
        # a large model's batch (128 heads, 64 x 32768), short trees: every page is read once
        dict(name="attn_64x32768_128h_2n", op="attn", B=64, H=128, ctx=32768, nodes=2, ragged=False),
        # one long document (128 heads), a wide tree: the KV of one request is split over the GPU
        dict(name="attn_1x16384_128h_61n", op="attn", B=1, H=128, ctx=16384, nodes=61, ragged=False),
        # mixed traffic: contexts from a few rows to thousands, odd tree sizes, a head count that divides nothing
        dict(name="attn_ragged_23x5000_24h", op="attn", B=23, H=24, ctx=5000, nodes=13, ragged=True),
        # one request, a short chain of drafts
        dict(name="verify_1x8", op="verify", B=1, nodes=8, vocab=VOCAB, q=False),
        # a full batch with top-k trees of 32 nodes
        dict(name="verify_64x32", op="verify", B=64, nodes=32, vocab=VOCAB, q=False),
        # children sampled from a draft model whose probabilities take part in the test
        dict(name="verify_16x24_draft_probs", op="verify", B=16, nodes=24, vocab=VOCAB, q=True),
        # two requests admitted, one step, released: bookkeeping alone
        dict(name="pages_step_2", op="step", B=2, ctx=300, nodes=8, layers=4),
        # a full batch's step over every layer's cache
        dict(name="pages_step_64", op="step", B=64, ctx=4000, nodes=32, layers=32),
        # parallel sampling: 64 branches of 16 prompts, their partial pages copied in every layer
        dict(name="pages_fork_64", op="fork", B=16, forks=64, ctx=2000, layers=32),
        # moving a quarter of a cache to other pages
        dict(name="pages_copy_1500", op="copy", pages=6000, n=1500, layers=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "verify", "verify", "step", "fork", "copy"])
    if op == "attn":
        H = rng.choice([1, 7, 16, 16, 24, 32, 40, 64, 100, 128, 128])
        B, n = _log(rng, 1, 64), _log(rng, 1, 64)
        top = max(1, min(32768, int(1.1e12 / (B * n * H * 2176.0)), 2_000_000 // B))
        return dict(op="attn", B=B, H=H, ctx=_log(rng, 1, top), nodes=n, ragged=rng.random() < 0.6)
    if op == "verify":
        B = _log(rng, 1, 64)
        return dict(op="verify", B=B, nodes=_log(rng, 1, 64 if B <= 24 else 32), vocab=_log(rng, 50, VOCAB),
                    q=rng.random() < 0.4 and B <= 24)
    if op == "step":
        return dict(op="step", B=_log(rng, 1, 64), ctx=_log(rng, 1, 4000), nodes=_log(rng, 1, 64), layers=_log(rng, 1, 24))
    if op == "fork":
        return dict(op="fork", B=_log(rng, 1, 16), forks=_log(rng, 1, 64), ctx=_log(rng, 1, 2000), layers=_log(rng, 1, 32))
    n = _log(rng, 1, 1500)
    return dict(op="copy", pages=2 * n + rng.randrange(3 * n), n=n, layers=_log(rng, 1, 16))


# -------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return x.normal_(0.0, std, generator=g)


def _tree(rng, n, shape):
    """Parents of n nodes (parent[0] = -1): a chain, or a tree whose nodes hang on one of the last few."""
    par = np.full(n, -1, np.int32)
    for i in range(1, n):
        par[i] = i - 1 if shape == "chain" else int(rng.integers(max(0, (i - 1) // 4 - 1), (i - 1) // 2 + 1))
    return par


def _ancestors(par):
    """seen[i, k]: node k is i or one of its ancestors."""
    seen = np.eye(len(par), dtype=bool)
    for i in range(1, len(par)):
        seen[i] |= seen[par[i]]
    return seen


def _sized(case):
    """Random numbers of a case's lengths: another seed gives other values, not other sizes."""
    return np.random.default_rng([case["B"], case["ctx"], case.get("nodes", 0)])


def _lengths(case):
    """Contexts and tree sizes of a batch: all alike, or spread over their range."""
    B, ctx, n = case["B"], case["ctx"], case["nodes"]
    rng = _sized(case)
    if not case.get("ragged"):
        return np.full(B, ctx, np.int32), np.full(B, n, np.int32)
    c = np.exp(rng.uniform(0.0, math.log(ctx + 1.0), B)).astype(np.int32)
    c[0] = ctx
    k = rng.integers(1, n + 1, B).astype(np.int32)
    k[0] = n
    return np.clip(c, 0, ctx).astype(np.int32), k


def prepare(case, seed):
    g, rng = _gen(seed), np.random.default_rng(int(seed) % (1 << 32))
    return {"attn": _prepare_attn, "verify": _prepare_verify, "step": _prepare_step, "fork": _prepare_fork,
            "copy": _prepare_copy}[case["op"]](case, g, rng)


def _prepare_attn(case, g, rng):
    ctx, n = _lengths(case)
    B, H = case["B"], case["H"]
    indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T, words = int(indptr[-1]), (int(n.max()) + 31) // 32
    mask = np.zeros((T, words * 32), bool)
    for b in range(B):
        mask[indptr[b]:indptr[b + 1], :n[b]] = _ancestors(_tree(rng, int(n[b]), "tree"))
    bits = np.packbits(mask, axis=1, bitorder="little").view(np.int32)
    pages = (ctx + n + PAGE - 1) // PAGE
    table = np.full((B, int(pages.max())), -1, np.int32)
    order, at = rng.permutation(int(pages.sum())).astype(np.int32), 0
    for b in range(B):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
    return dict(op="attn", H=H, ctx=ctx, indptr=indptr, kv=_normal(g, (int(pages.sum()), PAGE, D_ROW)),
                table=torch.from_numpy(table).cuda(), mask=torch.from_numpy(bits).cuda(),
                q_lat=_normal(g, (T, H, D_LAT), 1.0 / math.sqrt(192.0)), q_rope=_normal(g, (T, H, D_ROPE), 1.0 / math.sqrt(192.0)))


def _prepare_verify(case, g, rng):
    B, n, V, q = case["B"], case["nodes"], case["vocab"], case["q"]
    T = B * n
    indptr = (np.arange(B + 1) * n).astype(np.int32)
    par = np.concatenate([_tree(rng, n, "tree") for _ in range(B)])
    rank = np.zeros(T, np.int64)  # how many earlier nodes share the parent
    for b in range(B):
        p = par[b * n:(b + 1) * n]
        rank[b * n:(b + 1) * n] = np.tril(p[:, None] == p[None, :], -1).sum(1)
    logits = torch.empty((T, V), device="cuda").normal_(0.0, 3.0, generator=g)
    draft = torch.softmax(logits + torch.empty((T, V), device="cuda").normal_(0.0, 0.7, generator=g), 1)
    logits = torch.softmax(logits, 1)
    row = torch.from_numpy(np.maximum(np.repeat(indptr[:-1], n) + par, 0)).cuda().long()  # each node's parent's row
    if q:  # drawn from the draft model at the parent, one by one
        tokens = torch.multinomial(draft[row], 1, generator=g)[:, 0]
    else:  # the draft model's best tokens at the parent
        k = min(int(rank.max()) + 1, V)
        tokens = draft.topk(k, 1).indices[row, torch.from_numpy(np.minimum(rank, k - 1)).cuda()]
    return dict(op="verify", indptr=indptr, parents=torch.from_numpy(par).cuda(), tokens=tokens.int(), target=logits,
                draft=draft if q else None, uniforms=torch.rand(T, generator=g, device="cuda"), n=n)


def _prepare_step(case, g, rng):
    B, ctx, n, L = case["B"], case["ctx"], case["nodes"], case["layers"]
    base = _sized(case).integers(max(1, ctx // 2), ctx + 1, B).astype(np.int32)
    wide = (ctx + n + PAGE - 1) // PAGE
    depth = np.zeros(B, np.int32)
    path = np.full((B, n), -1, np.int32)
    for b in range(B):  # a path of the tree, as verification leaves it
        par, u, k = _tree(rng, n, "tree"), 0, 1
        path[b, 0] = 0
        while rng.random() < 0.75 and (kids := np.nonzero(par == u)[0]).size:
            u = int(rng.choice(kids))
            path[b, k] = u
            k += 1
        depth[b] = k
    pages = int(((base + n + PAGE - 1) // PAGE).sum()) + 64
    refcount = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refcount[torch.from_numpy(rng.choice(pages, 64, replace=False)).cuda()] = 1  # other requests' pages
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    return dict(op="step", kv=_normal(g, (L, pages, PAGE, D_ROW)), table=torch.full((B, wide), -1, dtype=torch.int32, device="cuda"),
                refcount=refcount, seq=torch.zeros(B, dtype=torch.int32, device="cuda"), base=dev(base), drafted=dev(base + n),
                kept=dev(base + depth), path=dev(path), depth=dev(depth), none=torch.zeros(B, dtype=torch.int32, device="cuda"))


def _prepare_fork(case, g, rng):
    B, F, ctx, L = case["B"], case["forks"], case["ctx"], case["layers"]
    length = np.zeros(B + F, np.int32)
    length[:B] = _sized(case).integers(max(1, ctx // 2), ctx + 1, B)
    held = (length + PAGE - 1) // PAGE
    pages = int(held.sum()) + F + 16
    order, at = rng.permutation(pages).astype(np.int32), 0
    table = np.full((B + F, (ctx + PAGE - 1) // PAGE), -1, np.int32)
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    refcount = np.zeros(pages, np.int32)
    refcount[order[:at]] = 1
    src, dst = rng.integers(0, B, F).astype(np.int32), (B + rng.permutation(F)).astype(np.int32)
    back = length.copy()
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    return dict(op="fork", kv=_normal(g, (L, pages, PAGE, D_ROW)), table=dev(table), refcount=dev(refcount), seq=dev(length),
                src=src, dst=dst, src_dev=dev(src).long(), dst_dev=dev(dst).long(), back=dev(back))


def _prepare_copy(case, g, rng):
    order = rng.permutation(case["pages"]).astype(np.int32)
    src, dst = order[:case["n"]].copy(), order[case["n"]:2 * case["n"]].copy()
    return dict(op="copy", kv=_normal(g, (case["layers"], case["pages"], PAGE, D_ROW)), src=src, dst=dst,
                src_dev=torch.from_numpy(src).cuda().long(), dst_dev=torch.from_numpy(dst).cuda().long())


# ----------------------------------------------------------------------------------- run

def run(state):
    return {"attn": _run_attn, "verify": _run_verify, "step": _run_step, "fork": _run_fork, "copy": _run_copy}[state["op"]](state)


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
    kv = s["kv"][s["table"].clamp(min=0).long()].reshape(B, -1, D_ROW).float()
    S = kv.shape[1]
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


def _run_verify(s):
    if own:
        import mla_position_independent_gb300 as irm
        if "ws" not in s:
            s["ws"] = irm.new_workspace(irm.WORKSPACE_HEADER)
        return irm.irm_tree_verify(s["target"], s["tokens"], s["parents"], s["uniforms"], s["indptr"], draft_probs=s["draft"],
                                   workspace=s["ws"])[:3]
    n, B = s["n"], len(s["indptr"]) - 1
    dev, V = s["target"].device, s["target"].shape[1]
    first = torch.arange(B, device=dev) * n
    tokens, parents, r = (s[k].reshape(B, n) for k in ("tokens", "parents", "uniforms"))
    at = torch.zeros(B, dtype=torch.int64, device=dev)  # the node that the walk has reached
    w = s["target"][first].double()
    left = torch.ones(B, dtype=torch.float64, device=dev)
    path = torch.full((B, n), -1, dtype=torch.int32, device=dev)
    path[:, 0] = 0
    depth = torch.ones(B, dtype=torch.int64, device=dev)
    for i in range(1, n):  # a node is looked at after its earlier siblings, and they after their parent
        child = parents[:, i] == at
        x = tokens[:, i:i + 1].long()
        wx = w.gather(1, x)[:, 0]
        if s["draft"] is not None:
            q = s["draft"][first + at].double()
            taken = child & (r[:, i].double() * q.gather(1, x)[:, 0] * left < wx)
            rest = torch.clamp(w - q * left[:, None], min=0.0)
            rest_sum = rest.sum(1)
        else:
            taken = child & (r[:, i].double() * left < wx)
            rest = w.scatter(1, x, 0.0)
            rest_sum = left - wx
        lost = child & ~taken
        w = torch.where(lost[:, None], rest, w)
        left = torch.where(lost, rest_sum, left)
        at = torch.where(taken, i, at)
        w = torch.where(taken[:, None], s["target"][first + at].double(), w)
        left = torch.where(taken, 1.0, left)
        path.scatter_(1, depth.clamp(max=n - 1)[:, None], torch.where(taken, i, path.gather(1, depth.clamp(max=n - 1)[:, None])[:, 0]).int()[:, None])
        depth = depth + taken
    w = torch.where(w.sum(1, keepdim=True) > 0, w, s["target"][first + at].double())
    sums = w.cumsum(1)
    token = (sums <= r[:, :1].double() * sums[:, -1:]).sum(1).clamp(max=V - 1)
    return depth.int(), path, token.int()


def _resize(s, new_len):
    """Releases, then the lowest free pages in request order; nothing grows where they do not suffice."""
    i = torch.arange(s["table"].shape[1], device=new_len.device)
    old, new = (s["seq"] + PAGE - 1) // PAGE, (new_len + PAGE - 1) // PAGE
    gone = (i >= new[:, None]) & (i < old[:, None])
    s["refcount"].scatter_add_(0, torch.where(gone, s["table"], 0).flatten().long(), -gone.flatten().int())
    want = (i >= old[:, None]) & (i < new[:, None])
    free = s["refcount"] == 0
    enough = want.sum() <= free.sum()
    want &= enough
    order = torch.argsort((~free).int(), stable=True)
    page = order[(want.flatten().cumsum(0) - 1).clamp(0, len(free) - 1)].reshape(want.shape).int()
    s["table"].copy_(torch.where(want, page, torch.where(gone, -1, s["table"])))
    s["refcount"].scatter_add_(0, torch.where(want, page, 0).flatten().long(), want.flatten().int())
    s["seq"].copy_(torch.where(enough | (new_len <= s["seq"]), new_len, s["seq"]))


def _run_step(s):
    """A batch's pages are taken (prompt and drafts), the accepted drafts' rows moved up, the rest given back, and at last all."""
    if own:
        import mla_position_independent_gb300 as irm
        if "ws" not in s:
            s["ws"] = irm.new_workspace(irm.pages_workspace_size(s["table"].shape[0]))
        pages = (s["seq"], s["table"], s["refcount"])
        irm.irm_pages_resize(s["drafted"], *pages, workspace=s["ws"])
        irm.irm_pages_compact(s["kv"], s["table"], s["base"], s["path"], s["depth"], workspace=s["ws"])
        irm.irm_pages_resize(s["kept"], *pages, workspace=s["ws"])
        irm.irm_pages_resize(s["none"], *pages, workspace=s["ws"])
        return s["kv"], s["table"], s["refcount"], s["seq"]
    _resize(s, s["drafted"])
    k = torch.arange(s["path"].shape[1], device=s["path"].device)
    moved = k < s["depth"][:, None]
    of, to = (s["base"][:, None] + torch.where(moved, x, 0) for x in (s["path"], k))
    row = lambda p: torch.gather(s["table"], 1, (p // PAGE).long()).long() * PAGE + p % PAGE  # noqa: E731
    rows = s["kv"].view(s["kv"].shape[0], -1, D_ROW)
    rows[:, row(to).flatten()] = rows[:, row(of).flatten()]
    _resize(s, s["kept"])
    _resize(s, s["none"])
    return s["kv"], s["table"], s["refcount"], s["seq"]


def _run_fork(s):
    """Branches of some requests are made, and given back."""
    if own:
        import mla_position_independent_gb300 as irm
        if "ws" not in s:
            s["ws"] = irm.new_workspace(irm.pages_workspace_size(s["table"].shape[0]))
        irm.irm_pages_fork(s["src"], s["dst"], s["kv"], s["seq"], s["table"], s["refcount"], workspace=s["ws"])
        irm.irm_pages_resize(s["back"], s["seq"], s["table"], s["refcount"], workspace=s["ws"])
        return s["kv"], s["table"], s["refcount"], s["seq"]
    src, dst = s["src_dev"], s["dst_dev"]
    length = s["seq"][src]
    i = torch.arange(s["table"].shape[1], device=length.device)
    old = s["table"][src]
    whole = i < (length // PAGE)[:, None]
    part = (i == (length // PAGE)[:, None]) & (length % PAGE > 0)[:, None]
    s["refcount"].scatter_add_(0, torch.where(whole, old, 0).flatten().long(), whole.flatten().int())
    order = torch.argsort((s["refcount"] != 0).int(), stable=True)
    has = length % PAGE > 0
    fresh = order[(has.cumsum(0) - 1).clamp(min=0)]
    s["refcount"].scatter_add_(0, torch.where(has, fresh, 0), has.int())
    s["table"][dst] = torch.where(whole, old, torch.where(part, fresh[:, None].int(), -1))
    s["seq"][dst] = length
    r = torch.arange(PAGE, device=length.device)
    of = torch.gather(old, 1, (length // PAGE).clamp(max=old.shape[1] - 1)[:, None].long()).long() * PAGE + r
    to = torch.where(r < (length % PAGE)[:, None], fresh[:, None] * PAGE + r, -1)
    of = torch.where(to >= 0, of, of[:, :1].clamp(min=0))
    to = torch.where(to >= 0, to, of)  # rows that are not copied stay as they are
    rows = s["kv"].view(s["kv"].shape[0], -1, D_ROW)
    rows[:, to.flatten()] = rows[:, of.flatten()]
    _resize(s, s["back"])
    return s["kv"], s["table"], s["refcount"], s["seq"]


def _run_copy(s):
    if own:
        import mla_position_independent_gb300 as irm
        irm.irm_pages_copy(s["kv"], s["src"], s["dst"])
        return s["kv"]
    s["kv"][:, s["dst_dev"]] = s["kv"][:, s["src_dev"]]
    return s["kv"]


# ---------------------------------------------------------------------------------- work

def _sizes(case):
    """Mean lengths of a batch: ragged ones are spread over the logarithm of their range."""
    if not case.get("ragged"):
        return float(case["ctx"]), float(case["nodes"])
    rest = case["ctx"] / math.log(case["ctx"] + 1.0)
    mean = lambda first, other: (first + (case["B"] - 1) * other) / case["B"]  # noqa: E731
    return mean(case["ctx"], rest), mean(case["nodes"], (case["nodes"] + 1) / 2.0)


def work(case):
    if case["op"] == "attn":
        ctx, n = _sizes(case)
        rows = case["B"] * n * case["H"]
        return {"bytes": case["B"] * (ctx + n) * 2 * D_ROW + rows * (2 * D_ROW + 2 * D_LAT + 4),
                "flops": rows * (ctx + n) * 2.0 * (D_ROW + D_LAT)}
    if case["op"] == "verify":  # the row that the next token is drawn from, and the tree
        return {"bytes": case["B"] * (case["vocab"] * 4.0 * (2 if case["q"] else 1) + case["nodes"] * 24), "flops": case["B"] * case["vocab"] * 2.0}
    if case["op"] == "step":  # some four rows of each request and layer move; the tables are written and read
        pages = case["B"] * (case["ctx"] * 0.75 + case["nodes"]) / PAGE
        return {"bytes": case["B"] * case["layers"] * min(4, case["nodes"]) * 4.0 * D_ROW + pages * 16, "flops": 0}
    if case["op"] == "fork":  # half a page of each fork and layer
        pages = case["forks"] * case["ctx"] * 0.75 / PAGE
        return {"bytes": case["forks"] * case["layers"] * (min(case["ctx"], PAGE) / 2.0) * 4 * D_ROW + pages * 16, "flops": 0}
    return {"bytes": case["n"] * case["layers"] * PAGE * 4.0 * D_ROW, "flops": 0}


# --------------------------------------------------------------------------------- exact

def exact(case, seed):
    """Attention in 64 bits, request by request; the other operators give whole numbers or moved rows."""
    if case["op"] != "attn" or work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    outs, lses = [], []
    for b in range(case["B"]):
        lo, hi, ctx = int(s["indptr"][b]), int(s["indptr"][b + 1]), int(s["ctx"][b])
        n, H = hi - lo, case["H"]
        rows = s["kv"][s["table"][b][: (ctx + n + PAGE - 1) // PAGE].long()].reshape(-1, D_ROW)[: ctx + n].double()
        words = s["mask"][lo:hi].cpu().numpy().view(np.uint8)
        seen = torch.from_numpy(np.unpackbits(words, axis=1, bitorder="little")[:, :n].astype(bool)).cuda()
        for at in range(0, n, 8):  # a few nodes at a time
            ql, qr = (s[k][lo + at:min(hi, lo + at + 8)].double() for k in ("q_lat", "q_rope"))
            z = (ql.reshape(-1, D_LAT) @ rows[:, :D_LAT].T + qr.reshape(-1, D_ROPE) @ rows[:, D_LAT:].T) / math.sqrt(192.0)
            z = z.reshape(ql.shape[0], H, -1)
            z[:, :, ctx:].masked_fill_(~seen[at:at + 8, None, :], -math.inf)
            lse = torch.logsumexp(z, 2)
            p = torch.exp(z - lse[..., None])
            outs.append((p.reshape(-1, ctx + n) @ rows[:, :D_LAT]).reshape(-1, H, D_LAT))
            lses.append(lse)
    return torch.cat(outs), torch.cat(lses)
