"""A speculative-decoding step, its operators together: a prompt assembled into pages by
irm_assemble_kv, then steps of resize -> drafts' rows -> tree attention -> verification ->
compaction -> resize.  After each step the pages must hold exactly the rows of the tokens that
were emitted, in order, and a plain decode over them must agree with the tree's own attention."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
import spec_reference as ref
from helpers import SCALE
from mla_position_independent_gb300 import synth
from test_gpu_tree import check as check_attention

pytestmark = pytest.mark.gpu
V, H = 50, 16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


def test_steps_over_assembled_pages():
    rng = np.random.default_rng(0)
    embed = torch.from_numpy(rng.standard_normal((V, 4000, 576)).astype(np.float32) * 0.5).to(torch.bfloat16)  # [token, position]
    prompt = [rng.integers(0, V, n) for n in (150, 64)]
    rows = torch.cat([embed[t, np.arange(len(t))] for t in prompt])
    chunks, indptr = synth.make_table([[(0, 150, 0, 0)], [(150, 64, 0, 0)]])
    S, L = 2, 1
    seq, refcount = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros(20, dtype=torch.int32, device="cuda")
    table = torch.full((S, 6), -1, dtype=torch.int32, device="cuda")
    kv = torch.full((20, 64, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = irm.new_workspace(1 << 24)
    irm.irm_pages_resize(torch.tensor([150, 64], dtype=torch.int32, device="cuda"), seq, table, refcount, workspace=ws)
    irm.device_status(irm.irm_assemble_kv(irm.ChunkTable(chunks, indptr), rows.cuda(), kv, table))
    have = [list(map(int, t)) for t in prompt]
    pending = [3, 7]  # sampled, not yet in the cache
    for step in range(12):
        nodes = [int(rng.integers(1, 20)), int(rng.integers(1, 20))]
        q_indptr = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        ctx = np.array([len(h) for h in have], np.int32)
        assert seq.tolist() == ctx.tolist()
        par = [np.array([-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, n)]) for n in nodes]
        seen = [ref.ancestors(p) for p in par]
        tokens = [np.concatenate([[pending[b]], rng.integers(0, V, nodes[b] - 1)]).astype(np.int32) for b in range(S)]
        base = torch.from_numpy(ctx).cuda()
        irm.irm_pages_resize(torch.from_numpy(ctx + np.array(nodes, np.int32)).cuda(), seq, table, refcount, workspace=ws)
        for b in range(S):  # the model writes the drafts' rows, each at its depth's position
            for i in range(nodes[b]):
                t, pos = int(ctx[b]) + i, int(ctx[b]) + int(seen[b][i].sum()) - 1
                kv[int(table[b, t // 64]), t % 64] = embed[tokens[b][i], pos].cuda()
        T = int(q_indptr[-1])
        W = 1
        c = dict(ctx=ctx, indptr=q_indptr, H=H, kv=kv, table=table, seen=seen,
                 mask=torch.from_numpy(np.concatenate([ref.mask_words(s, W) for s in seen])).cuda(),
                 q_lat=torch.randn((T, H, 512), device="cuda").to(torch.bfloat16), q_rope=torch.randn((T, H, 64), device="cuda").to(torch.bfloat16))
        out, lse, _ = irm.irm_mla_attn_tree(c["q_lat"], c["q_rope"], ctx, q_indptr, kv, table, c["mask"], SCALE,
                                            lse=torch.empty((T, H), dtype=torch.float32, device="cuda"), workspace=ws)
        irm.device_status(ws)
        check_attention(c, out, lse)
        p = torch.softmax(4 * torch.randn((T, V), device="cuda"), 1)
        for b in range(S):  # make the drafts likely
            for i in range(1, nodes[b]):
                p[q_indptr[b] + par[b][i], int(tokens[b][i])] += 0.5
        p /= p.sum(1, keepdim=True)
        n, path, nxt, _ = irm.irm_tree_verify(p, torch.from_numpy(np.concatenate(tokens)).cuda(), torch.from_numpy(np.concatenate(par).astype(np.int32)).cuda(),
                                              torch.rand(T, device="cuda"), q_indptr, workspace=ws)
        irm.irm_pages_compact(kv, table, base, path, n, workspace=ws)
        irm.irm_pages_resize(base + n, seq, table, refcount, workspace=ws)
        irm.device_status(ws)
        for b in range(S):
            k = int(n[b])
            have[b] += [int(tokens[b][i]) for i in path[b, :k].tolist()]
            pending[b] = int(nxt[b])
            got = kv[table[b, :-(-len(have[b]) // 64)].long()].reshape(-1, 576)[:len(have[b])].cpu()
            want = embed[np.array(have[b]), np.arange(len(have[b]))]
            assert torch.equal(got.view(torch.int16), want.view(torch.int16)), f"step {step}, request {b}"
        assert int((refcount > 0).sum()) == sum(-(-len(h) // 64) for h in have)
    assert sum(map(len, have)) > 214 + 24 + 4  # more than the root was accepted now and then
    # a tree of one node is the decode: the same rows through the chunk-table entry point
    qi = np.array([0, 1, 2], np.int32)
    ctx = np.array([len(h) - 1 for h in have], np.int32)
    one = torch.ones((2, 1), dtype=torch.int32, device="cuda")
    ql, qr = torch.randn((2, H, 512), device="cuda").to(torch.bfloat16), torch.randn((2, H, 64), device="cuda").to(torch.bfloat16)
    out, _, _ = irm.irm_mla_attn_tree(ql, qr, ctx, qi, kv, table, one, SCALE, workspace=ws)
    recs = [[], []]
    for b in range(2):
        for t in range(0, len(have[b]), 64):
            recs[b].append((int(table[b, t // 64]) * 64, min(64, len(have[b]) - t), 0, 0))
    dec, _, dws = irm.irm_mla_attn_decode(ql, qr, irm.ChunkTable(*synth.make_table(recs)), kv.reshape(-1, 576), SCALE)
    irm.device_status(dws)
    d, o = dec.double(), out.double()
    assert float((d - o).norm() / o.norm()) <= 5e-3
