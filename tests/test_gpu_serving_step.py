"""Steps of decoding over the paged cache with the calls as a program makes them: pages taken, queries rotated, rows
appended (rotated on the way), attention, probabilities from logits, drafts verified, the path's rows
moved up, the rest given back; then single tokens by irm_sample.  After every step the pages must hold
the rows of the tokens that were emitted, encoded at their positions, and the attention is checked
against the 64-bit formula over what the cache holds."""
import numpy as np
import pytest
import torch

import mla_position_independent_gb300 as irm
import row8_reference as ref8
import sample_reference
import spec_reference as ref
from helpers import SCALE, rope_tables
from test_gpu_tree import check as check_attention

pytestmark = pytest.mark.gpu
V, H, S = 60, 16, 3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    irm.lib()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def content(kv):
    """The rows that a cache holds, bf16 [n_pages, 64, 576]."""
    if kv.dtype != torch.uint8:
        return kv
    rows = ref8.decode(kv.cpu().numpy().reshape(-1, 656)).astype(np.float32)
    return torch.from_numpy(rows).to(torch.bfloat16).reshape(kv.shape[0], 64, 576).cuda()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("pairing", [irm.ROPE_NEOX, irm.ROPE_INTERLEAVED])
def test_steps(bits, pairing):
    rng = np.random.default_rng(bits + pairing)
    inv_freq, factor = rope_tables()["yarn"], 1.25
    rope = irm.Rope.make(inv_freq, pairing)
    hidden = torch.from_numpy(rng.standard_normal((V, 576)).astype(np.float32)).to(torch.bfloat16).cuda()  # a token's [cKV | k_r]
    n_pages = 30
    kv = torch.zeros((n_pages, 64, 656), dtype=torch.uint8, device="cuda") if bits == 8 else torch.zeros((n_pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    seq, count, table = i32(np.zeros(S)), i32(np.zeros(n_pages)), i32(np.full((S, 6), -1))
    ws = irm.new_workspace(1 << 24)

    def append(tokens, request, row, position):
        x = hidden[torch.from_numpy(np.asarray(tokens)).cuda().long()]
        irm.irm_pages_append(x[:, :512], x[:, 512:], kv, table, i32(row), i32(request), i32(position), rope, factor, workspace=ws)

    # prompts, appended in one call
    have = [list(rng.integers(0, V, n)) for n in (130, 64, 7)]
    irm.irm_pages_resize(i32([len(h) for h in have]), seq, table, count, workspace=ws)
    append(np.concatenate(have), np.repeat(np.arange(S), [len(h) for h in have]), *[np.concatenate([np.arange(len(h)) for h in have])] * 2)
    irm.device_status(ws)
    pending = [int(x) for x in rng.integers(0, V, S)]
    for step in range(8):
        nodes = [int(x) for x in rng.integers(1, 14, S)] if step < 6 else [1] * S  # the last steps token by token
        indptr = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        ctx = np.array([len(h) for h in have], np.int32)
        assert seq.tolist() == ctx.tolist()
        par = [np.array([-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, n)]) for n in nodes]
        seen = [ref.ancestors(p) for p in par]
        tokens = [np.concatenate([[pending[b]], rng.integers(0, V, nodes[b] - 1)]).astype(np.int32) for b in range(S)]
        request = np.repeat(np.arange(S), nodes)
        row = np.concatenate([ctx[b] + np.arange(nodes[b]) for b in range(S)])
        position = np.concatenate([ctx[b] + seen[b].sum(1) - 1 for b in range(S)])
        irm.irm_pages_resize(i32(ctx + np.array(nodes)), seq, table, count, workspace=ws)
        append(np.concatenate(tokens), request, row, position)
        T = int(indptr[-1])
        q = torch.randn((T, H, 192), device="cuda").to(torch.bfloat16)
        qr = irm.irm_rope_apply(q[:, :, 128:], i32(position), rope, factor)
        ql = torch.randn((T, H, 512), device="cuda").mul_(0.07).to(torch.bfloat16)
        mask = torch.from_numpy(np.concatenate([ref.mask_words(x, 1) for x in seen])).cuda()
        out, lse, _ = irm.irm_mla_attn_tree(ql, qr, ctx, indptr, kv, table, mask, SCALE, lse=torch.empty((T, H), device="cuda"), workspace=ws)
        irm.device_status(ws)
        check_attention(dict(ctx=ctx, indptr=indptr, H=H, kv=content(kv), table=table, seen=seen, q_lat=ql, q_rope=qr), out, lse)
        logits = torch.randn((T, V), device="cuda") * 2
        for b in range(S):  # make the drafts likely
            for i in range(1, nodes[b]):
                logits[indptr[b] + par[b][i], int(tokens[b][i])] += 6.0
        r = torch.rand(T, device="cuda")
        temperature, top_p = torch.full((T,), 0.8, device="cuda"), torch.full((T,), 0.95, device="cuda")
        if step < 6:
            probs = torch.empty((T, V), device="cuda")
            irm.irm_sample(logits, None, temperature, top_p=top_p, probs=probs, workspace=ws)
            n, path, token, _ = irm.irm_tree_verify(probs, i32(np.concatenate(tokens)), i32(np.concatenate(par)), r, indptr, workspace=ws)
            irm.irm_pages_compact(kv, table, i32(ctx), path, n, workspace=ws)
            irm.irm_pages_resize(i32(ctx) + n, seq, table, count, workspace=ws)
        else:
            token, _, _ = irm.irm_sample(logits, r, temperature, top_p=top_p, workspace=ws)
            n, path = i32(np.ones(S)), i32(np.zeros((S, 1)))
            for b in range(S):
                w, _, _, _ = sample_reference.kept(logits[b].cpu().numpy(), np.float32(0.8), 0, float(np.float32(0.95)))
                want, gap = sample_reference.draw(w, float(r[b]))
                assert int(token[b]) == want or gap < 1e-9
        irm.device_status(ws)
        held = content(kv)
        for b in range(S):
            k = int(n[b])
            have[b] += [int(tokens[b][i]) for i in path[b, :k].tolist()]
            pending[b] = int(token[b])
            got = held[table[b, :-(-len(have[b]) // 64)].long()].reshape(-1, 576)[:len(have[b])].double().cpu().numpy()
            x = hidden[torch.tensor(have[b]).cuda()].double().cpu().numpy()
            lat = x[:, :512]
            if bits == 8:
                codes, scales = ref8.encode(lat)
                lat = ref8.E4M3[codes] * np.repeat(scales, 128, 1)
            assert np.array_equal(got[:, :512], lat), f"step {step}, request {b}"
            want = ref8.rotate(x[:, 512:], np.arange(len(have[b])), inv_freq, pairing == irm.ROPE_INTERLEAVED, factor)
            assert np.abs(got[:, 512:] - want).max() <= 2.0 ** -8 * np.abs(want).max() + 2.0 ** -17
    assert sum(map(len, have)) > 201 + 24 + 3  # more than the roots were accepted now and then


def test_assembled_rows_into_the_8_bit_cache():
    """A reused request's rows, assembled in bf16 and appended as they are (already encoded)."""
    from mla_position_independent_gb300 import synth
    case = synth.custom_case([[(0, 32, 0, 0), (40, 100, 7, 1), (300, 61, 500, 1)]], n_rows=512, n_q=1, H=16, q_std=1.0)
    flat = torch.zeros((4, 64, 576), dtype=torch.bfloat16, device="cuda")
    order = i32(np.arange(4)[None])
    irm.device_status(irm.irm_assemble_kv(irm.ChunkTable(case.chunks, case.indptr), case.kv_rows.cuda(), flat, order))
    n = 193
    rows = flat.reshape(-1, 576)[:n]
    kv = torch.zeros((6, 64, 656), dtype=torch.uint8, device="cuda")
    table = i32([[5, 0, 3, 1]])
    irm.device_status(irm.irm_pages_append(rows[:, :512], rows[:, 512:], kv, table, i32(np.arange(n)), i32(np.zeros(n)), encoded=True))
    got = content(kv)[table[0].long()].reshape(-1, 576)[:n]
    codes, scales = ref8.encode(rows[:, :512].double().cpu().numpy())
    assert np.array_equal(got[:, :512].double().cpu().numpy(), ref8.E4M3[codes] * np.repeat(scales, 128, 1))
    assert torch.equal(got[:, 512:], rows[:, 512:])
