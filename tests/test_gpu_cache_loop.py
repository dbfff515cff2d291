"""The cache operators and the verify step together, as a decode loop uses them:
prompts in ragged chunks (append, chunk attention), then steps of tree build,
append of the tree's nodes, tree attention, acceptance and commit, and a plain
token between.  After every step the cache holds exactly the accepted tokens'
keys and values, and the next attention over it equals the 64-bit attention
over the whole accepted sequence."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_jt_gb300 as jt
from kv_util import HALF_STEP, PAGE, chunk_bounds, chunk_ref, slots
from test_gpu_kv_cache import bits, heads_ref

pytestmark = pytest.mark.gpu
Hq, Hkv, D, V, LAYERS = 8, 4, 128, 400, 2
I32 = dict(dtype=torch.int32, device="cuda")


class Model:
    """Random projections of token embeddings: what a layer's q, k, v are."""

    def __init__(self, dtype, seed=5):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.dtype = dtype
        width = (Hq + 2 * Hkv) * D
        self.emb = [torch.randn(V, width, generator=g, device="cuda").to(dtype) for _ in range(LAYERS)]
        self.qw = (torch.randn(D, generator=g, device="cuda") * 0.2 + 1).to(dtype)
        self.kw = (torch.randn(D, generator=g, device="cuda") * 0.2 + 1).to(dtype)
        self.cs = jt.rope_table(600, D)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_steps_and_tokens(dtype):
    m = Model(dtype)
    rng = np.random.default_rng(3)
    nseq, N, W, max_tree = 3, 6, 3, 40
    prompts = [rng.integers(0, V, n).tolist() for n in (150, 37, 1)]
    max_pages = 24
    table = torch.tensor(rng.permutation(nseq * max_pages).reshape(nseq, max_pages), **I32)
    k = torch.full((LAYERS, nseq * max_pages, PAGE, Hkv, D), float("nan"), dtype=dtype, device="cuda")
    v = k.clone()
    L = torch.zeros(nseq, **I32)
    ws_a = jt.workspace(256)
    ws_c = jt.workspace(jt.jt_workspace_size(jt.JT_OP_KV_COMMIT, nseq))
    ws_q = jt.workspace(jt.jt_workspace_size(jt.JT_OP_CHUNK_ATTN, nseq, 0, 0, 0, 400, Hq, Hkv, D, max_pages, 100))
    history = [[] for _ in range(nseq)]

    def append(tokens, off, depth=None):
        qs = []
        for layer in range(LAYERS):
            qs.append(jt.jt_qkv_append(m.emb[layer][tokens.long()], Hq, k[layer], v[layer], table, L, off, q_weight=m.qw,
                                       k_weight=m.kw, cos_sin=m.cs, depth=depth, ws=ws_a))
        jt.jt_check(ws_a)
        return qs

    def cache_holds_the_history():
        """Keys and values of every accepted token, each at its own position."""
        for b, h in enumerate(history):
            assert int(L[b]) == len(h)
            page, row = slots(table, b, 0, len(h))
            tok, pos = torch.tensor(h, device="cuda"), torch.arange(len(h), device="cuda")
            for layer in range(LAYERS):
                x = m.emb[layer][tok].view(len(h), Hq + 2 * Hkv, D)
                y, mag = heads_ref(x[:, Hq:Hq + Hkv], m.kw, 1e-6, m.cs, pos, False)
                err = (k[layer][page, row].double() - y).abs()
                tol = (D + 12) * 2.0 ** -24
                assert bool((err <= tol * mag + HALF_STEP[dtype] * (y.abs() + tol * mag)).all())
                assert torch.equal(bits(v[layer][page, row]), bits(x[:, Hq + Hkv:]))

    def attend(tokens, new):
        """Append new tokens (in order) and check their attention in every layer."""
        off = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **I32)
        qs = append(tokens, off)
        for layer, q in enumerate(qs):
            out, lse = jt.jt_chunk_attn_paged(q, k[layer], v[layer], table, L, off, max_chunk=max(new), ws=ws_q)
            jt.jt_check(ws_q)
            s = dict(q=q, k=k[layer], v=v[layer], table=table, prefix=L.tolist(), new=new)
            ref, rlse, A, S = chunk_ref(s)
            e_out, e_lse = chunk_bounds(s, ref, A, S)
            assert bool(((out.double() - ref).abs() <= e_out).all()) and bool(((lse.double() - rlse).abs() <= e_lse).all())

    # prompts, two ragged chunks each (the second request's second chunk is empty)
    for part in ([100, 37, 0], [50, 0, 1]):
        toks = []
        for b in range(nseq):
            at = len(history[b])
            toks += prompts[b][at:at + part[b]]
            history[b] += prompts[b][at:at + part[b]]
        attend(torch.tensor(toks, **I32), part)
        L += torch.tensor(part, **I32)
    cache_holds_the_history()

    root = torch.tensor(rng.integers(0, V, nseq), **I32)
    for step in range(4):
        budgets = [int(x) for x in rng.integers(5, max_tree, nseq)]
        off = torch.tensor(np.concatenate([[0], np.cumsum(budgets)]), **I32)
        total = sum(budgets)
        draft = torch.randn(nseq, N, V, device="cuda") * 2
        parent, token, depth, anc = jt.jt_tree_build(draft, root, off, W, total_nodes=total)
        qs = append(token, off, depth)
        target = torch.randn(total, V, device="cuda")
        seq_of = torch.repeat_interleave(torch.arange(nseq, device="cuda"), torch.tensor(budgets, device="cuda"))
        rows = (off[seq_of].long() + parent.long()).clamp(min=0)
        # most parents prefer one of their children: paths of several nodes are accepted
        pick = torch.rand(total, device="cuda") < 0.8
        nonroot = (parent >= 0) & pick
        target[rows[nonroot], token[nonroot].long()] += 20.0
        for layer, q in enumerate(qs):
            out, _ = jt.jt_tree_attn_paged(q, k[layer], v[layer], table, L, off, anc, max_tree=max_tree)
            assert bool(torch.isfinite(out).all())
        acc, path, bonus = jt.jt_verify_accept(target, parent, token, off, N)
        for b in range(nseq):
            a = int(acc[b])
            nodes = (off[b] + path[b, :a + 1]).long()
            history[b] += token[nodes].tolist()
        jt.jt_kv_commit(k, v, table, L, off, acc, path, new_prefix=L, ws=ws_c)
        jt.jt_check(ws_c)
        cache_holds_the_history()
        root = bonus
        if step == 1:  # a plain step in between: the bonus tokens alone
            for b in range(nseq):
                history[b].append(int(root[b]))
            attend(root, [1] * nseq)
            L += 1
            cache_holds_the_history()
            root = torch.tensor(rng.integers(0, V, nseq), **I32)
    assert max(len(h) for h in history) > 155  # trees were accepted in part
