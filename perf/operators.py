"""The operators around the tree verify step, as they are measured.

Three operators that stand beside tree-causal attention over a paged cache:

* ``append``  jt_qkv_append: per-head RMS norm of queries and keys, position
  rotation, and the write of keys and values into the paged cache, in one pass
  over the packed projection;
* ``chunk``   jt_chunk_attn_paged: causal attention of a ragged batch of new
  tokens (one token to whole prompts) over the paged cache;
* ``commit``  jt_kv_commit: after the acceptance, the keys and values of the
  accepted path move to the slots right behind the prefix, in every layer.

``run`` computes them in elementary torch operations, or, with ``own`` set,
through the library's calls.
"""
import itertools
import math
import random

import torch

own = False
PAGE = 16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    big = dict(Hq=32, Hkv=8, D=128)
    return [
        # one generated token of one request: latency
        dict(name="append token b1", op="append", dtype="bf16", nseq=1, prefix_lo=4096, prefix_hi=4096, new_lo=1,
             new_hi=1, rot=128, interleaved=False, norm=True, tree=False, layout=1, **big),
        # the tree of a verify step: 8 requests of 256 nodes, positions by node depth
        dict(name="append tree b8 B256", op="append", dtype="bf16", nseq=8, prefix_lo=2048, prefix_hi=16384,
             new_lo=256, new_hi=256, rot=128, interleaved=False, norm=True, tree=True, layout=2, **big),
        # prompts: four ragged chunks, memory-bound
        dict(name="append prompts b4", op="append", dtype="bf16", nseq=4, prefix_lo=0, prefix_hi=4096, new_lo=4000,
             new_hi=8200, rot=128, interleaved=False, norm=True, tree=False, layout=3, **big),
        # fp32, odd head dim, half of it rotated in neighbouring pairs, no norm, ragged
        dict(name="append f32 D96", op="append", dtype="f32", nseq=7, prefix_lo=0, prefix_hi=1000, new_lo=1,
             new_hi=333, rot=48, interleaved=True, norm=False, tree=False, layout=4, Hq=12, Hkv=4, D=96),
        # one generated token of one request over 4096 cached ones: latency
        dict(name="chunk token b1 L4k", op="chunk", dtype="bf16", nseq=1, prefix_lo=4096, prefix_hi=4096, new_lo=1,
             new_hi=1, layout=5, **big),
        # one token each of 32 long requests: the cache's bandwidth
        dict(name="chunk tokens b32 L32k", op="chunk", dtype="bf16", nseq=32, prefix_lo=32768, prefix_hi=32768,
             new_lo=1, new_hi=1, layout=6, **big),
        # a serving batch: chunks of 1 to 512 tokens over ragged prefixes
        dict(name="chunk serving b16", op="chunk", dtype="bf16", nseq=16, prefix_lo=1024, prefix_hi=8192, new_lo=1,
             new_hi=512, layout=7, **big),
        # half of a long prompt behind its first half: compute
        dict(name="chunk prompt 8k on 8k", op="chunk", dtype="bf16", nseq=1, prefix_lo=8192, prefix_hi=8192,
             new_lo=8192, new_hi=8192, layout=8, **big),
        # head dim 64, odd ragged lengths from an empty cache on
        dict(name="chunk D64 ragged", op="chunk", dtype="bf16", nseq=5, prefix_lo=0, prefix_hi=2500, new_lo=1,
             new_hi=1500, layout=9, Hq=32, Hkv=8, D=64),
        # fp32
        dict(name="chunk f32 D64", op="chunk", dtype="f32", nseq=4, prefix_lo=128, prefix_hi=1500, new_lo=16,
             new_hi=512, layout=10, Hq=8, Hkv=2, D=64),
        # one request's accepted path in all layers: latency
        dict(name="commit b1 B256", op="commit", dtype="bf16", nseq=1, prefix_lo=4096, prefix_hi=4096, new_lo=256,
             new_hi=256, N=16, layers=36, layout=11, Hkv=8, D=128),
        # 32 requests' accepted paths in all layers
        dict(name="commit b32 B64", op="commit", dtype="bf16", nseq=32, prefix_lo=32768, prefix_hi=32768, new_lo=64,
             new_hi=64, N=8, layers=36, layout=12, Hkv=8, D=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["append", "chunk", "chunk", "commit"])
    c = dict(op=op, layout=rng.randrange(1 << 30), dtype="f32" if rng.random() < 0.2 else "bf16")
    f32 = c["dtype"] == "f32"
    c["D"] = rng.choice([32, 64, 96, 128] if f32 else [64, 128])
    c["Hkv"] = rng.choice([1, 2, 4, 8])
    if op == "commit":
        c.update(nseq=_log_int(rng, 1, 64), N=rng.randint(2, 16), layers=_log_int(rng, 1, 48))
        c["prefix_lo"] = rng.choice([0, rng.randint(1, 3000)])
        c["prefix_hi"] = c["prefix_lo"] + _log_int(rng, 1, 30000)
        c["new_hi"] = _log_int(rng, c["N"] + 1, 256)
        c["new_lo"] = rng.randint(c["N"] + 1, c["new_hi"])
        return c
    c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 8])
    c["nseq"] = _log_int(rng, 1, 32)
    new = _log_int(rng, 1, 8192 if not f32 else 512)
    c["new_lo"], c["new_hi"] = rng.choice([1, new, (new + 1) // 2]), new
    pre = _log_int(rng, 1, 32768 if not f32 else 4096)
    c["prefix_lo"], c["prefix_hi"] = rng.choice([0, pre, pre // 2]), pre
    if op == "append":
        c["rot"] = rng.choice([c["D"], c["D"] // 2])
        c.update(interleaved=rng.random() < 0.3, norm=rng.random() < 0.7, tree=False)
        if new <= 256:
            c["tree"] = rng.random() < 0.5
    # no dearer than the largest listed case: the padded score matrix, the
    # padded keys and the new tokens' rows
    while c["nseq"] > 1 and (
            c["nseq"] * c["Hq"] * new * (pre + new) > (4 << 30 if not f32 else 1 << 28)
            or c["nseq"] * c["Hkv"] * c["D"] * (pre + new) > (1 << 30 if not f32 else 1 << 27)
            or c["nseq"] * new * (c["Hq"] + 2 * c["Hkv"]) * c["D"] > 4 * 6144 * 8200):
        c["nseq"] -= 1
    if c["Hq"] * new * (pre + new) > 4 << 30:
        c["prefix_lo"], c["prefix_hi"] = min(c["prefix_lo"], 2048), min(pre, 2048)
    return c


def _lens(case):
    """The batch's prefix and new-token lengths, from the case alone."""
    r = random.Random(case["layout"])
    return ([r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(case["nseq"])],
            [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["nseq"])])


def _accepts(case):
    """Accepted lengths, from the case alone: 1 to N, most of them short."""
    r = random.Random(case["layout"] + 1)
    return [min(case["N"], 1 + int(r.expovariate(0.25))) for _ in range(case["nseq"])]


def _esize(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    L, B = _lens(case)
    e, D = _esize(case), case["D"]
    if case["op"] == "append":
        heads = case["Hq"] + 2 * case["Hkv"]
        return dict(bytes=2 * sum(B) * heads * D * e + sum(B) * case["rot"] * 4,
                    flops=sum(B) * (case["Hq"] + case["Hkv"]) * D * 7)
    if case["op"] == "chunk":
        keys = sum(l + b for l, b in zip(L, B))
        pairs = sum(b * l + b * (b + 1) // 2 for l, b in zip(L, B))
        return dict(bytes=2 * keys * case["Hkv"] * D * e + 2 * sum(B) * case["Hq"] * D * e + sum(B) * case["Hq"] * 4,
                    flops=4 * pairs * case["Hq"] * D)
    rows = sum(_accepts(case))
    return dict(bytes=2 * 2 * rows * case["layers"] * case["Hkv"] * D * e, flops=0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    L, B = _lens(case)
    nseq, D, Hkv = case["nseq"], case["D"], case["Hkv"]
    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(op=case["op"], prefix_len=torch.tensor(L, **i32), off=torch.tensor([0, *itertools.accumulate(B)], **i32),
             max_new=max(B), span=max(l + b for l, b in zip(L, B)))
    r = random.Random(seed)
    need = [(l + b + PAGE - 1) // PAGE for l, b in zip(L, B)]
    first = [0] * nseq
    if case["op"] == "commit":
        # only the tree's pages are touched: the prefix's pages are one spare
        # page here, so that all layers of the pool stay small
        first = [l // PAGE for l in L]
    pages = sum(n - f for n, f in zip(need, first)) + 1
    ids = list(range(1, pages))
    r.shuffle(ids)
    table = torch.zeros((nseq, max(need)), dtype=torch.int32)
    at = 0
    for b in range(nseq):
        n = need[b] - first[b]
        table[b, first[b]:need[b]] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    s["table"] = table.to(dev)

    def normal(*shape, std=0.5):
        return torch.randn(shape, generator=g, device=dev, dtype=dt).mul_(std)

    shape = (pages, PAGE, Hkv, D)
    if case["op"] == "commit":
        shape = (case["layers"],) + shape
        acc = _accepts(case)
        path = torch.full((nseq, case["N"] + 1), -1, dtype=torch.int32)
        for b in range(nseq):
            path[b, :acc[b] + 1] = torch.tensor([0] + sorted(r.sample(range(1, B[b]), acc[b])), dtype=torch.int32)
        s["accept"], s["path"] = torch.tensor(acc, **i32), path.to(dev)
        s["new_prefix"] = torch.zeros(nseq, **i32)
    s["k"], s["v"] = normal(*shape), normal(*shape)
    total = sum(B)
    if case["op"] == "append":
        Hq, rot = case["Hq"], case["rot"]
        s["Hq"], s["interleaved"] = Hq, case["interleaved"]
        s["qkv"] = normal(total, (Hq + 2 * Hkv) * D, std=1.0)
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"], s["kw"] = normal(D, std=0.1) + 1, normal(D, std=0.1) + 1
        s["cos_sin"] = _angles(max(l + b for l, b in zip(L, B)), rot, dev)
        s["depth"] = None
        if case["tree"]:
            # depths as a tree of these sizes has them: the root 0, then 1 to 16
            s["depth"] = torch.cat([torch.sort(torch.randint(1, 17, (b,), generator=g, device=dev, dtype=torch.int32)
                                               * (torch.arange(b, **i32) > 0))[0] for b in B]).to(torch.int32)
            s["depth"] = torch.minimum(s["depth"], torch.cat([torch.arange(b, **i32) for b in B]))
        s["q_out"] = torch.zeros((total, Hq, D), dtype=dt, device=dev)
    if case["op"] == "chunk":
        s["q"] = normal(total, case["Hq"], D, std=2.0)
    if own:  # the workspace that a user's program keeps from call to call
        import tree_speculative_decoding_jt_gb300 as jt

        if case["op"] == "chunk":
            s["ws"] = jt.workspace(jt.jt_workspace_size(jt.JT_OP_CHUNK_ATTN, nseq, 0, 0, 0, total, case["Hq"], Hkv, D,
                                                        table.shape[1], max(B)))
        else:
            s["ws"] = jt.workspace(256)
    return s


def _angles(positions, rot, dev):
    """cos and sin of every position's angles, [positions, rot], rounded once from 64 bits."""
    inv = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * inv[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float()


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"append": _append, "chunk": _chunk, "commit": _commit}[s["op"]](s)


def _run_own(s):
    import tree_speculative_decoding_jt_gb300 as jt

    if s["op"] == "append":
        q = jt.jt_qkv_append(s["qkv"], s["Hq"], s["k"], s["v"], s["table"], s["prefix_len"], s["off"],
                             q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, cos_sin=s["cos_sin"],
                             interleaved=s["interleaved"], depth=s["depth"], q_out=s["q_out"], ws=s["ws"])
        return dict(q=q, k=s["k"], v=s["v"])
    if s["op"] == "chunk":
        out, lse = jt.jt_chunk_attn_paged(s["q"], s["k"], s["v"], s["table"], s["prefix_len"], s["off"],
                                          max_chunk=s["max_new"], ws=s["ws"])
        return dict(out=out, lse=lse)
    n = jt.jt_kv_commit(s["k"], s["v"], s["table"], s["prefix_len"], s["off"], s["accept"], s["path"],
                        new_prefix=s["new_prefix"], ws=s["ws"])
    return dict(k=s["k"], v=s["v"], prefix=n)


def _rows(s, n):
    """Sequence and place in it of each of the batch's n new tokens."""
    i = torch.arange(n, dtype=torch.int32, device=s["off"].device)
    seq = torch.bucketize(i, s["off"][1:], right=True)
    return seq, i - s["off"][seq]


def _append(s):
    n, Hq, D = s["qkv"].shape[0], s["Hq"], s["k"].shape[-1]
    Hkv = s["k"].shape[-2]
    seq, local = _rows(s, n)
    pos = (s["prefix_len"][seq] + (local if s["depth"] is None else s["depth"])).long()
    x = s["qkv"].float().view(n, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    q, k = (_rotate(_norm(t, w), s["cos_sin"][pos], s["interleaved"]) for t, w in ((q, s["qw"]), (k, s["kw"])))
    slot = (s["prefix_len"][seq] + local).long()
    page = s["table"][seq, slot // PAGE].long()
    s["k"][page, slot % PAGE] = k.to(s["k"].dtype)
    s["v"][page, slot % PAGE] = v.to(s["v"].dtype)
    s["q_out"].copy_(q)
    return dict(q=s["q_out"], k=s["k"], v=s["v"])


def _norm(x, w):
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.to(x.dtype)


def _rotate(x, cs, interleaved):
    h = cs.shape[1] // 2
    cos, sin = cs[:, None, :h], cs[:, None, h:]
    x = x.clone()
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    a0, b0 = a.clone(), b.clone()
    a.copy_(a0 * cos - b0 * sin)
    b.copy_(b0 * cos + a0 * sin)
    return x


def _chunk(s):
    q, off, L = s["q"], s["off"].long(), s["prefix_len"].long()
    n, Hq, D = q.shape
    Hkv, nseq, C = s["k"].shape[2], len(L), s["max_new"]
    G, dev = Hq // Hkv, q.device
    S = s["table"].shape[1] * PAGE
    k, v = (c[s["table"].long()].reshape(nseq, S, Hkv, D).permute(0, 2, 1, 3).float() for c in (s["k"], s["v"]))
    i = torch.arange(C, device=dev)
    rows = (off[:-1, None] + i).clamp(max=n - 1)  # [nseq, C], past a sequence's end: any row
    qp = q[rows].view(nseq, C, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(nseq, Hkv, G * C, D).float()
    z = torch.matmul(qp, k.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(nseq, Hkv, G, C, S)
    hidden = torch.arange(S, device=dev) > (L[:, None, None] + i[:, None])  # [nseq, C, S]
    z.masked_fill_(hidden[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    z.sub_(m).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(nseq, Hkv, G * C, S), v).view(nseq, Hkv, G, C, D) / total
    lse = (m + total.log()).squeeze(-1)
    seq, local = _rows(s, n)
    seq, local = seq.long(), local.long()
    return dict(out=o.permute(0, 3, 1, 2, 4)[seq, local].reshape(n, Hq, D).to(q.dtype),
                lse=lse.permute(0, 3, 1, 2)[seq, local].reshape(n, Hq))


def _commit(s):
    acc, L = s["accept"].long(), s["prefix_len"].long()
    nseq, width = s["path"].shape
    d = torch.arange(width, device=acc.device)
    # steps behind the accepted path move slot L (the root's) onto itself
    take = torch.where(d <= acc[:, None], s["path"].long(), 0)
    to = torch.where(d <= acc[:, None], d, 0)
    b = torch.arange(nseq, device=acc.device)[:, None]
    src, dst = L[:, None] + take, L[:, None] + to
    sp, dp = s["table"][b, src // PAGE].long(), s["table"][b, dst // PAGE].long()
    s["k"][:, dp, dst % PAGE] = s["k"][:, sp, src % PAGE]
    s["v"][:, dp, dst % PAGE] = s["v"][:, sp, src % PAGE]
    s["new_prefix"].copy_(L + acc + 1)
    return dict(k=s["k"], v=s["v"], prefix=s["new_prefix"])


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits, one sequence at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    off, L = s["off"].tolist(), s["prefix_len"].tolist()
    table = s["table"].long()

    def slots(b, first, count):
        t = torch.arange(first, first + count, device=table.device)
        return table[b, t // PAGE], t % PAGE

    if case["op"] == "commit":
        k, v = s["k"].clone(), s["v"].clone()
        acc, path = s["accept"].tolist(), s["path"].long()
        for b in range(case["nseq"]):
            src = L[b] + path[b, :acc[b] + 1]
            dp, dr = slots(b, L[b], acc[b] + 1)
            k[:, dp, dr] = s["k"][:, table[b, src // PAGE], src % PAGE]
            v[:, dp, dr] = s["v"][:, table[b, src // PAGE], src % PAGE]
        return dict(k=k, v=v, prefix=torch.tensor([l + a + 1 for l, a in zip(L, acc)], dtype=torch.int32))
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "append":
        k, v = s["k"].double(), s["v"].double()
        out = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=table.device)
        half = case["rot"] // 2
        x = torch.arange(case["rot"], device=table.device)
        # element x of the rotated part: its partner, its angle and the sign of its sine
        if case["interleaved"]:
            partner, angle, sign = x ^ 1, x // 2, torch.where(x % 2 == 0, -1.0, 1.0).double()
        else:
            partner, angle, sign = (x + half) % (2 * half), x % half, torch.where(x < half, -1.0, 1.0).double()
        for b in range(case["nseq"]):
            lo, hi = off[b], off[b + 1]
            rows = s["qkv"][lo:hi].double().view(hi - lo, Hq + 2 * Hkv, D)
            at = torch.arange(hi - lo, device=table.device) if s["depth"] is None else s["depth"][lo:hi].long()
            cs = s["cos_sin"][L[b] + at].double()
            cos, sin = cs[:, :half][:, angle][:, None], cs[:, half:][:, angle][:, None] * sign
            both = []
            for h0, h1, w in ((0, Hq, s["qw"]), (Hq, Hq + Hkv, s["kw"])):
                y = rows[:, h0:h1]
                if w is not None:
                    y = y / ((y * y).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
                r = y[..., :2 * half]
                both.append(torch.cat([r * cos + r[..., partner] * sin, y[..., 2 * half:]], -1))
            out[lo:hi] = both[0]
            page, row = slots(b, L[b], hi - lo)
            k[page, row], v[page, row] = both[1], rows[:, Hq + Hkv:]
        return dict(q=out, k=k, v=v)
    pairs = sum((l + e - a) * (e - a) for l, a, e in zip(L, off, off[1:])) * Hq
    if pairs * D > 1 << 41:
        return None
    n, G = off[-1], Hq // Hkv
    out = torch.empty((n, Hq, D), dtype=torch.float64, device=table.device)
    lse = torch.empty((n, Hq), dtype=torch.float64, device=table.device)
    for b in range(case["nseq"]):
        lo, hi = off[b], off[b + 1]
        S = L[b] + hi - lo
        page, row = slots(b, 0, S)
        later = torch.arange(S, device=table.device) > L[b] + torch.arange(hi - lo, device=table.device)[:, None]
        for h in range(Hkv):
            k, v = s["k"][page, row, h].double(), s["v"][page, row, h].double()
            for j in range(h * G, (h + 1) * G):
                z = s["q"][lo:hi, j].double() @ k.T / math.sqrt(D)
                z.masked_fill_(later, -math.inf)
                lse[lo:hi, j] = torch.logsumexp(z, 1)
                out[lo:hi, j] = z.sub_(lse[lo:hi, j, None]).exp_() @ v
    return dict(out=out, lse=lse)
