"""Plain 64-bit forms of the cache operators, and seeded ragged batches for their tests."""
import math

import numpy as np
import torch

PAGE = 16
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # finfo.eps / 2


def batch(seed, prefix, new, Hq, Hkv, D, dtype=torch.bfloat16, device="cuda", spare_pages=3, spare_rows=0,
          max_pages=None, q_std=2.0, std=0.5):
    """A ragged batch over a shuffled page pool.  Spare pages and the slots past
    every sequence's last token hold NaN; unused table entries are -1."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    nseq = len(prefix)
    need = [(l + b + PAGE - 1) // PAGE for l, b in zip(prefix, new)]
    pages = sum(need) + spare_pages
    perm = rng.permutation(pages)
    table = np.full((nseq, max(max_pages or 0, max(need), 1)), -1, np.int32)
    at = 0
    for b in range(nseq):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]

    def normal(*shape, std=std):
        return (torch.randn(shape, generator=g, device=device) * std).to(dtype)

    k, v = normal(pages, PAGE, Hkv, D), normal(pages, PAGE, Hkv, D)
    for c in (k, v):
        c[torch.as_tensor(perm[at:], device=device).long()] = math.nan
        for b in range(nseq):
            used = prefix[b] + new[b]
            if used % PAGE:
                c[int(table[b, need[b] - 1]), used % PAGE:] = math.nan
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    total = int(off[-1]) + spare_rows
    i32 = dict(dtype=torch.int32, device=device)
    return dict(k=k, v=v, table=torch.tensor(table, **i32), L=torch.tensor(prefix, **i32), off=torch.tensor(off, **i32),
                q=normal(total, Hq, D, std=q_std), prefix=list(prefix), new=list(new), normal=normal, total=total)


def slots(table, b, first, count):
    t = torch.arange(first, first + count, device=table.device)
    return table[b].long()[t // PAGE], t % PAGE


def chunk_ref(s, scale=None):
    """(out, lse, A, S) in 64 bits for the rows of every sequence: A = sum p |v|
    / l, S = the largest sum |q_d k_d| scale of the row (both for the bounds)."""
    q, k, v, table = s["q"], s["k"], s["v"], s["table"]
    n, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.full((n, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    A, lse, S = out.clone(), out[..., 0].clone(), out[..., 0].clone()
    at = 0
    for b, (L, B) in enumerate(zip(s["prefix"], s["new"])):
        if B == 0:
            continue
        page, row = slots(table, b, 0, L + B)
        later = torch.arange(L + B, device=q.device) > L + torch.arange(B, device=q.device)[:, None]
        for h in range(Hkv):
            kk, vv = k[page, row, h].double(), v[page, row, h].double()
            for j in range(h * G, (h + 1) * G):
                qq = q[at:at + B, j].double()
                z = (qq @ kk.T * scale).masked_fill(later, -math.inf)
                S[at:at + B, j] = (qq.abs() @ kk.abs().T * scale).masked_fill(later, 0).amax(1)
                lse[at:at + B, j] = torch.logsumexp(z, 1)
                p = torch.exp(z - lse[at:at + B, j, None])
                out[at:at + B, j] = p @ vv
                A[at:at + B, j] = p @ vv.abs()
        at += B
    return out, lse, A, S


def chunk_bounds(s, ref, A, S):
    """Elementwise bounds on |out - ref| and |lse - ref|.

    Scores: D products summed in fp32, at most D half steps of sum |q k| (2^-23
    each, for an accumulator that truncates); exp adds 2^-22, the sum over n
    keys n half steps.  So p is off by r = 2 S D 2^-23 + 2^-22 + n 2^-24
    relative (score and normaliser); P rounded to bf16 adds its half step; O is
    a sum of n terms in fp32.  The output is rounded once more."""
    D = s["q"].shape[-1]
    n = max(l + b for l, b in zip(s["prefix"], s["new"]))
    half = HALF_STEP[s["q"].dtype]
    r = 2 * S * D * 2.0 ** -23 + 2.0 ** -22 + n * 2.0 ** -24
    p_round = half if s["q"].dtype == torch.bfloat16 else 0.0
    err = A * (r[..., None] + p_round * (1 + 2.0 ** -7) + n * 2.0 ** -23)
    return err + half * (ref.abs() + err) + 1e-30, r + 2.0 ** -20
