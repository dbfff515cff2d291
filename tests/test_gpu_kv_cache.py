"""jt_qkv_append and jt_kv_commit against plain 64-bit / bit-exact forms."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_decoding_jt_gb300 as jt
from kv_util import HALF_STEP, PAGE, batch, slots

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def heads_ref(x, w, eps, cos_sin, pos, interleaved):
    """Norm and rotation of [n, H, D] in 64 bits, and the sum of the magnitudes
    of what each element is made of."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if cos_sin is None:
        return x, x.abs()
    h = cos_sin.shape[1] // 2
    cos, sin = cos_sin[pos, None, :h].double(), cos_sin[pos, None, h:].double()
    y, mag = x.clone(), x.abs()
    ia, ib = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
    mag[..., ia], mag[..., ib] = (a * cos).abs() + (b * sin).abs(), (b * cos).abs() + (a * sin).abs()
    return y, mag


def append_case(seed, prefix, new, Hq, Hkv, D, dtype, rot, interleaved=False, norm=True, tree=False, stride=0,
                spare_rows=0):
    s = batch(seed, prefix, new, max(Hq, 1), Hkv, D, dtype, spare_rows=spare_rows)
    n, width = s["total"], (Hq + 2 * Hkv) * D
    rows = s["normal"](n, width + stride, std=1.0)
    s.update(Hq=Hq, qkv=rows[:, :width], interleaved=interleaved, eps=1e-6, qw=None, kw=None, cs=None, depth=None)
    if norm:
        s["qw"], s["kw"] = s["normal"](D, std=0.2) + 1, s["normal"](D, std=0.2) + 1
    if rot:
        s["cs"] = jt.rope_table(max(l + b for l, b in zip(prefix, new)) + 1, rot)
    if tree:
        s["depth"] = (torch.arange(n, dtype=torch.int32, device="cuda") * 7 % 5).minimum(
            torch.cat([torch.arange(b, dtype=torch.int32) for b in new]
                      + [torch.zeros(spare_rows, dtype=torch.int32)]).cuda())
    return s


def run_append(s, ws=None, **kw):
    ws = jt.workspace(256) if ws is None else ws
    q = jt.jt_qkv_append(s["qkv"], s["Hq"], s["k"], s["v"], s["table"], s["L"], s["off"], q_weight=s["qw"],
                         k_weight=s["kw"], eps=s["eps"], cos_sin=s["cs"], interleaved=s["interleaved"],
                         depth=s["depth"], ws=ws, **kw)
    jt.jt_check(ws)
    return q


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF16 else torch.int32)


def check_append(s, q_out, k0, v0):
    """q within one rounding of the 64-bit form, k the same in its slots, v bit
    for bit, every other slot of the pool untouched."""
    Hq, Hkv, D = s["Hq"], s["k"].shape[2], s["k"].shape[3]
    n = sum(s["new"])
    x = s["qkv"][:n].reshape(n, Hq + 2 * Hkv, D)
    pos, page, row = [], [], []
    at = 0
    for b, (L, B) in enumerate(zip(s["prefix"], s["new"])):
        pos.append(L + (torch.arange(B, device="cuda") if s["depth"] is None else s["depth"][at:at + B].long()))
        p, r = slots(s["table"], b, L, B)
        page.append(p), row.append(r)
        at += B
    pos, page, row = torch.cat(pos), torch.cat(page), torch.cat(row)
    half = HALF_STEP[x.dtype]
    # fp32 arithmetic: the mean of D squares, rsqrt and two products, the
    # rotation: D + 12 half steps of the magnitudes; then the output's rounding
    tol = (D + 12) * 2.0 ** -24
    for got, lo, hi, w in ((q_out, 0, Hq, s["qw"]), (s["k"][page, row], Hq, Hq + Hkv, s["kw"])):
        if hi == lo:
            continue
        y, mag = heads_ref(x[:, lo:hi], w, s["eps"], s["cs"], pos, s["interleaved"])
        err = (got[:n].double() - y).abs()
        bound = tol * mag + half * (y.abs() + tol * mag) + 1e-37
        if w is None and s["cs"] is None:
            bound = torch.zeros_like(bound)
        assert bool((err <= bound).all()), (err - bound).max().item()
    assert torch.equal(bits(s["v"][page, row]), bits(x[:, Hq + Hkv:]))
    k0[page, row], v0[page, row] = s["k"][page, row], s["v"][page, row]
    assert torch.equal(bits(s["k"]), bits(k0)) and torch.equal(bits(s["v"]), bits(v0))


APPEND = [
    # prefix, new, Hq, Hkv, D, dtype, rot, options
    ([4096], [1], 32, 8, 128, BF16, 128, {}),
    ([0], [1], 32, 8, 128, BF16, 128, {}),
    ([100, 5, 0, 31], [40, 0, 17, 1], 32, 8, 128, BF16, 128, {}),
    ([100, 5, 0, 31], [40, 0, 17, 1], 32, 8, 128, BF16, 128, dict(tree=True)),
    ([7, 300], [600, 900], 12, 4, 128, BF16, 64, dict(interleaved=True)),
    ([7, 300], [3, 9], 6, 2, 64, BF16, 32, dict(norm=False)),
    ([7, 300], [3, 9], 5, 1, 64, BF16, 64, dict(interleaved=True, stride=64)),
    ([20, 1], [33, 2], 0, 3, 128, BF16, 128, {}),                       # keys and values only
    ([20, 1], [33, 2], 4, 2, 128, BF16, 0, dict(norm=False)),            # a copy
    ([20, 1], [33, 2], 4, 2, 128, BF16, 0, {}),                          # norm without rotation
    ([20, 1], [33, 2], 7, 7, 128, BF16, 16, dict(tree=True, stride=8, spare_rows=5)),
    ([50, 3], [64, 1], 8, 2, 128, F32, 128, {}),
    ([50, 3], [64, 1], 12, 4, 96, F32, 48, dict(interleaved=True, norm=False)),
    ([50, 3], [200, 31], 12, 4, 96, F32, 96, dict(tree=True)),
    ([50, 3], [64, 1], 8, 8, 64, F32, 8, {}),
    ([50, 3], [64, 1], 3, 1, 32, F32, 32, dict(interleaved=True, stride=4)),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_matches_the_64_bit_form(case):
    prefix, new, Hq, Hkv, D, dtype, rot, opt = APPEND[case]
    s = append_case(100 + case, prefix, new, Hq, Hkv, D, dtype, rot, **opt)
    k0, v0 = s["k"].clone(), s["v"].clone()
    q_out = torch.full((s["total"], Hq, D), 3.0, dtype=dtype, device="cuda") if Hq else None
    q = run_append(s, q_out=q_out)
    check_append(s, q, k0, v0)
    if Hq:
        assert bool((q[sum(new):] == 3).all())


def test_append_many_sequences():
    """More sequences than one search step of the offsets covers, empty ones among them."""
    prefix = [(13 * i) % 40 for i in range(1100)]
    new = [i % 3 for i in range(1100)]
    s = append_case(130, prefix, new, 4, 2, 64, BF16, 64)
    k0, v0 = s["k"].clone(), s["v"].clone()
    check_append(s, run_append(s), k0, v0)


def test_append_extremes():
    """Zero rows (norm of 0 is 0), the largest and smallest numbers, NaN and
    infinity in one head leave the other heads alone."""
    s = append_case(131, [5], [4], 4, 2, 128, BF16, 128)
    x = s["qkv"].reshape(4, 8, 128)
    x[0, 0] = 0
    x[1, 1, 5] = math.nan
    x[1, 4, 7] = math.inf
    x[2, 2] = 1e-20
    x[3, 3] = 1e18
    s["qkv"] = x.reshape(4, -1)
    k0, v0 = s["k"].clone(), s["v"].clone()
    q = run_append(s)
    assert bool((q[0, 0] == 0).all())
    assert bool(torch.isnan(q[1, 1]).all()) and bool(torch.isfinite(q[1, [0, 2, 3]]).all())
    assert bool(torch.isnan(s["k"][s["table"][0, 0].long(), 6, 0]).any())
    x[1, 1], x[1, 4] = 1, 1  # the rest as ever
    s["qkv"], s["k"], s["v"] = x.reshape(4, -1), k0.clone(), v0.clone()
    check_append(s, run_append(s), k0, v0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_infinity_stays_in_its_element(dtype, interleaved):
    """An infinity among the elements that are not rotated: the norm's factor is
    0, so its head is 0 but for the NaN that infinity times 0 is, in its own place."""
    s = append_case(31, [5], [3], 4, 2, 128, dtype, 64, interleaved)
    s["qkv"] = s["qkv"].contiguous()
    x = s["qkv"].view(3, 8, 128)
    for h in (1, 5):  # a query and a key head
        x[1, h, 99] = math.inf
    q = run_append(s)
    page, row = slots(s["table"], 0, 6, 1)
    for got in (q[1, 1], s["k"][page[0], row[0], 1]):
        assert bool(torch.isnan(got[99])) and int(torch.isnan(got).sum()) == 1
        assert bool((got[:99] == 0).all()) and bool((got[100:] == 0).all())
    assert bool(torch.isfinite(q[[0, 2]]).all()) and bool(torch.isfinite(q[1, [0, 2, 3]]).all())


def test_append_skips_and_flags_what_is_out_of_range():
    s = append_case(132, [10, 20, 30], [4, 5, 6], 4, 2, 128, BF16, 128)
    ws = jt.workspace(256)
    good = (s["k"].clone(), s["v"].clone(), s["L"].clone(), s["table"].clone())

    def attempt(**change):
        s["k"], s["v"], s["L"], s["table"] = (t.clone() for t in good)
        off, cs = change.pop("off", s["off"]), change.pop("cs", s["cs"])
        for name, (at, val) in change.items():
            s[name].view(-1)[at] = val
        q = torch.full((15, 4, 128), 3.0, dtype=BF16, device="cuda")
        jt.jt_qkv_append(s["qkv"], 4, s["k"], s["v"], s["table"], s["L"], off, q_weight=s["qw"], k_weight=s["kw"],
                         cos_sin=cs, q_out=q, ws=ws)
        with pytest.raises(jt.JtError) as e:
            jt.jt_check(ws)
        assert e.value.status == jt.JT_ERR_INVALID
        return q

    P = s["table"].shape[1]
    for change in (dict(L=(1, -3)), dict(L=(1, 1 << 20)), dict(table=(P + 1, -1)), dict(table=(P + 1, 999))):
        q = attempt(**change)
        assert bool((q[4:9] == 3).all()) and not bool((q[:4] == 3).all()) and not bool((q[9:] == 3).all())
    q = attempt(cs=s["cs"][:33])  # positions 33 .. 35 of the last sequence have no angles
    assert bool((q[12:] == 3).all()) and not bool((q[:12] == 3).any(-1).all())
    q = attempt(off=torch.tensor([0, 4, 2, 15], dtype=torch.int32, device="cuda"))
    q = attempt(off=torch.tensor([0, 4, 9, 40], dtype=torch.int32, device="cuda"))
    assert bool((q[9:] == 3).all())


def test_append_captured_and_replayed():
    s = append_case(133, [40, 9], [1, 1], 8, 2, 128, BF16, 128)
    ws, q = jt.workspace(256), torch.empty((2, 8, 128), dtype=BF16, device="cuda")
    s["L"].copy_(torch.tensor([38, 7], dtype=torch.int32))
    run_append(s, ws, q_out=q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        jt.jt_qkv_append(s["qkv"], 8, s["k"], s["v"], s["table"], s["L"], s["off"], q_weight=s["qw"], k_weight=s["kw"],
                         cos_sin=s["cs"], q_out=q, ws=ws)
    for step in range(3):  # the replay reads the lengths of its time
        s["prefix"] = [38 + step, 7 + step]
        s["L"].copy_(torch.tensor(s["prefix"], dtype=torch.int32))
        s["qkv"].copy_(torch.randn_like(s["qkv"]))
        k0, v0 = s["k"].clone(), s["v"].clone()
        g.replay()
        jt.jt_check(ws)
        check_append(s, q, k0, v0)


def test_append_offsets_past_32_bits():
    Hkv, D = 8, 128
    pages = (1 << 31) // (PAGE * Hkv * D) + 200
    s = append_case(134, [30], [40], 16, Hkv, D, BF16, 128)
    n = s["k"].shape[0]
    for name in ("k", "v"):
        pool = torch.zeros((pages, PAGE, Hkv, D), dtype=BF16, device="cuda")
        pool[pages - n:] = s[name]
        s[name] = pool
    s["table"] = torch.where(s["table"] >= 0, s["table"] + (pages - n), s["table"])
    k0, v0 = s["k"].clone(), s["v"].clone()
    check_append(s, run_append(s), k0, v0)
    del s, k0, v0
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------
def commit_case(seed, prefix, new, accept, N, Hkv, D, dtype, layers, rising=None):
    s = batch(seed, prefix, new, 1, Hkv, D, dtype)
    r = np.random.default_rng(seed)
    path = np.full((len(new), N + 1), -1, np.int32)
    for b, a in enumerate(accept):
        path[b, :a + 1] = np.concatenate([[0], np.sort(r.choice(np.arange(1, new[b]), a, replace=False))])
        if rising == "chain":
            path[b, :a + 1] = np.arange(a + 1)
        if rising == "dense":  # sources that are later steps' targets
            path[b, :a + 1] = np.concatenate([[0], np.arange(new[b] - a, new[b])]) if a else [0]
    shape = s["k"].shape
    s["k"], s["v"] = s["normal"](layers, *shape), s["normal"](layers, *shape)
    s.update(accept=torch.tensor(accept, dtype=torch.int32, device="cuda"), path=torch.tensor(path, device="cuda"))
    return s


def commit_ref(s):
    k, v = s["k"].clone(), s["v"].clone()
    for b, a in enumerate(s["accept"].tolist()):
        src = s["prefix"][b] + s["path"][b, :a + 1].long()
        dp, dr = slots(s["table"], b, s["prefix"][b], a + 1)
        sp = s["table"][b].long()[src // PAGE]
        k[:, dp, dr], v[:, dp, dr] = s["k"][:, sp, src % PAGE], s["v"][:, sp, src % PAGE]
    return k, v, s["L"] + s["accept"] + 1


COMMIT = [
    ([100], [256], [5], 16, 8, 128, BF16, 36, None),
    ([0, 33, 15], [17, 64, 40], [0, 8, 3], 8, 8, 128, BF16, 3, None),
    ([7, 40], [256, 200], [64, 40], 64, 2, 64, BF16, 2, None),
    ([7, 40], [30, 20], [15, 19], 19, 2, 64, BF16, 1, "dense"),
    ([7, 40], [30, 20], [15, 19], 20, 2, 64, BF16, 1, "chain"),
    ([3, 16, 31], [12, 20, 9], [9, 1, 8], 10, 3, 32, F32, 5, "dense"),
    ([5] * 70, [9] * 70, [i % 9 for i in range(70)], 8, 1, 8, BF16, 40, None),   # 16-byte rows
    ([1, 2], [40, 50], [30, 31], 40, 16, 256, F32, 2, "dense"),                   # 16 KB rows
]


@pytest.mark.parametrize("case", range(len(COMMIT)))
@pytest.mark.parametrize("in_place", [False, True])
def test_commit_moves_the_path_bit_for_bit(case, in_place):
    prefix, new, accept, N, Hkv, D, dtype, layers, rising = COMMIT[case]
    s = commit_case(200 + case, prefix, new, accept, N, Hkv, D, dtype, layers, rising)
    k, v, n = commit_ref(s)
    ws = jt.workspace(jt.jt_workspace_size(jt.JT_OP_KV_COMMIT, len(new)))
    out = jt.jt_kv_commit(s["k"], s["v"], s["table"], s["L"], s["off"], s["accept"], s["path"],
                          new_prefix=s["L"] if in_place else None, ws=ws)
    jt.jt_check(ws)
    assert torch.equal(bits(s["k"]), bits(k)) and torch.equal(bits(s["v"]), bits(v)) and torch.equal(out, n)
    assert in_place == (out.data_ptr() == s["L"].data_ptr())


def test_commit_in_place_again_and_captured():
    """The arrival count is back at 0 after every call: the same workspace, call
    after call and in a replayed graph, single-layer caches without a layer axis."""
    s = commit_case(220, [50, 60], [40, 40], [2, 3], 8, 2, 64, BF16, 1)
    s["k"], s["v"] = s["k"][0].contiguous(), s["v"][0].contiguous()
    ws = jt.workspace(jt.jt_workspace_size(jt.JT_OP_KV_COMMIT, 2))
    args = (s["k"], s["v"], s["table"], s["L"], s["off"], s["accept"], s["path"])
    for i in range(1, 4):
        jt.jt_kv_commit(*args, new_prefix=s["L"], ws=ws)
        jt.jt_check(ws)
        assert s["L"].tolist() == [50 + 3 * i, 60 + 4 * i]
        s["L"].copy_(torch.tensor([50 + 3 * i, 60 + 4 * i], dtype=torch.int32))
    s["L"].copy_(torch.tensor([0, 1], dtype=torch.int32))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        jt.jt_kv_commit(*args, new_prefix=s["L"], ws=ws)
    for i in range(1, 4):
        g.replay()
        jt.jt_check(ws)
        assert s["L"].tolist() == [3 * i, 1 + 4 * i]


@pytest.mark.parametrize("in_place", [False, True])
def test_commit_leaves_bad_sequences_alone(in_place):
    s = commit_case(221, [50, 60, 5], [40, 40, 40], [2, 3, 4], 8, 2, 64, BF16, 2)
    k, v, n = commit_ref(s)
    ws = jt.workspace(jt.jt_workspace_size(jt.JT_OP_KV_COMMIT, 3))
    page, row = slots(s["table"], 1, 0, 100)
    k[:, page, row], v[:, page, row] = s["k"][:, page, row], s["v"][:, page, row]
    width, P = 9, s["table"].shape[1]
    start = {name: s[name].clone() for name in ("k", "v", "L", "accept", "path", "table", "off")}
    bad = [("accept", 1, -1), ("accept", 1, 9), ("path", width + 0, 1), ("path", width + 2, 0), ("path", width + 3, 40),
           ("path", width + 1, -1), ("L", 1, -5), ("L", 1, 1 << 20),
           ("table", P + 60 // PAGE, -1), ("table", P + 60 // PAGE, s["k"].shape[1])]
    for name, at, val in bad:
        for key, t in start.items():
            s[key] = t.clone()
        s[name].view(-1)[at] = val
        before = int(s["L"][1])
        out = s["L"] if in_place else torch.full((3,), before, dtype=torch.int32, device="cuda")
        jt.jt_kv_commit(s["k"], s["v"], s["table"], s["L"], s["off"], s["accept"], s["path"], new_prefix=out, ws=ws)
        with pytest.raises(jt.JtError) as e:
            jt.jt_check(ws)
        assert e.value.status == jt.JT_ERR_INVALID, (name, at, val)
        assert out.tolist() == [int(n[0]), before, int(n[2])], (name, at, val)
        assert torch.equal(bits(s["k"]), bits(k)) and torch.equal(bits(s["v"]), bits(v)), (name, at, val)


@pytest.mark.parametrize("layout", ["alternating", "apart", "split"])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit_in_pools_whose_layers_lie_apart(layout, in_place):
    """Keys and values of a layer side by side in one pool, layers with other
    tensors between them, and the halves of one pool: what lies between stays."""
    s = commit_case(230, [100, 0, 15], [64, 17, 40], [8, 0, 3], 8, 4, 64, BF16, 5)
    k, v, n = commit_ref(s)
    shape = s["k"].shape
    if layout == "alternating":
        pool = torch.zeros((5, 2) + shape[1:], dtype=BF16, device="cuda")
        kc, vc = pool[:, 0], pool[:, 1]
    elif layout == "apart":
        pool = torch.zeros((5, 3) + shape[1:], dtype=BF16, device="cuda")
        kc, vc = pool[:, 2], pool[:, 0]
    else:
        pool = torch.zeros((2,) + shape, dtype=BF16, device="cuda")
        kc, vc = pool[1], pool[0]
    kc.copy_(s["k"])
    vc.copy_(s["v"])
    ws = jt.workspace(jt.jt_workspace_size(jt.JT_OP_KV_COMMIT, 3))
    out = jt.jt_kv_commit(kc, vc, s["table"], s["L"], s["off"], s["accept"], s["path"],
                          new_prefix=s["L"] if in_place else None, ws=ws)
    jt.jt_check(ws)
    assert torch.equal(bits(kc.contiguous()), bits(k)) and torch.equal(bits(vc.contiguous()), bits(v))
    assert torch.equal(out, n)
    if layout == "apart":
        assert not bool(pool[:, 1].any())


def test_commit_refuses_layers_that_it_cannot_step_through():
    s = commit_case(231, [10], [8], [2], 4, 4, 64, BF16, 4)
    rest = (s["table"], s["L"], s["off"], s["accept"], s["path"])
    shape = s["k"].shape
    wide = torch.zeros((4, 2) + shape[1:], dtype=BF16, device="cuda")
    heads = torch.zeros(shape[:3] + (8, 64), dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="distances apart"):
        jt.jt_kv_commit(s["k"], wide[:, 0], *rest)
    for k, v in ((heads[:, :, :, :4], heads[:, :, :, 4:]), (s["k"], heads[:, :, :, :4])):
        with pytest.raises(ValueError):
            jt.jt_kv_commit(k, v, *rest)
    with pytest.raises(ValueError):
        jt.jt_kv_commit(s["k"], s["v"][:3], *rest)
    with pytest.raises(jt.JtError):  # layers that overlap
        jt.jt_kv_commit(wide[0, 0].expand(4, *shape[1:]), wide[0, 1].expand(4, *shape[1:]), *rest)
    with pytest.raises(jt.JtError):  # the same pool twice
        jt.jt_kv_commit(wide[:, 0], wide[:, 0], *rest)
