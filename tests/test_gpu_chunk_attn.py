"""jt_chunk_attn_paged against the 64-bit form: every row of every case, within
bounds counted from the roundings (kv_util.chunk_bounds); spare pages and the
slots past each sequence's last token hold NaN in every case."""
import math
import random

import pytest
import torch

import tree_speculative_decoding_jt_gb300 as jt
from kv_util import batch, chunk_bounds, chunk_ref, slots

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def run(s, ws=None, **kw):
    ws = workspace(s) if ws is None else ws
    out, lse = jt.jt_chunk_attn_paged(s["q"], s["k"], s["v"], s["table"], s["L"], s["off"], max_chunk=max(s["new"]),
                                      ws=ws, **kw)
    jt.jt_check(ws)
    return out, lse


def workspace(*batches):
    return jt.workspace(max(jt.jt_workspace_size(
        jt.JT_OP_CHUNK_ATTN, len(s["new"]), 0, 0, 0, s["total"], s["q"].shape[1], s["k"].shape[2], s["q"].shape[2],
        s["table"].shape[1], max(s["new"])) for s in batches))


def check(s, out, lse, scale=None):
    ref, rlse, A, S = chunk_ref(s, scale)
    n = sum(s["new"])
    e_out, e_lse = chunk_bounds(s, ref, A, S)
    d = (out[:n].double() - ref[:n]).abs()
    assert bool((d <= e_out[:n]).all()), (d - e_out[:n]).max().item()
    d = (lse[:n].double() - rlse[:n]).abs()
    assert bool((d <= e_lse[:n]).all()), (d - e_lse[:n]).max().item()


CASES = [
    # prefix lengths, new tokens, Hq, Hkv, D
    ([0], [1], 4, 1, 128),                                 # one key
    ([1, 15, 16, 17], [1, 1, 1, 1], 32, 8, 128),
    ([127, 128, 129, 126], [1, 1, 1, 2], 32, 8, 128),
    ([4096], [1], 32, 8, 128),                             # one token: units cut into many pieces
    ([5000, 0, 777], [1, 300, 0], 32, 8, 128),             # tokens, a prompt and an idle sequence
    ([0, 0, 100], [0, 0, 5], 8, 8, 128),
    ([0], [512], 32, 8, 128),
    ([3, 500, 64], [31, 33, 65], 32, 8, 128),
    ([200, 3], [130, 257], 8, 8, 128),                     # G = 1
    ([64, 257], [48, 300], 16, 8, 128),                    # G = 2
    ([100, 50], [70, 43], 9, 3, 128),                      # G = 3
    ([10, 900], [60, 26], 10, 2, 128),                     # G = 5
    ([33, 1], [17, 55], 28, 4, 128),                       # G = 7
    ([100, 50], [20, 140], 64, 8, 128),                    # G = 8
    ([2000], [40], 32, 2, 128),                            # G = 16
    ([300, 7], [3, 9], 48, 1, 128),                        # G = 48
    ([40], [5], 128, 1, 128),                              # G = 128
    ([500, 33, 0], [77, 1, 129], 32, 8, 64),               # D = 64
    ([1024, 5], [1, 700], 16, 8, 64),
    ([0, 130], [300, 1], 6, 6, 64),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_matches_the_64_bit_form(case, dtype):
    prefix, new, Hq, Hkv, D = case
    if dtype == F32 and Hq // Hkv > 64:
        pytest.skip("fp32 takes Hq / Hkv up to 64")
    s = batch(1000 + CASES.index(case), prefix, new, Hq, Hkv, D, dtype)
    check(s, *run(s))


@pytest.mark.parametrize("D", [32, 96])
def test_f32_head_dims(D):
    s = batch(5, [100, 0, 65], [33, 70, 1], 12, 4, D, F32)
    check(s, *run(s))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_short_sequences(dtype):
    """Hundreds of one- to three-token sequences: many whole units per work slot."""
    prefix = [(37 * i) % 50 for i in range(300)]
    new = [(i % 4 > 0) + (i % 7 == 0) + (i % 11 == 0) for i in range(300)]
    s = batch(6, prefix, new, 8, 2, 128, dtype)
    check(s, *run(s))


def test_long_prompt():
    s = batch(7, [1000], [3000], 8, 2, 128)
    check(s, *run(s))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_running_maximum_jumps(dtype):
    """Keys of late pages scaled up in steps: the running maximum grows by more
    than 2^32 (log2 units) twice, so O is rescaled, in tiles of either parity."""
    s = batch(8, [2000, 600], [40, 130], 16, 4, 128, dtype, q_std=8.0)
    for b, L in enumerate(s["prefix"]):
        for at, f in ((L // 3, 8), (L // 3 + 128, 16), (L - 40, 32)):
            page, _ = slots(s["table"], b, at, 1)
            s["k"][page] = s["k"][page] * f
    check(s, *run(s))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_a_token_does_not_see_has_no_effect(dtype, bad):
    """Values and keys of later tokens of the same chunk that are not finite
    leave the rows before them as they are, bit for bit where no tensor-core
    tile holds them and within the bounds elsewhere; rows that see them differ."""
    s = batch(9, [200, 37], [150, 1], 8, 2, 128, dtype)
    page, row = slots(s["table"], 0, 200 + 100, 50)
    s["v"][page[7:], row[7:]] = bad
    out, lse = run(s)
    ref, rlse, A, S = chunk_ref({**s, "v": torch.nan_to_num(s["v"], 0, 0, 0), "k": s["k"]})
    e_out, e_lse = chunk_bounds(s, ref, A, S)
    rows = torch.tensor([i for i in range(151) if not 107 <= i < 150], device="cuda")
    assert bool(((out.double() - ref).abs()[rows] <= e_out[rows]).all())
    assert bool(((lse.double() - rlse).abs() <= e_lse).all())  # the scores are finite everywhere
    assert not bool(torch.isfinite(out[107:150]).any())
    s["v"] = torch.nan_to_num(s["v"], 0, 0, 0)
    s["k"][page[7:], row[7:]] = bad
    out, lse = run(s)
    assert bool(((out.double() - ref).abs()[rows] <= e_out[rows]).all())
    assert bool(((lse.double() - rlse).abs()[rows] <= e_lse[rows]).all())
    assert bool(torch.isnan(out[107:150]).all())  # a score that is not finite: NaN, as the softmax has it


def test_a_cut_unit_with_values_that_are_not_finite():
    """One token over a long prefix (pieces merged from partials) whose values hold an infinity: seen, so it shows."""
    s = batch(10, [6000], [3], 8, 2, 128)
    page, row = slots(s["table"], 0, 6001, 1)
    s["v"][page, row, 0] = math.inf
    out, _ = run(s)
    ref, _, A, S = chunk_ref({**s, "v": torch.nan_to_num(s["v"], 0, 0, 0)})
    e_out, _ = chunk_bounds(s, ref, A, S)
    assert bool(((out.double() - ref).abs()[0] <= e_out[0]).all())
    assert bool((out[1:, :4] == math.inf).all())
    assert bool(((out.double() - ref).abs()[1:, 4:] <= e_out[1:, 4:]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefix,new", [([300], [2]), ([6000], [3]), ([2000], [300])])
def test_runs_of_keys_that_are_nan(dtype, prefix, new):
    """Whole key tiles, and whole pieces of a cut unit, whose scores are all NaN, at
    the front, in the middle and at the end: output and lse of every row are NaN."""
    L = prefix[0]
    for first, count in ((0, 256), (L // 2 // 128 * 128, 128), (L // 4, L // 2), (0, L)):
        s = batch(32, prefix, new, 8, 2, 128, dtype)
        page, row = slots(s["table"], 0, first, count)
        s["k"][page, row] = math.nan
        out, lse = run(s)
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all()), (first, count)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_behind_the_last_sequence_stay(dtype):
    s = batch(11, [50, 3], [7, 20], 8, 2, 64, dtype, spare_rows=9)
    out = torch.full_like(s["q"], 5.0)
    lse = torch.full(s["q"].shape[:2], 7.0, device="cuda")
    run(s, out=out, lse=lse)
    check(s, out, lse)
    assert bool((out[27:] == 5).all()) and bool((lse[27:] == 7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_workspace_for_calls_of_every_shape_and_identical_bits(dtype):
    shapes = [batch(12, [3000], [1], 32, 8, 128, dtype), batch(13, [900, 20, 400], [200, 64, 1], 16, 8, 64, dtype),
              batch(14, [10] * 40, [1] * 40, 8, 8, 128, dtype), batch(15, [0, 2500], [600, 2], 32, 8, 128, dtype)]
    ws = workspace(*shapes)
    first = [tuple(t.clone() for t in run(s, ws)) for s in shapes]
    for _ in range(3):
        for s, (out, lse) in zip(shapes, first):
            o, l = run(s, ws)
            assert torch.equal(o, out) and torch.equal(l, lse)
    for s, (out, lse) in zip(shapes, first):
        check(s, out, lse)
    # calls of the other dtype in between leave the workspace usable
    other = batch(16, [700], [5], 8, 8, 64, F32 if dtype == BF16 else BF16)
    ws = workspace(other, *shapes)
    for s, (out, lse) in zip(shapes, first):
        run(other, ws)
        o, l = run(s, ws)
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_replayed_and_two_streams(dtype):
    """A captured call replayed after its lengths changed on the device, and two
    calls on two streams at once, each with its own workspace."""
    s = batch(17, [800, 90], [3, 40], 16, 4, 128, dtype)
    t = batch(18, [1500], [20], 16, 4, 128, dtype)
    ws, wt = workspace(s), workspace(t)
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    args = (s["q"], s["k"], s["v"], s["table"], s["L"], s["off"])
    jt.jt_chunk_attn_paged(*args, max_chunk=40, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        jt.jt_chunk_attn_paged(*args, max_chunk=40, out=out, lse=lse, ws=ws)
    for prefix in ([800, 90], [500, 33], [0, 89]):
        s["prefix"] = prefix
        s["L"].copy_(torch.tensor(prefix, dtype=torch.int32))
        out.fill_(9)
        g.replay()
        jt.jt_check(ws)
        check(s, out, lse)
    want_s, want_t = (out.clone(), lse.clone()), run(t)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            a = jt.jt_chunk_attn_paged(*args, max_chunk=40, ws=ws)
        b = jt.jt_chunk_attn_paged(t["q"], t["k"], t["v"], t["table"], t["L"], t["off"], max_chunk=20, ws=wt,
                                   stream=streams[1])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a + b, want_s + want_t))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sequences_with_contents_out_of_range_are_skipped(dtype):
    s = batch(19, [50, 60, 70], [4, 5, 6], 8, 2, 128, dtype, max_pages=8)
    ref = chunk_ref(s)
    e_out, _ = chunk_bounds(s, ref[0], ref[2], ref[3])
    ws = workspace(s)
    for L1, max_chunk in ((-1, 6), (125, 6), (1 << 30, 6), (60, 4)):  # negative, past the table, chunk above max_chunk
        L = s["L"].clone()
        L[1] = L1
        out = torch.full_like(s["q"], 3.0)
        jt.jt_chunk_attn_paged(s["q"], s["k"], s["v"], s["table"], L, s["off"], max_chunk=max_chunk, out=out, ws=ws)
        with pytest.raises(jt.JtError) as e:
            jt.jt_check(ws)
        assert e.value.status == jt.JT_ERR_INVALID
        assert bool((out[4:9] == 3).all())
        assert bool(((out.double() - ref[0]).abs()[:4] <= e_out[:4]).all())
    # offsets past the capacity
    off = s["off"].clone()
    off[3] = 40
    out = torch.full_like(s["q"], 3.0)
    jt.jt_chunk_attn_paged(s["q"], s["k"], s["v"], s["table"], s["L"], off, max_chunk=40, out=out, ws=ws)
    with pytest.raises(jt.JtError):
        jt.jt_check(ws)
    assert bool((out[9:] == 3).all())


def test_f32_page_outside_the_pool_is_flagged():
    s = batch(20, [50], [4], 8, 2, 64, F32)
    s["table"][0, 1] = s["k"].shape[0]
    ws = workspace(s)
    jt.jt_chunk_attn_paged(s["q"], s["k"], s["v"], s["table"], s["L"], s["off"], max_chunk=4, ws=ws)
    with pytest.raises(jt.JtError) as e:
        jt.jt_check(ws)
    assert e.value.status == jt.JT_ERR_INVALID


def test_scale_and_no_lse():
    s = batch(21, [300], [10], 8, 2, 128)
    out, lse = run(s, scale=0.3)
    check(s, out, lse, scale=0.3)
    out2, none = run(s, scale=0.3, with_lse=False)
    assert none is None and torch.equal(out, out2)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_past_32_bits(dtype):
    """A pool of more than 2^31 elements whose last pages hold the sequence."""
    Hkv, D = 8, 128
    pages = (1 << 31) // (16 * Hkv * D) + 200
    s = batch(22, [1000], [3], 16, Hkv, D, dtype)
    n = s["k"].shape[0]
    for name in ("k", "v"):
        pool = torch.empty((pages, 16, Hkv, D), dtype=dtype, device="cuda")
        pool[pages - n:] = s[name]
        s[name] = pool
    s["table"] = torch.where(s["table"] >= 0, s["table"] + (pages - n), s["table"])
    check(s, *run(s))
    del s
    torch.cuda.empty_cache()


def test_agrees_with_the_tree_attention_on_a_chain():
    """A chain tree is a chunk: both operators read the same cache."""
    s = batch(23, [500, 37], [64, 100], 32, 8, 128)
    anc = torch.zeros((s["total"], 8), dtype=torch.int64)
    at = 0
    for B in s["new"]:
        for i in range(B):
            for j in range(i + 1):
                anc[at + i, j // 32] |= 1 << (j % 32)
        at += B
    anc = torch.where(anc >= 1 << 31, anc - (1 << 32), anc).to(torch.int32).cuda()
    want, wl = jt.jt_tree_attn_paged(s["q"], s["k"], s["v"], s["table"], s["L"], s["off"], anc, max_tree=100)
    out, lse = run(s)
    ref, _, A, S = chunk_ref(s)
    e_out, e_lse = chunk_bounds(s, ref, A, S)
    assert bool(((out.double() - want.double()).abs() <= 2 * e_out).all())
    assert bool(((lse - wl).abs() <= 2 * e_lse).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ragged_batches_in_a_row(dtype):
    """Serving batches of chunks of 1 to 300 tokens, partly filled query tiles
    beside full ones in every work slot: no wait runs out, every row right."""
    ws = None
    for seed in range(12):
        r = random.Random(seed)
        n = r.randint(6, 20)
        s = batch(300 + seed, [r.randint(0, 3000) for _ in range(n)], [r.choice([1, r.randint(1, 300)]) for _ in range(n)],
                  16, 4, 128, dtype)
        ws = jt.workspace(1 << 27) if ws is None else ws
        first = run(s, ws)
        check(s, *first)
        for _ in range(6):
            out, lse = run(s, ws)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_batches_of_mostly_idle_sequences(dtype):
    """No new token at all; two of fifty sequences active."""
    s = batch(24, [5, 0], [0, 0], 8, 2, 128, dtype, spare_rows=3)
    s["new"] = [1, 1]  # max_chunk and workspace of a batch that could have had tokens
    out = torch.full_like(s["q"], 5.0)
    run(s, out=out)
    assert bool((out == 5).all())
    new = [0] * 50
    new[17], new[41] = 3, 70
    s = batch(25, [(7 * i) % 300 for i in range(50)], new, 8, 2, 128, dtype)
    check(s, *run(s))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shared_prefix_pages(dtype):
    """Two sequences whose tables name the same physical pages for a common prefix."""
    s = batch(26, [320, 320], [5, 40], 8, 2, 128, dtype)
    s["table"][1, :20] = s["table"][0, :20]
    check(s, *run(s))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_graphs_that_share_a_workspace_and_a_given_stream(dtype):
    """Two captured graphs with one workspace, replayed in turn; calls on a
    given stream that allocate their own workspace and outputs there."""
    a, b = batch(27, [2000], [1], 32, 8, 128, dtype), batch(28, [100, 700, 5], [200, 1, 33], 16, 4, 128, dtype)
    ws = workspace(a, b)
    want = [tuple(t.clone() for t in run(s, ws)) for s in (a, b)]
    graphs, outs = [], []
    for s in (a, b):
        out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            jt.jt_chunk_attn_paged(s["q"], s["k"], s["v"], s["table"], s["L"], s["off"], max_chunk=max(s["new"]), out=out,
                                   lse=lse, ws=ws)
        graphs.append(g)
        outs.append((out, lse))
    for _ in range(3):
        for g, got, w in zip(graphs, outs, want):
            got[0].zero_()
            g.replay()
            jt.jt_check(ws)
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = [jt.jt_chunk_attn_paged(s["q"], s["k"], s["v"], s["table"], s["L"], s["off"], max_chunk=max(s["new"]), stream=st)
           for s in (a, b, a, b)]
    torch.cuda.current_stream().wait_stream(st)
    for g, w in zip(got, want * 2):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_a_page_outside_the_pool_is_reported(dtype, D):
    """In a sequence's first, middle and last page, for a token and for a prompt; the
    other sequences' rows are right, and entries that no token sees stay unread."""
    s = batch(41, [50, 300, 0, 7], [4, 1, 200, 1], 8, 2, D, dtype, max_pages=24)
    ref, _, A, S = chunk_ref(s)
    e_out, _ = chunk_bounds(s, ref, A, S)
    ws = workspace(s)
    run(s, ws)
    table = s["table"].clone()
    for b, page in ((0, 1), (0, 3), (1, 0), (1, 18), (2, 7), (2, 12), (3, 0)):
        for bad in (-1, s["k"].shape[0], (1 << 31) - 1, -(1 << 31)):
            s["table"] = table.clone()
            s["table"][b, page] = bad
            out, _ = jt.jt_chunk_attn_paged(s["q"], s["k"], s["v"], s["table"], s["L"], s["off"], max_chunk=200, ws=ws)
            with pytest.raises(jt.JtError) as e:
                jt.jt_check(ws)
            assert e.value.status == jt.JT_ERR_INVALID
            keep = torch.ones(s["total"], dtype=torch.bool, device="cuda")
            keep[int(s["off"][b]):int(s["off"][b + 1])] = False
            assert bool(((out.double() - ref).abs()[keep] <= e_out[keep]).all())
    s["table"] = table
    check(s, *run(s, ws))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_workspace_for_prompts_serves_the_tokens_after_them(dtype):
    prompt = batch(42, [0] * 12, [300 - 7 * i for i in range(12)], 8, 2, 64, dtype, max_pages=128)
    ws = workspace(prompt)
    check(prompt, *run(prompt, ws))
    for n in (12, 3, 1):
        s = batch(43 + n, [1900] * n, [1] * n, 8, 2, 64, dtype, max_pages=128)
        check(s, *run(s, ws))


def test_a_call_without_a_workspace_takes_what_its_type_needs():
    s = batch(47, [4000] * 4, [1] * 4, 32, 8, 128)
    run(s)
    args = (s["q"], s["k"], s["v"], s["table"], s["L"], s["off"])
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out, lse = jt.jt_chunk_attn_paged(*args, max_chunk=1)
    assert torch.cuda.max_memory_allocated() - before < 32 << 20
    check(s, out, lse)


@pytest.mark.parametrize("D", [128, 64])
def test_a_probability_is_rounded_once_when_the_maximum_jumps(D):
    """Scores of 0 in the first key tile, 40 to 48 (log2 units) for a key of the
    second, 0 to 24 for a key of the third: the third tile's P is worked out before
    its warp knows of the jump and scaled afterwards.  Only that key has a value, so a
    row's error is P's rounding and the output's: two half steps of 2^-8 (and 2^-15
    for the fp32 terms: some 50 half steps of 2^-24 in the score, 2^-22 in exp2)."""
    nseq, L, B, Hq, Hkv = 40, 384, 32, 16, 4
    s = batch(60, [L] * nseq, [B] * nseq, Hq, Hkv, D)
    unit = math.log2(math.e) / math.sqrt(D)  # of a score in log2 units
    g = torch.Generator(device="cuda")
    g.manual_seed(61)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    q = torch.zeros_like(s["q"])
    q[..., 0] = (1 + 0.2 * rand(*q.shape[:2])).to(BF16)
    q[..., 1] = (24 * rand(*q.shape[:2])).to(BF16)
    s["q"] = q
    k, v = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    for b in range(nseq):
        page, row = slots(s["table"], b, 128 + 5, 1)
        k[page, row, :, 0] = 40 / unit
        page, row = slots(s["table"], b, 256 + 7, 1)
        k[page, row, :, 1] = 1 / unit
        v[page, row] = ((1 + rand(Hkv, D)) * 2.0 ** 40).to(BF16)
    s["k"], s["v"] = k, v
    out, lse = run(s)
    ref, rlse, _, _ = chunk_ref(s)
    half = 2.0 ** -8
    assert bool(((out.double() - ref).abs() <= ref * ((1 + half) ** 2 * (1 + 2.0 ** -15) - 1)).all())
    assert bool(((lse.double() - rlse).abs() <= 2.0 ** -16).all())
