"""Host-side checks of jt_qkv_append, jt_chunk_attn_paged and jt_kv_commit: what
they refuse, before anything is enqueued (no GPU; the pointers are never
dereferenced), and their workspace sizes."""
import ctypes

import pytest

import tree_speculative_decoding_jt_gb300 as jt
from tree_speculative_decoding_jt_gb300 import binding

A, B, C = (ctypes.c_void_p(4096 * i) for i in (1, 2, 3))
ODD = ctypes.c_void_p(4096 + 8)
INVALID, UNSUPPORTED, WORKSPACE = jt.JT_ERR_INVALID, jt.JT_ERR_UNSUPPORTED, jt.JT_ERR_WORKSPACE


OPS = dict(jt_qkv_append=jt.JT_OP_QKV_APPEND, jt_chunk_attn_paged=jt.JT_OP_CHUNK_ATTN, jt_kv_commit=jt.JT_OP_KV_COMMIT)


def call(name, defaults, **change):
    """The entry point's status, and the same through jt_call's packed arguments."""
    assert set(change) <= set(defaults), change
    args = list({**defaults, **change}.values())
    rc = getattr(jt.load(), name)(*args)
    s = binding._PACK[OPS[name]]
    packed = s.pack(*((a.value if isinstance(a, ctypes.c_void_p) else a or 0) for a in args))
    assert jt.load().jt_call(OPS[name], packed, s.size) == rc
    return rc


def test_packed_calls_of_another_size_or_operator_are_refused():
    s = binding._PACK[jt.JT_OP_KV_COMMIT]
    lib = jt.load()
    assert lib.jt_call(jt.JT_OP_KV_COMMIT, bytes(s.size), s.size - 8) == jt.JT_ERR_INVALID
    assert lib.jt_call(jt.JT_OP_KV_COMMIT, None, s.size) == jt.JT_ERR_INVALID
    assert lib.jt_call(jt.JT_OP_TREE_ATTN, bytes(s.size), s.size) == jt.JT_ERR_INVALID


APPEND = dict(qkv=A, dtype=1, row_stride=6144, q_weight=None, k_weight=None, eps=1e-6, cos_sin=A, max_pos=100,
              rot_dim=128, interleaved=0, depth=None, block_table=A, max_pages=4, num_pages=9, prefix_len=A, tree_off=A,
              nseq=2, total=5, Hq=32, Hkv=8, D=128, page_size=16, q_out=A, k_cache=A, v_cache=A, ws=A, ws_bytes=0,
              stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(qkv=None), INVALID), (dict(q_out=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(block_table=None), INVALID), (dict(prefix_len=None), INVALID), (dict(tree_off=None), INVALID),
    (dict(cos_sin=None), INVALID), (dict(max_pos=0), INVALID), (dict(row_stride=6136), INVALID),
    (dict(row_stride=6148), INVALID), (dict(qkv=ODD), INVALID), (dict(k_weight=ODD), INVALID), (dict(cos_sin=ODD), INVALID),
    (dict(q_out=ODD), INVALID), (dict(v_cache=ODD), INVALID), (dict(nseq=0), INVALID), (dict(nseq=65536), INVALID),
    (dict(total=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hkv=0), INVALID), (dict(page_size=32), INVALID),
    (dict(dtype=2), INVALID), (dict(rot_dim=144), INVALID), (dict(rot_dim=-16), INVALID), (dict(interleaved=2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(D=96, rot_dim=96), UNSUPPORTED), (dict(rot_dim=120), UNSUPPORTED), (dict(dtype=0, D=48), INVALID),
    (dict(dtype=0, D=48, rot_dim=8), UNSUPPORTED), (dict(dtype=0, rot_dim=12), UNSUPPORTED),
    (dict(), WORKSPACE), (dict(ws=None, ws_bytes=256), WORKSPACE), (dict(ws=ODD, ws_bytes=256), WORKSPACE),
    (dict(total=0), jt.JT_OK), (dict(total=0, qkv=None, q_out=None), jt.JT_OK),
])
def test_append_refusals(change, status):
    assert call("jt_qkv_append", APPEND, **change) == status


CHUNK = dict(q=A, k_cache=A, v_cache=A, dtype=1, block_table=A, max_pages=4, num_pages=9, prefix_len=A, chunk_off=A,
             nseq=2, total=5, max_chunk=4, Hq=32, Hkv=8, D=128, page_size=16, scale=0.1, out=A, lse=None, ws=A,
             ws_bytes=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(out=None), INVALID),
    (dict(block_table=None), INVALID), (dict(prefix_len=None), INVALID), (dict(chunk_off=None), INVALID),
    (dict(q=ODD), INVALID), (dict(out=ODD), INVALID), (dict(k_cache=ODD), INVALID), (dict(nseq=0), INVALID),
    (dict(nseq=65536), INVALID), (dict(total=-1), INVALID), (dict(max_chunk=0), INVALID), (dict(Hq=33), INVALID),
    (dict(Hkv=0), INVALID), (dict(page_size=8), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-0.1), INVALID), (dict(dtype=3), INVALID),
    (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(dtype=0, D=80), UNSUPPORTED), (dict(Hq=129, Hkv=1), UNSUPPORTED), (dict(dtype=0, Hq=65, Hkv=1), UNSUPPORTED),
    (dict(dtype=0, nseq=65535, Hq=64, Hkv=64, max_chunk=1 << 30), UNSUPPORTED),
    (dict(), WORKSPACE), (dict(dtype=0), WORKSPACE), (dict(ws=None, ws_bytes=1 << 30), WORKSPACE),
    (dict(ws=ODD, ws_bytes=1 << 30), WORKSPACE), (dict(total=0), jt.JT_OK), (dict(total=0, q=None, out=None), jt.JT_OK),
])
def test_chunk_refusals(change, status):
    assert call("jt_chunk_attn_paged", CHUNK, **change) == status


COMMIT = dict(k_cache=A, v_cache=A, dtype=1, layers=2, layer_stride=9 * 16 * 8 * 128, block_table=A, max_pages=4,
              num_pages=9, prefix_len=A, tree_off=A, accept_len=A, path=A, nseq=2, N=8, Hkv=8, D=128, page_size=16,
              new_prefix=B, ws=C, ws_bytes=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(block_table=None), INVALID),
    (dict(prefix_len=None), INVALID), (dict(tree_off=None), INVALID), (dict(accept_len=None), INVALID),
    (dict(path=None), INVALID), (dict(new_prefix=None), INVALID), (dict(k_cache=ODD), INVALID), (dict(nseq=0), INVALID),
    (dict(nseq=65536), INVALID), (dict(N=-1), INVALID), (dict(N=257), INVALID), (dict(layers=0), INVALID),
    (dict(layer_stride=9 * 16 * 8 * 128 - 8), INVALID), (dict(layer_stride=9 * 16 * 8 * 128 + 4), INVALID),
    (dict(page_size=64), INVALID), (dict(dtype=5), INVALID), (dict(Hkv=0), INVALID), (dict(D=0), INVALID),
    (dict(new_prefix=ctypes.c_void_p(4096 + 4)), INVALID),  # overlaps prefix_len in part
    (dict(Hkv=1, D=4, layers=1), UNSUPPORTED), (dict(Hkv=3, D=7, layers=1, dtype=0), UNSUPPORTED),
    (dict(), WORKSPACE), (dict(new_prefix=A, ws_bytes=256), WORKSPACE), (dict(ws=None, ws_bytes=4096), WORKSPACE),
])
def test_commit_refusals(change, status):
    assert call("jt_kv_commit", COMMIT, **change) == status


W = ctypes.c_void_p(1 << 40)  # a workspace far from the arrays


@pytest.mark.parametrize("a,b", [("qkv", "q_out"), ("qkv", "k_cache"), ("qkv", "v_cache"), ("q_out", "k_cache"),
                                 ("q_out", "v_cache"), ("k_cache", "v_cache")])
@pytest.mark.parametrize("shift", [0, 16])
def test_append_refuses_arrays_that_overlap(a, b, shift):
    apart = {n: ctypes.c_void_p((i + 1) << 32) for i, n in enumerate(("qkv", "q_out", "k_cache", "v_cache"))}
    apart[b] = ctypes.c_void_p(apart[a].value + shift)
    assert call("jt_qkv_append", APPEND, **apart, ws=W, ws_bytes=256) == INVALID


@pytest.mark.parametrize("dtype,shift", [(1, 0), (1, 5 * 32 * 128 * 2 - 16), (0, 0), (0, 5 * 32 * 128 * 4 - 16)])
def test_chunk_refuses_an_output_over_its_queries(dtype, shift):
    out = ctypes.c_void_p(A.value + shift)
    assert call("jt_chunk_attn_paged", CHUNK, dtype=dtype, out=out, ws=W, ws_bytes=1 << 34) == INVALID


def test_commit_refuses_one_cache_for_keys_and_values():
    assert call("jt_kv_commit", COMMIT, ws=W, ws_bytes=1 << 20) == INVALID


def test_a_longest_chunk_of_any_int_has_a_workspace_size():
    size = jt.jt_workspace_size
    big = size(jt.JT_OP_CHUNK_ATTN, 1, 0, 0, 0, 5, 1, 1, 64, 4, (1 << 31) - 1)
    assert big >= 4096


def test_a_stream_of_another_device_is_refused(monkeypatch):
    class Other:
        device_index = 1

    monkeypatch.setattr(binding, "_device_of", lambda objs, idx, where: 0)
    for fn in (jt.jt_qkv_append, jt.jt_chunk_attn_paged, jt.jt_kv_commit):
        with pytest.raises(ValueError, match="stream on cuda:1"):
            fn(None, stream=Other())


def test_workspace_sizes():
    size = jt.jt_workspace_size
    assert size(jt.JT_OP_QKV_APPEND) == 256
    assert size(jt.JT_OP_KV_COMMIT, 1) == 512 and size(jt.JT_OP_KV_COMMIT, 65) == 768
    assert size(jt.JT_OP_KV_COMMIT, 0) == 0
    assert size(jt.JT_OP_CHUNK_ATTN, 2, 0, 0, 0, 5, 32, 8, 128, 4, 4) > 4096
    assert size(jt.JT_OP_CHUNK_ATTN, 2, 0, 0, 0, 5, 33, 8, 128, 4, 4) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import torch

    z = torch.zeros
    i32 = dict(dtype=torch.int32)
    k = z(3, 16, 2, 64)
    with pytest.raises(ValueError):
        jt.jt_qkv_append(z(4, 8 * 64), 4, k, k, z(1, 2, **i32), z(1, **i32), z(2, **i32))
    with pytest.raises(ValueError):
        jt.jt_chunk_attn_paged(z(4, 4, 64), k, k, z(1, 2, **i32), z(1, **i32), z(2, **i32), max_chunk=4)
    with pytest.raises(ValueError):
        jt.jt_kv_commit(k, k, z(1, 2, **i32), z(1, **i32), z(2, **i32), z(1, **i32), z(1, 3, **i32))
    with pytest.raises(TypeError):
        jt.jt_chunk_attn_paged(z(4, 4, 64).half(), k, k, z(1, 2, **i32), z(1, **i32), z(2, **i32), max_chunk=4)


def test_rope_table():
    import math

    t = jt.rope_table(1001, 16, theta=1e4, device="cpu")
    assert t.shape == (1001, 16)
    for pos in (0, 1, 1000):
        for j in range(8):
            a = pos * 1e4 ** (-2 * j / 16)
            assert abs(t[pos, j].item() - math.cos(a)) <= 2 ** -24 and abs(t[pos, 8 + j].item() - math.sin(a)) <= 2 ** -24


SIZES = [(Hq, Hkv, D) for Hq, Hkv in ((32, 8), (8, 2), (64, 1), (128, 1), (6, 6)) for D in (32, 64, 96, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", SIZES)
def test_chunk_workspace_size_does_not_fall_when_sizes_grow(Hq, Hkv, D):
    def size(nseq, pages, chunk):
        return jt.jt_workspace_size(jt.JT_OP_CHUNK_ATTN, nseq, 0, 0, 0, nseq * chunk, Hq, Hkv, D, pages, chunk)

    seqs, tables, chunks = (1, 2, 3, 7, 32, 100, 1000, 65535), (1, 2, 31, 32, 64, 512, 1 << 20), (1, 2, 16, 65, 512, 8192)
    for n, n2 in zip(seqs, seqs[1:] + seqs[-1:]):
        for p, p2 in zip(tables, tables[1:] + tables[-1:]):
            for c, c2 in zip(chunks, chunks[1:] + chunks[-1:]):
                at = size(n, p, c)
                assert at <= size(n2, p, c) and at <= size(n, p2, c) and at <= size(n, p, c2), (n, p, c)


@pytest.mark.parametrize("dtype", [0, 1])
def test_a_chunk_workspace_serves_smaller_calls(dtype):
    """A workspace for the most sequences, pages and tokens is accepted by every
    smaller call (an output over its queries is refused after the workspace has been
    accepted, so nothing is enqueued)."""
    for nseq, pages, chunk in ((32, 512, 512), (8, 64, 8192), (300, 2048, 33)):
        have = jt.jt_workspace_size(jt.JT_OP_CHUNK_ATTN, nseq, 0, 0, 0, 99, 32, 8, 128, pages, chunk)
        for n in (1, 2, nseq // 2, nseq):
            for p in (1, 32, pages):
                for c in (1, 5, chunk):
                    got = call("jt_chunk_attn_paged", CHUNK, dtype=dtype, nseq=n, max_pages=p, max_chunk=c, out=A, ws=W,
                               ws_bytes=have)
                    assert got == INVALID, (n, p, c)
    if dtype == 1:  # bf16 needs the size for one page
        small = jt.jt_workspace_size(jt.JT_OP_CHUNK_ATTN, 4, 0, 0, 0, 4, 32, 8, 128, 1, 1)
        assert call("jt_chunk_attn_paged", CHUNK, nseq=4, max_pages=512, max_chunk=1, out=A, ws=W, ws_bytes=small) == INVALID


POOL = 9 * 16 * 8 * 128 * 2  # bytes of one layer of COMMIT


def far(**at):
    """COMMIT's arrays, each far from the others, and a workspace that is enough."""
    names = ("k_cache", "v_cache", "block_table", "prefix_len", "tree_off", "accept_len", "path", "new_prefix")
    apart = {n: ctypes.c_void_p((i + 1) << 32) for i, n in enumerate(names)}
    return dict(apart, ws=W, ws_bytes=1 << 20, **{n: ctypes.c_void_p(apart[m].value + shift) for n, (m, shift) in at.items()})


@pytest.mark.parametrize("name,size", [("prefix_len", 8), ("accept_len", 8), ("tree_off", 12), ("path", 2 * 9 * 4),
                                       ("block_table", 2 * 4 * 4)])
def test_commit_refuses_new_lengths_over_what_it_reads(name, size):
    """The CTAs of one cache write the new lengths while those of the others may still read."""
    for shift in (-4, 4, size - 4) + ((0,) if name != "prefix_len" else ()):
        assert call("jt_kv_commit", COMMIT, **far(new_prefix=(name, shift))) == INVALID, shift


@pytest.mark.parametrize("layers,stride,shift", [
    (1, POOL, 0), (1, POOL, 16), (1, POOL, POOL - 16), (1, POOL, 16 - POOL),
    (2, POOL, POOL), (2, POOL, -POOL), (2, POOL, 2 * POOL - 16), (2, 2 * POOL, POOL + 16), (2, 2 * POOL, 16 - POOL),
    (36, 2 * POOL, 35 * 2 * POOL), (36, 2 * POOL, 34 * 2 * POOL + POOL - 16), (36, 2 * POOL, -35 * 2 * POOL - 16),
    (36, 3 * POOL + 64, 7 * (3 * POOL + 64) + POOL - 16),
])
def test_commit_refuses_layers_of_keys_that_meet_layers_of_values(layers, stride, shift):
    """Two CTAs would move the same rows."""
    assert call("jt_kv_commit", COMMIT, **far(v_cache=("k_cache", shift)), layers=layers,
                layer_stride=stride // 2) == INVALID


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("a,b", [("out", "q"), ("out", "k_cache"), ("out", "v_cache"), ("lse", "q"), ("lse", "out"),
                                 ("lse", "k_cache"), ("lse", "v_cache")])
def test_chunk_refuses_outputs_over_what_it_reads(a, b, dtype):
    apart = {n: ctypes.c_void_p((i + 1) << 32) for i, n in enumerate(("q", "k_cache", "v_cache", "out", "lse"))}
    esize = 2 if dtype else 4
    size = dict(q=5 * 32 * 128 * esize, out=5 * 32 * 128 * esize, lse=5 * 32 * 4)
    size["k_cache"] = size["v_cache"] = 9 * 16 * 8 * 128 * esize
    for shift in (0, 16, 16 - size[a], size[b] - 16):
        apart[a] = ctypes.c_void_p(apart[b].value + shift)
        assert call("jt_chunk_attn_paged", CHUNK, **apart, dtype=dtype, ws=W, ws_bytes=1 << 34) == INVALID, shift
