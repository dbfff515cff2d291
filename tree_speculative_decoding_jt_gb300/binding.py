"""Thin ctypes binding of libjt (include/jt.h) for torch tensors.

Argument marshalling only: every step runs in the library's CUDA kernels.
Each function takes CUDA tensors, passes their device pointers and the
current torch stream to the C entry point of the same name, and raises
``JtError`` on a non-OK status.  Workspaces and outputs are allocated with
torch when the caller does not pass them.  There is no CPU path: without a
GPU or without the built library the calls fail.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
import threading

import torch

from . import build as _build

JT_OK, JT_ERR_INVALID, JT_ERR_UNSUPPORTED, JT_ERR_CUDA, JT_ERR_TIMEOUT, JT_ERR_WORKSPACE = 0, -1, -2, -3, -4, -5
JT_DTYPE_F32, JT_DTYPE_BF16 = 0, 1
JT_RULE_GREEDY, JT_RULE_MARGIN = 0, 1
(JT_OP_TREE_BUILD, JT_OP_TREE_ATTN, JT_OP_VERIFY_ACCEPT, JT_OP_TREE_TOPW, JT_OP_TREE_BUILD_MIXED,
 JT_OP_TREE_POLICY, JT_OP_CHUNK_ATTN, JT_OP_KV_COMMIT, JT_OP_QKV_APPEND) = range(9)
JT_MAX_TREE, JT_MAX_W, JT_MAX_N, JT_PAGE_SIZE = 256, 8, 64, 16

# every symbol include/jt.h declares
EXPORTS = ("jt_workspace_size", "jt_tree_build", "jt_tree_topw", "jt_tree_expand",
           "jt_tree_attn_paged", "jt_verify_accept", "jt_check", "jt_status_str", "jt_version",
           "jt_tree_build_noalloc", "jt_verify_accept_stochastic", "jt_tree_build_mixed",
           "jt_tree_expand_capped", "jt_tree_policy", "jt_tree_build_adaptive", "jt_selftest_wait_timeout",
           "jt_qkv_append", "jt_chunk_attn_paged", "jt_kv_commit", "jt_call")

_lock = threading.Lock()
_lib = None


class PolicyParams(ctypes.Structure):
    """jt_policy_params of include/jt.h (field order and types as there)."""
    _fields_ = [("b_min", ctypes.c_int32), ("b_max", ctypes.c_int32), ("node_cap", ctypes.c_int32),
                ("w_min", ctypes.c_int32), ("n_min", ctypes.c_int32), ("n_slack", ctypes.c_int32),
                ("beta", ctypes.c_double), ("log_conf", ctypes.c_double), ("acc_thresh", ctypes.c_double)]


def policy_params(b_min=16, b_max=256, node_cap=0, w_min=2, n_min=2, n_slack=3, beta=0.25,
                  log_conf=-0.6931471805599453, acc_thresh=3.0) -> PolicyParams:
    """Policy parameters with the defaults used by the tests and bench.py."""
    return PolicyParams(b_min, b_max, node_cap, w_min, n_min, n_slack, float(beta), float(log_conf),
                        float(acc_thresh))


def policy_ceiling(params: PolicyParams, nseq: int) -> int:
    """Per-request budget ceiling of the policy (min(b_max, max(b_min,
    node_cap // nseq)) with a node cap, else b_max)."""
    if params.node_cap > 0:
        return min(params.b_max, max(params.b_min, params.node_cap // nseq))
    return params.b_max


class JtError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {jt_status_str(status)}")


def library_variant() -> str:
    """The library variant this process loads: JT_LIB_VARIANT ("" = the
    default build, "checks" = extra device-side input checks and NVTX
    ranges)."""
    return os.environ.get("JT_LIB_VARIANT", "")


def library_path() -> str:
    return _build.lib_path(library_variant())


def load(build_if_missing: bool = True):
    """Load libjt (building it with nvcc first if it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        variant = library_variant()
        path = _build.build(variant=variant) if build_if_missing else _build.lib_path(variant)
        if not os.path.exists(path):
            raise RuntimeError(f"libjt.so not found at {path}; run tree_speculative_decoding_jt_gb300.build")
        lib = ctypes.CDLL(path)
        P, i32, i64, f32, f64, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                     ctypes.c_double, ctypes.c_size_t)
        lib.jt_workspace_size.argtypes = [i32, i32, i32, i32, i64, i32, i32, i32, i32, i32, i32]
        lib.jt_workspace_size.restype = sz
        lib.jt_tree_build.argtypes = [P, P, P, i32, i32, i32, i64, i32, P, P, P, P, P, sz, P]
        lib.jt_tree_build_mixed.argtypes = [P, P, P, i32, i32, i32, i64, i32, f64, P, P, P, P, P, sz, P]
        lib.jt_tree_topw.argtypes = [P, i64, i64, i32, P, P, P, P, sz, P]
        lib.jt_tree_build_noalloc.argtypes = [P, P, P, i32, i32, i32, i64, i32, P, P, P, P, i32, P]
        lib.jt_tree_expand.argtypes = [P, P, P, P, i32, i32, i32, i32, P, P, P, P, P, sz, P]
        lib.jt_tree_expand_capped.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, P, P, P, P, P, sz, P]
        lib.jt_tree_policy.argtypes = [P, i32, i32, i32, P, ctypes.POINTER(PolicyParams), P, P, P, P, P, P,
                                       sz, P]
        lib.jt_tree_build_adaptive.argtypes = [P, P, i32, i32, i32, i64, i32, P, ctypes.POINTER(PolicyParams),
                                               P, P, P, P, P, P, P, P, P, P, sz, P]
        lib.jt_tree_attn_paged.argtypes = [P, P, P, i32, P, i32, i32, P, P, P, i32, i32, i32, i32,
                                           i32, i32, i32, f32, P, P, P, sz, P]
        lib.jt_verify_accept.argtypes = [P, P, P, P, i32, i32, i64, i32, i32, f64, P, P, P, P, sz, P]
        lib.jt_verify_accept_stochastic.argtypes = [P, P, P, P, P, i32, i32, i64, i32, P, P, P, P, P,
                                                    P, sz, P]
        lib.jt_qkv_append.argtypes = [P, i32, i64, P, P, f32, P, i32, i32, i32, P, P, i32, i32, P, P, i32, i32,
                                      i32, i32, i32, i32, P, P, P, P, sz, P]
        lib.jt_chunk_attn_paged.argtypes = [P, P, P, i32, P, i32, i32, P, P, i32, i32, i32, i32, i32, i32, i32,
                                            f32, P, P, P, sz, P]
        lib.jt_kv_commit.argtypes = [P, P, i32, i32, i64, P, i32, i32, P, P, P, P, i32, i32, i32, i32, i32, P, P,
                                     sz, P]
        lib.jt_call.argtypes = [i32, ctypes.c_char_p, sz]
        lib.jt_check.argtypes = [P, P]
        lib.jt_selftest_wait_timeout.argtypes = [P, sz, P]
        lib.jt_status_str.argtypes = [i32]
        lib.jt_status_str.restype = ctypes.c_char_p
        lib.jt_version.argtypes = []
        for name in ("jt_tree_build", "jt_tree_topw", "jt_tree_expand", "jt_tree_attn_paged",
                     "jt_verify_accept", "jt_check", "jt_version", "jt_tree_build_noalloc",
                     "jt_verify_accept_stochastic", "jt_tree_build_mixed", "jt_tree_expand_capped",
                     "jt_tree_policy", "jt_tree_build_adaptive", "jt_selftest_wait_timeout", "jt_qkv_append",
                     "jt_chunk_attn_paged", "jt_kv_commit", "jt_call"):
            getattr(lib, name).restype = i32
        _lib = lib
        return lib


def jt_status_str(status: int) -> str:
    return load().jt_status_str(int(status)).decode()


def jt_version() -> int:
    return int(load().jt_version())


def _ptr(t):
    # a plain int: every pointer argument's argtype is c_void_p
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _need(t, name, dtype, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libjt has no CPU path)")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _check(rc, where):
    if rc != JT_OK:
        raise JtError(rc, where)


def _device_of(objs, idx, where):
    """The device index of the CUDA tensors among objs (nested tuples and lists
    included), or idx when there is none; refuses a second device."""
    for o in objs:
        if isinstance(o, torch.Tensor):
            i = o.get_device()
            if i >= 0 and i != idx:
                if idx >= 0:
                    raise ValueError(f"{where}: tensors on several devices (cuda:{idx}, cuda:{i})")
                idx = i
        elif isinstance(o, (tuple, list)):
            idx = _device_of(o, idx, where)
    return idx


def _on_tensor_device(fn):
    """Run a binding call with its tensors' device current.  The library
    launches on the current device (its stream, its per-device set-up and
    fixed scratch), so a call whose tensors live on another device than the
    current one is moved there; tensors on different devices are refused."""
    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        idx = _device_of(kwargs.values(), _device_of(args, -1, fn.__name__), fn.__name__)
        if idx < 0 or idx == torch.cuda.current_device():
            return fn(*args, **kwargs)
        with torch.cuda.device(idx):
            return fn(*args, **kwargs)
    return wrapper


def jt_workspace_size(op, nseq=0, N=0, W=0, V=0, total_nodes=0, Hq=0, Hkv=0, D=0, max_pages=0,
                      max_tree=0) -> int:
    return int(load().jt_workspace_size(op, nseq, N, W, V, total_nodes, Hq, Hkv, D, max_pages,
                                        max_tree))


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zeroed device buffer usable as a libjt workspace (torch allocations
    are 256-byte aligned; the library needs the header zero before first
    use)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


@_on_tensor_device
def jt_verify_accept_stochastic(target_logits, draft_logits, parent, token, tree_off, N, u_accept,
                                u_bonus, out=None, ws=None, stream=None):
    """Temperature-1 tree acceptance by rejection sampling with the caller's
    uniforms (fp64 [total_nodes] each).  Returns (accept_len, path, bonus)."""
    lib = load()
    _need(target_logits, "target_logits", torch.float32)
    _need(draft_logits, "draft_logits", torch.float32)
    for t, n in ((parent, "parent"), (token, "token"), (tree_off, "tree_off")):
        _need(t, n, torch.int32)
    _need(u_accept, "u_accept", torch.float64)
    _need(u_bonus, "u_bonus", torch.float64)
    total, V = target_logits.shape
    nseq = tree_off.numel() - 1
    dev = target_logits.device
    if out is None:
        out = (torch.empty(nseq, dtype=torch.int32, device=dev),
               torch.empty((nseq, N + 1), dtype=torch.int32, device=dev),
               torch.empty(nseq, dtype=torch.int32, device=dev))
    acc, path, bonus = out
    if ws is None:
        ws = workspace(jt_workspace_size(JT_OP_VERIFY_ACCEPT, nseq, 0, 0, 0, total), dev)
    rc = lib.jt_verify_accept_stochastic(_ptr(target_logits), _ptr(draft_logits), _ptr(parent), _ptr(token),
                                         _ptr(tree_off), nseq, N, V, total, _ptr(u_accept), _ptr(u_bonus),
                                         _ptr(acc), _ptr(path), _ptr(bonus), _ptr(ws), ws.numel(),
                                         _stream(stream))
    _check(rc, "jt_verify_accept_stochastic")
    return acc, path, bonus


@_on_tensor_device
def jt_check(ws: torch.Tensor, stream=None) -> None:
    """Synchronise and raise if a kernel flagged a device-side error in ws."""
    _check(load().jt_check(_ptr(ws), _stream(stream)), "jt_check")


@_on_tensor_device
def jt_tree_build(draft_logits, root_token, tree_off, W, total_nodes=None, out=None, ws=None,
                  stream=None):
    """Best-first draft tree from per-depth draft logits [nseq, N, V] (fp32).

    Returns (parent, token, depth, anc) on the device."""
    lib = load()
    _need(draft_logits, "draft_logits", torch.float32)
    _need(root_token, "root_token", torch.int32)
    _need(tree_off, "tree_off", torch.int32)
    nseq, N, V = draft_logits.shape
    if total_nodes is None:
        total_nodes = int(tree_off[-1].item())
    dev = draft_logits.device
    if out is None:
        out = (torch.empty(total_nodes, dtype=torch.int32, device=dev),
               torch.empty(total_nodes, dtype=torch.int32, device=dev),
               torch.empty(total_nodes, dtype=torch.int32, device=dev),
               torch.empty((total_nodes, 8), dtype=torch.int32, device=dev))
    parent, token, depth, anc = out
    if ws is None:
        ws = workspace(jt_workspace_size(JT_OP_TREE_BUILD, nseq, N, W, V), dev)
    rc = lib.jt_tree_build(_ptr(draft_logits), _ptr(root_token), _ptr(tree_off), nseq, N, W, V,
                           total_nodes, _ptr(parent), _ptr(token), _ptr(depth), _ptr(anc),
                           _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "jt_tree_build")
    return parent, token, depth, anc


@_on_tensor_device
def jt_tree_build_mixed(draft_logits, root_token, tree_off, W, alpha, total_nodes=None, out=None, ws=None,
                        stream=None):
    """jt_tree_build whose step scores are (1 - alpha) * log-prob - alpha *
    entropy(draft row), alpha in [0, 1] (1: pure entropy score).

    Returns (parent, token, depth, anc) on the device."""
    lib = load()
    _need(draft_logits, "draft_logits", torch.float32)
    _need(root_token, "root_token", torch.int32)
    _need(tree_off, "tree_off", torch.int32)
    nseq, N, V = draft_logits.shape
    if total_nodes is None:
        total_nodes = int(tree_off[-1].item())
    dev = draft_logits.device
    if out is None:
        out = (torch.empty(total_nodes, dtype=torch.int32, device=dev),
               torch.empty(total_nodes, dtype=torch.int32, device=dev),
               torch.empty(total_nodes, dtype=torch.int32, device=dev),
               torch.empty((total_nodes, 8), dtype=torch.int32, device=dev))
    parent, token, depth, anc = out
    if ws is None:
        ws = workspace(jt_workspace_size(JT_OP_TREE_BUILD_MIXED, nseq, N, W, V), dev)
    rc = lib.jt_tree_build_mixed(_ptr(draft_logits), _ptr(root_token), _ptr(tree_off), nseq, N, W, V,
                                 total_nodes, float(alpha), _ptr(parent), _ptr(token), _ptr(depth),
                                 _ptr(anc), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "jt_tree_build_mixed")
    return parent, token, depth, anc


@_on_tensor_device
def jt_tree_build_noalloc(draft_logits, root_token, tree_off, W, total_nodes=None, out=None,
                          sync_check=True, stream=None):
    """jt_tree_build with the library's fixed device scratch instead of a
    workspace (no allocation inside the library; the output tensors are the
    caller's).  Calls whose executions overlap on one device race on that
    scratch.  Returns (parent, token, depth, anc) on the device."""
    lib = load()
    _need(draft_logits, "draft_logits", torch.float32)
    _need(root_token, "root_token", torch.int32)
    _need(tree_off, "tree_off", torch.int32)
    nseq, N, V = draft_logits.shape
    if total_nodes is None:
        total_nodes = int(tree_off[-1].item())
    dev = draft_logits.device
    if out is None:
        out = (torch.empty(total_nodes, dtype=torch.int32, device=dev),
               torch.empty(total_nodes, dtype=torch.int32, device=dev),
               torch.empty(total_nodes, dtype=torch.int32, device=dev),
               torch.empty((total_nodes, 8), dtype=torch.int32, device=dev))
    parent, token, depth, anc = out
    rc = lib.jt_tree_build_noalloc(_ptr(draft_logits), _ptr(root_token), _ptr(tree_off), nseq, N, W,
                                   V, total_nodes, _ptr(parent), _ptr(token), _ptr(depth), _ptr(anc),
                                   1 if sync_check else 0, _stream(stream))
    _check(rc, "jt_tree_build_noalloc")
    return parent, token, depth, anc


@_on_tensor_device
def jt_tree_topw(logits, W, ws=None, stream=None):
    """Top-W ids (int32), log-probs and lse (fp64) of every row of [..., V] fp32."""
    lib = load()
    _need(logits, "logits", torch.float32)
    V = logits.shape[-1]
    rows = logits.numel() // V
    dev = logits.device
    tok = torch.empty(logits.shape[:-1] + (W,), dtype=torch.int32, device=dev)
    lp = torch.empty(logits.shape[:-1] + (W,), dtype=torch.float64, device=dev)
    lse = torch.empty(logits.shape[:-1], dtype=torch.float64, device=dev)
    if ws is None:
        ws = workspace(jt_workspace_size(JT_OP_TREE_TOPW, rows, 1, W, V), dev)
    rc = lib.jt_tree_topw(_ptr(logits), rows, V, W, _ptr(tok), _ptr(lp), _ptr(lse), _ptr(ws),
                          ws.numel(), _stream(stream))
    _check(rc, "jt_tree_topw")
    return tok, lp, lse


@_on_tensor_device
def jt_tree_expand(tok, lp, root_token, tree_off, total_nodes=None, ws=None, stream=None):
    """Best-first expansion from given tables tok [nseq,N,W] int32, lp fp64."""
    lib = load()
    _need(tok, "tok", torch.int32)
    _need(lp, "lp", torch.float64)
    _need(root_token, "root_token", torch.int32)
    _need(tree_off, "tree_off", torch.int32)
    nseq, N, W = tok.shape
    if total_nodes is None:
        total_nodes = int(tree_off[-1].item())
    dev = tok.device
    parent = torch.empty(total_nodes, dtype=torch.int32, device=dev)
    token = torch.empty_like(parent)
    depth = torch.empty_like(parent)
    anc = torch.empty((total_nodes, 8), dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(256, dev)
    rc = lib.jt_tree_expand(_ptr(tok), _ptr(lp), _ptr(root_token), _ptr(tree_off), nseq, N, W,
                            total_nodes, _ptr(parent), _ptr(token), _ptr(depth), _ptr(anc),
                            _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "jt_tree_expand")
    return parent, token, depth, anc


@_on_tensor_device
def jt_tree_expand_capped(tok, lp, root_token, tree_off, w_cap=None, n_cap=None, total_nodes=None, ws=None,
                          stream=None):
    """jt_tree_expand with optional per-sequence width / depth caps
    (int32 [nseq] device tensors)."""
    lib = load()
    _need(tok, "tok", torch.int32)
    _need(lp, "lp", torch.float64)
    _need(root_token, "root_token", torch.int32)
    _need(tree_off, "tree_off", torch.int32)
    for t, name in ((w_cap, "w_cap"), (n_cap, "n_cap")):
        if t is not None:
            _need(t, name, torch.int32)
    nseq, N, W = tok.shape
    if total_nodes is None:
        total_nodes = int(tree_off[-1].item())
    dev = tok.device
    parent = torch.empty(total_nodes, dtype=torch.int32, device=dev)
    token = torch.empty_like(parent)
    depth = torch.empty_like(parent)
    anc = torch.empty((total_nodes, 8), dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(256, dev)
    rc = lib.jt_tree_expand_capped(_ptr(tok), _ptr(lp), _ptr(root_token), _ptr(tree_off), _ptr(w_cap),
                                   _ptr(n_cap), nseq, N, W, total_nodes, _ptr(parent), _ptr(token),
                                   _ptr(depth), _ptr(anc), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "jt_tree_expand_capped")
    return parent, token, depth, anc


@_on_tensor_device
def jt_tree_policy(lp, accept_len, budget_state, acc_ema, params=None, out=None, ws=None, stream=None):
    """One step of the adaptive tree policy.  lp fp64 [nseq, N, W];
    accept_len int32 [nseq] or None; budget_state int32 / acc_ema fp64
    [nseq] are updated in place.  Returns (tree_off, w_cap, n_cap)."""
    lib = load()
    _need(lp, "lp", torch.float64)
    _need(budget_state, "budget_state", torch.int32)
    _need(acc_ema, "acc_ema", torch.float64)
    if accept_len is not None:
        _need(accept_len, "accept_len", torch.int32)
    nseq, N, W = lp.shape
    params = params or policy_params()
    dev = lp.device
    if out is None:
        out = (torch.empty(nseq + 1, dtype=torch.int32, device=dev),
               torch.empty(nseq, dtype=torch.int32, device=dev),
               torch.empty(nseq, dtype=torch.int32, device=dev))
    tree_off, w_cap, n_cap = out
    if ws is None:
        ws = workspace(jt_workspace_size(JT_OP_TREE_POLICY), dev)
    rc = lib.jt_tree_policy(_ptr(lp), nseq, N, W, _ptr(accept_len), ctypes.byref(params), _ptr(budget_state),
                            _ptr(acc_ema), _ptr(tree_off), _ptr(w_cap), _ptr(n_cap), _ptr(ws), ws.numel(),
                            _stream(stream))
    _check(rc, "jt_tree_policy")
    return tree_off, w_cap, n_cap


@_on_tensor_device
def jt_tree_build_adaptive(draft_logits, root_token, accept_len, budget_state, acc_ema, W, params=None,
                           capacity=None, out=None, ws=None, stream=None):
    """Top-W tables, adaptive policy and capped expansion in one call.
    Returns (tree_off, w_cap, n_cap, parent, token, depth, anc); the node
    arrays have `capacity` rows (default nseq * the policy's ceiling)."""
    lib = load()
    _need(draft_logits, "draft_logits", torch.float32)
    _need(root_token, "root_token", torch.int32)
    _need(budget_state, "budget_state", torch.int32)
    _need(acc_ema, "acc_ema", torch.float64)
    if accept_len is not None:
        _need(accept_len, "accept_len", torch.int32)
    nseq, N, V = draft_logits.shape
    params = params or policy_params()
    if capacity is None:
        capacity = nseq * policy_ceiling(params, nseq)
    dev = draft_logits.device
    if out is None:
        out = (torch.empty(nseq + 1, dtype=torch.int32, device=dev),
               torch.empty(nseq, dtype=torch.int32, device=dev),
               torch.empty(nseq, dtype=torch.int32, device=dev),
               torch.empty(capacity, dtype=torch.int32, device=dev),
               torch.empty(capacity, dtype=torch.int32, device=dev),
               torch.empty(capacity, dtype=torch.int32, device=dev),
               torch.empty((capacity, 8), dtype=torch.int32, device=dev))
    tree_off, w_cap, n_cap, parent, token, depth, anc = out
    if ws is None:
        ws = workspace(jt_workspace_size(JT_OP_TREE_BUILD, nseq, N, W, V), dev)
    rc = lib.jt_tree_build_adaptive(_ptr(draft_logits), _ptr(root_token), nseq, N, W, V, capacity,
                                    _ptr(accept_len), ctypes.byref(params), _ptr(budget_state), _ptr(acc_ema),
                                    _ptr(tree_off), _ptr(w_cap), _ptr(n_cap), _ptr(parent), _ptr(token),
                                    _ptr(depth), _ptr(anc), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "jt_tree_build_adaptive")
    return tree_off, w_cap, n_cap, parent, token, depth, anc


@_on_tensor_device
def jt_tree_attn_paged(q, k_cache, v_cache, block_table, prefix_len, tree_off, anc, scale=None,
                       max_tree=None, out=None, lse=None, ws=None, stream=None, with_lse=True):
    """Tree-causal attention over a paged KV cache.

    q [total, Hq, D]; k/v [pages, 16, Hkv, D] (both bf16, or both fp32);
    block_table [nseq, max_pages] int32; prefix_len [nseq] int32;
    tree_off [nseq+1] int32; anc [total, 8] int32/uint32 ancestor sets.
    Returns (out, lse)."""
    lib = load()
    if q.dtype == torch.bfloat16:
        dtype = JT_DTYPE_BF16
    elif q.dtype == torch.float32:
        dtype = JT_DTYPE_F32
    else:
        raise TypeError("q must be bf16 or fp32")
    _need(q, "q", None)
    _need(k_cache, "k_cache", q.dtype)
    _need(v_cache, "v_cache", q.dtype)
    _need(block_table, "block_table", torch.int32)
    _need(prefix_len, "prefix_len", torch.int32)
    _need(tree_off, "tree_off", torch.int32)
    _need(anc, "anc", None)
    total, Hq, D = q.shape
    num_pages, page, Hkv, D2 = k_cache.shape
    if D2 != D:
        raise ValueError("q and k_cache head dims differ")
    nseq, max_pages = block_table.shape
    if max_tree is None:
        max_tree = int((tree_off[1:] - tree_off[:-1]).max().item())
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and with_lse:
        lse = torch.empty((total, Hq), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(jt_workspace_size(JT_OP_TREE_ATTN, nseq, 0, 0, 0, total, Hq, Hkv, D,
                                         max_pages, max_tree), q.device)
    rc = lib.jt_tree_attn_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), dtype, _ptr(block_table),
                                max_pages, num_pages, _ptr(prefix_len), _ptr(tree_off), _ptr(anc),
                                nseq, total, max_tree, Hq, Hkv, D, page, float(scale), _ptr(out),
                                _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "jt_tree_attn_paged")
    return out, lse


@_on_tensor_device
def jt_verify_accept(target_logits, parent, token, tree_off, N, rule=JT_RULE_GREEDY, t=None,
                     log_t=None, out=None, ws=None, stream=None):
    """Tree acceptance: returns (accept_len [nseq], path [nseq, N+1], bonus [nseq])."""
    lib = load()
    _need(target_logits, "target_logits", torch.float32)
    _need(parent, "parent", torch.int32)
    _need(token, "token", torch.int32)
    _need(tree_off, "tree_off", torch.int32)
    total, V = target_logits.shape
    nseq = tree_off.numel() - 1
    if isinstance(rule, str):
        rule = {"greedy": JT_RULE_GREEDY, "margin": JT_RULE_MARGIN}[rule]
    if log_t is None:
        log_t = math.log(t) if t is not None else 0.0
    dev = target_logits.device
    if out is None:
        out = (torch.empty(nseq, dtype=torch.int32, device=dev),
               torch.empty((nseq, N + 1), dtype=torch.int32, device=dev),
               torch.empty(nseq, dtype=torch.int32, device=dev))
    acc, path, bonus = out
    if ws is None:
        ws = workspace(jt_workspace_size(JT_OP_VERIFY_ACCEPT, nseq, 0, 0, 0, total), dev)
    rc = lib.jt_verify_accept(_ptr(target_logits), _ptr(parent), _ptr(token), _ptr(tree_off), nseq,
                              N, V, total, rule, float(log_t), _ptr(acc), _ptr(path), _ptr(bonus),
                              _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "jt_verify_accept")
    return acc, path, bonus


# The cache operators run once per layer and token, where the host's time per
# call counts: one pass of checks per tensor, the arguments packed for jt_call.
_PACK = {op: struct.Struct(fmt) for op, fmt in (
    (JT_OP_QKV_APPEND, "@PiqPPfPiiiPPiiPPiiiiiiPPPPNP"),
    (JT_OP_CHUNK_ATTN, "@PPPiPiiPPiiiiiiifPPPNP"),
    (JT_OP_KV_COMMIT, "@PPiiqPiiPPPPiiiiiPPNP"))}
_FLOATS = {torch.bfloat16: JT_DTYPE_BF16, torch.float32: JT_DTYPE_F32}


def _lead(t, name):
    """Device index and jt dtype of the tensor that sets both for a call."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    dtype = _FLOATS.get(t.dtype)
    if dtype is None:
        raise TypeError(f"{name} must be bf16 or fp32")
    idx = t.get_device()
    if idx < 0:
        raise ValueError(f"{name} must be a CUDA tensor (libjt has no CPU path)")
    return idx, dtype


def _like(t, name, dtype, idx, shape):
    """Check a contiguous tensor of the call's device, a type and a shape."""
    if (not isinstance(t, torch.Tensor) or t.get_device() != idx or t.dtype is not dtype or t.shape != shape
            or not t.is_contiguous()):
        _need(t, name, dtype)
        if t.get_device() != idx:
            raise ValueError(f"{name}: tensors on several devices (cuda:{idx}, cuda:{t.get_device()})")
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _layers(t, name, dtype, idx, shape):
    """Check a cache whose layers (the first of five dimensions) are contiguous,
    but may lie apart; the elements from one to the next."""
    if len(shape) == 5 and isinstance(t, torch.Tensor) and t.shape == shape and not t.is_contiguous():
        _like(t[0], name, dtype, idx, shape[1:])
        return t.stride(0)
    _like(t, name, dtype, idx, shape)
    return shape[-4] * shape[-3] * shape[-2] * shape[-1]


def _tables(block_table, prefix_len, off, off_name, idx):
    """(nseq, max_pages) of a batch's checked tables."""
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor of 2 dimensions")
    shape = block_table.shape
    _like(block_table, "block_table", torch.int32, idx, shape)
    nseq, max_pages = shape
    _like(prefix_len, "prefix_len", torch.int32, idx, (nseq,))
    _like(off, off_name, torch.int32, idx, (nseq + 1,))
    return nseq, max_pages


def _workspace_of(ws, idx):
    if not isinstance(ws, torch.Tensor) or ws.get_device() != idx or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on cuda:{idx}")
    return ws.numel() * ws.element_size()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # no Stream object made


def _packed(op, idx, *args):
    """jt_call on the tensors' device and its current stream."""
    lib = load()
    s = _PACK[op]
    if idx != torch.cuda.current_device():
        with torch.cuda.device(idx):
            return lib.jt_call(op, s.pack(*args, _stream()), s.size)
    return lib.jt_call(op, s.pack(*args, _raw_stream(idx) if _raw_stream is not None else _stream()), s.size)


def _on_given_stream(fn):
    """Make a given stream the current one for the call, so that what the call
    allocates (and frees, and zeroes) belongs to the stream that uses it."""
    @functools.wraps(fn)
    def wrapper(*args, stream=None, **kwargs):
        if stream is None:
            return fn(*args, **kwargs)
        idx = _device_of(kwargs.values(), _device_of(args, -1, fn.__name__), fn.__name__)
        if idx >= 0 and stream.device_index != idx:
            raise ValueError(f"{fn.__name__}: tensors on cuda:{idx}, stream on cuda:{stream.device_index}")
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return wrapper


def rope_table(max_pos, rot_dim, theta=1e6, device=None):
    """cos_sin table of jt_qkv_append for the usual angles pos * theta^(-2j /
    rot_dim): fp32 [max_pos, rot_dim], cosines then sines, computed in 64 bits
    and rounded once (made once per model)."""
    inv = float(theta) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().to(device or "cuda")


@_on_given_stream
def jt_qkv_append(qkv, Hq, k_cache, v_cache, block_table, prefix_len, tree_off, q_weight=None, k_weight=None,
                  eps=1e-6, cos_sin=None, interleaved=False, depth=None, q_out=None, ws=None):
    """Per-head norm of q and k, position rotation, and the write of k and v
    into the paged cache, from the packed projection.

    qkv [total, (Hq + 2 Hkv) * D] (rows may be strided); k/v_cache [pages, 16,
    Hkv, D]; q_weight, k_weight [D] or None; cos_sin fp32 [max_pos, rot_dim] or
    None (see rope_table); depth int32 [total] (tree nodes: position L_b +
    depth) or None (position L_b + i).  Returns q_out [total, Hq, D] (None for
    Hq = 0); the caches are updated in place.  stream (keyword): the stream to
    run on, as in every call here; default the current one."""
    idx, dtype = _lead(qkv, "qkv")
    kind, kv_shape = qkv.dtype, k_cache.shape
    if len(kv_shape) != 4:
        raise ValueError("k_cache must be [pages, 16, Hkv, D]")
    _like(k_cache, "k_cache", kind, idx, kv_shape)
    _like(v_cache, "v_cache", kind, idx, kv_shape)
    nseq, max_pages = _tables(block_table, prefix_len, tree_off, "tree_off", idx)
    num_pages, page, Hkv, D = kv_shape
    width = (Hq + 2 * Hkv) * D
    if qkv.dim() != 2 or qkv.shape[1] != width:
        raise ValueError(f"qkv must be [total, (Hq + 2 Hkv) * D = {width}], got {tuple(qkv.shape)}")
    total, row = qkv.shape[0], width
    if not qkv.is_contiguous():
        if qkv.stride(1) != 1:
            raise ValueError("qkv's rows must be contiguous")
        row = qkv.stride(0)
    qw = kw = table = steps = q_ptr = 0
    if q_weight is not None:
        _like(q_weight, "q_weight", kind, idx, (D,))
        qw = q_weight.data_ptr()
    if k_weight is not None:
        _like(k_weight, "k_weight", kind, idx, (D,))
        kw = k_weight.data_ptr()
    max_pos = rot = 0
    if cos_sin is not None:
        if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_pos, rot_dim]")
        max_pos, rot = cos_sin.shape
        _like(cos_sin, "cos_sin", torch.float32, idx, (max_pos, rot))
        table = cos_sin.data_ptr()
    if depth is not None:
        _like(depth, "depth", torch.int32, idx, (total,))
        steps = depth.data_ptr()
    if Hq > 0:
        if q_out is None:
            q_out = torch.empty((total, Hq, D), dtype=kind, device=qkv.device)
        else:
            _like(q_out, "q_out", kind, idx, (total, Hq, D))
        q_ptr = q_out.data_ptr()
    if ws is None:
        ws = workspace(256, qkv.device)
    rc = _packed(JT_OP_QKV_APPEND, idx, qkv.data_ptr(), dtype, row, qw, kw, eps, table, max_pos, rot,
                 1 if interleaved else 0, steps, block_table.data_ptr(), max_pages, num_pages, prefix_len.data_ptr(),
                 tree_off.data_ptr(), nseq, total, Hq, Hkv, D, page, q_ptr, k_cache.data_ptr(), v_cache.data_ptr(),
                 ws.data_ptr(), _workspace_of(ws, idx))
    if rc != JT_OK:
        raise JtError(rc, "jt_qkv_append")
    return q_out


@_on_given_stream
def jt_chunk_attn_paged(q, k_cache, v_cache, block_table, prefix_len, chunk_off, scale=None, max_chunk=None,
                        out=None, lse=None, ws=None, with_lse=True):
    """Causal attention of new tokens (chunks of any length, ragged) over a
    paged KV cache that already holds their keys and values.

    q [total, Hq, D]; k/v [pages, 16, Hkv, D] (both bf16, or both fp32);
    block_table [nseq, max_pages] int32; prefix_len [nseq] int32 (tokens cached
    before); chunk_off [nseq+1] int32; max_chunk: the longest chunk (an upper
    bound; None reads it from chunk_off, which waits for the device).  Returns
    (out, lse)."""
    idx, dtype = _lead(q, "q")
    kind, q_shape, kv_shape = q.dtype, q.shape, k_cache.shape
    if len(q_shape) != 3 or len(kv_shape) != 4:
        raise ValueError("q must be [total, Hq, D] and k_cache [pages, 16, Hkv, D]")
    _like(q, "q", kind, idx, q_shape)
    _like(k_cache, "k_cache", kind, idx, kv_shape)
    _like(v_cache, "v_cache", kind, idx, kv_shape)
    nseq, max_pages = _tables(block_table, prefix_len, chunk_off, "chunk_off", idx)
    total, Hq, D = q_shape
    num_pages, page, Hkv, D2 = kv_shape
    if D2 != D:
        raise ValueError("q and k_cache head dims differ")
    if max_chunk is None:
        max_chunk = max(1, int((chunk_off[1:] - chunk_off[:-1]).max().item()))
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    else:
        _like(out, "out", kind, idx, q_shape)
    if lse is not None:
        _like(lse, "lse", torch.float32, idx, (total, Hq))
    elif with_lse:
        lse = torch.empty((total, Hq), dtype=torch.float32, device=q.device)
    if ws is None:
        with torch.cuda.device(idx):  # sized for the tensors' device
            ws = torch.empty(jt_workspace_size(JT_OP_CHUNK_ATTN, nseq, 0, 0, 0, total, Hq, Hkv, D,
                                               1 if dtype == JT_DTYPE_BF16 else max_pages, max_chunk),
                             dtype=torch.uint8, device=q.device)
            ws[:4096].zero_()  # the part that must be zero
    rc = _packed(JT_OP_CHUNK_ATTN, idx, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), dtype,
                 block_table.data_ptr(), max_pages, num_pages, prefix_len.data_ptr(), chunk_off.data_ptr(), nseq,
                 total, max_chunk, Hq, Hkv, D, page, scale, out.data_ptr(), 0 if lse is None else lse.data_ptr(),
                 ws.data_ptr(), _workspace_of(ws, idx))
    if rc != JT_OK:
        raise JtError(rc, "jt_chunk_attn_paged")
    return out, lse


@_on_given_stream
def jt_kv_commit(k_cache, v_cache, block_table, prefix_len, tree_off, accept_len, path, new_prefix=None, ws=None):
    """Move the accepted path's keys and values behind the prefix and advance
    the prefix lengths.

    k/v_cache [pages, 16, Hkv, D] or [layers, pages, 16, Hkv, D] (bf16 or fp32,
    updated in place; the layers contiguous, and the same distance apart in both:
    kv[:, 0] and kv[:, 1] of a [layers, 2, pages, 16, Hkv, D] pool do); accept_len [nseq], path [nseq, N+1] int32 as
    jt_verify_accept returns them; new_prefix: int32 [nseq] output, prefix_len
    itself to update it in place, None for a new tensor.  Returns new_prefix."""
    idx, dtype = _lead(k_cache, "k_cache")
    kv_shape = k_cache.shape
    if len(kv_shape) not in (4, 5):
        raise ValueError("k_cache must be [pages, 16, Hkv, D] or [layers, pages, 16, Hkv, D]")
    layers = kv_shape[0] if len(kv_shape) == 5 else 1
    layer_stride = _layers(k_cache, "k_cache", k_cache.dtype, idx, kv_shape)
    if _layers(v_cache, "v_cache", k_cache.dtype, idx, kv_shape) != layer_stride:
        raise ValueError("the layers of k_cache and v_cache are different distances apart")
    nseq, max_pages = _tables(block_table, prefix_len, tree_off, "tree_off", idx)
    _like(accept_len, "accept_len", torch.int32, idx, (nseq,))
    if not isinstance(path, torch.Tensor) or path.dim() != 2:
        raise ValueError("path must be [nseq, N+1]")
    width = path.shape[1]
    _like(path, "path", torch.int32, idx, (nseq, width))
    num_pages, page, Hkv, D = kv_shape[-4:]
    if new_prefix is None:
        new_prefix = torch.empty_like(prefix_len)
    elif new_prefix is not prefix_len:
        _like(new_prefix, "new_prefix", torch.int32, idx, (nseq,))
    if ws is None:
        ws = workspace(jt_workspace_size(JT_OP_KV_COMMIT, nseq), k_cache.device)
    rc = _packed(JT_OP_KV_COMMIT, idx, k_cache.data_ptr(), v_cache.data_ptr(), dtype, layers,
                 layer_stride, block_table.data_ptr(), max_pages, num_pages, prefix_len.data_ptr(),
                 tree_off.data_ptr(), accept_len.data_ptr(), path.data_ptr(), nseq, width - 1, Hkv, D, page,
                 new_prefix.data_ptr(), ws.data_ptr(), _workspace_of(ws, idx))
    if rc != JT_OK:
        raise JtError(rc, "jt_kv_commit")
    return new_prefix


@_on_tensor_device
def jt_selftest_wait_timeout(ws=None, stream=None):
    """Run the bounded-wait timeout diagnostic; returns the workspace whose
    error word it sets (read it with jt_check: JT_ERR_TIMEOUT)."""
    lib = load()
    if ws is None:
        ws = workspace(256)
    _check(lib.jt_selftest_wait_timeout(_ptr(ws), ws.numel(), _stream(stream)), "jt_selftest_wait_timeout")
    return ws
