// jt_api.cu -- the extern "C" entry points of libjt (declared in include/jt.h):
// host-side argument checks, workspace carving, kernel launches.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "jt_common.cuh"
#include "jt_internal.h"

namespace jt {

int device_sm_count() {
    static PerDeviceCache cache;
    return cache.get([] {
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 0;
        return sms;
    });
}

static jt_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return JT_OK;
    if (e == cudaErrorInvalidValue) return JT_ERR_INVALID;
    if (e == cudaErrorNoKernelImageForDevice || e == cudaErrorNotSupported ||
        e == cudaErrorInvalidDeviceFunction)
        return JT_ERR_UNSUPPORTED;
    return JT_ERR_CUDA;
}

static bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

// Whether some layer of k meets some layer of v: `layers` pools of n bytes each,
// stride >= n bytes apart.
static bool layers_meet(const void* k, const void* v, int64_t n, int64_t stride, int layers) {
    const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(v) - reinterpret_cast<uintptr_t>(k));
    if (layers == 1) return d > -n && d < n;
    // layers t apart differ by d + t * stride: the nearest to 0 are beside t = -d / stride
    for (int64_t t = -d / stride - 1; t <= -d / stride + 1; ++t)
        if (t > -layers && t < layers && d + t * stride > -n && d + t * stride < n) return true;
    return false;
}

static jt_status check_ws(void* ws, size_t ws_bytes, size_t need) {
    if (!ws || !aligned(ws, kAlign) || ws_bytes < need) return JT_ERR_WORKSPACE;
    return JT_OK;
}

static size_t build_ws(int nseq, int N, int W, long long V, bool ent = false) {
    return kWsHeader + topw_workspace_bytes(static_cast<long long>(nseq) * N, V, W, ent);
}

}  // namespace jt

using namespace jt;

extern "C" {

int jt_version(void) { return 1 * 10000 + 1 * 100 + 0; }

const char* jt_status_str(jt_status s) {
    switch (s) {
        case JT_OK: return "JT_OK";
        case JT_ERR_INVALID: return "JT_ERR_INVALID: invalid argument or device array contents";
        case JT_ERR_UNSUPPORTED: return "JT_ERR_UNSUPPORTED: outside this build's limits or GPU";
        case JT_ERR_CUDA: return "JT_ERR_CUDA: a CUDA runtime call failed";
        case JT_ERR_TIMEOUT: return "JT_ERR_TIMEOUT: a bounded device-side wait ran out";
        case JT_ERR_WORKSPACE: return "JT_ERR_WORKSPACE: workspace missing, misaligned or too small";
    }
    return "unknown jt_status";
}

size_t jt_workspace_size(int op, int nseq, int N, int W, int64_t V, int total_nodes, int Hq,
                         int Hkv, int D, int max_pages, int max_tree) {
    switch (op) {
        case JT_OP_TREE_BUILD:
        case JT_OP_TREE_BUILD_MIXED:
            if (nseq < 1 || N < 0 || N > JT_MAX_N || W < 1 || W > JT_MAX_W || V < W) return 0;
            return build_ws(nseq, N, W, V, op == JT_OP_TREE_BUILD_MIXED);
        case JT_OP_TREE_TOPW:
            if (nseq < 0 || W < 1 || W > JT_MAX_W || V < W) return 0;
            return build_ws(nseq, 1, W, V);
        case JT_OP_TREE_ATTN: {
            if (nseq < 1 || total_nodes < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || D < 1 ||
                max_pages < 1 || max_tree < 1 || max_tree > JT_MAX_TREE)
                return 0;
            const AttnPlan pl = attn_plan(nseq, Hkv, Hq, D, max_tree, max_pages, JT_DTYPE_BF16);
            return attn_workspace_bytes(pl, total_nodes, Hq, D);
        }
        case JT_OP_VERIFY_ACCEPT:
            if (nseq < 1 || total_nodes < 1) return 0;
            return accept_workspace_bytes(nseq, total_nodes);
        case JT_OP_TREE_POLICY:
        case JT_OP_QKV_APPEND:
            return kWsHeader;
        case JT_OP_CHUNK_ATTN:
            if (nseq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || D < 1 || max_pages < 1 || max_tree < 1) return 0;
            return std::max(chunk_attn_bf16_workspace_bytes(D),
                            chunk_attn_f32_workspace_bytes(nseq, Hq, Hkv, D, max_pages, max_tree));
        case JT_OP_KV_COMMIT:
            return nseq < 1 ? 0 : kv_commit_workspace_bytes(nseq);
        default:
            return 0;
    }
}

jt_status jt_tree_topw(const float* logits, int64_t rows, int64_t V, int W, int32_t* tok,
                       double* lp, double* lse, void* ws, size_t ws_bytes, jt_stream_t stream) {
    JT_RANGE("jt_tree_topw");
    if (!logits || !tok || !lp || !lse || rows < 0 || W < 1 || W > JT_MAX_W || V < W ||
        V > 0x7FFFFFFFll || rows > 65535)
        return JT_ERR_INVALID;
    jt_status s = check_ws(ws, ws_bytes, build_ws(static_cast<int>(rows), 1, W, V));
    if (s != JT_OK) return s;
    if (rows == 0) return JT_OK;
    char* base = static_cast<char*>(ws);
    cudaError_t e = tree_topw_launch(logits, rows, V, W, tok, lp, lse, base + kWsHeader, stream);
    return from_cuda(e);
}

jt_status jt_tree_build_mixed(const float* draft_logits, const int32_t* root_token,
                              const int32_t* tree_off, int nseq, int N, int W, int64_t V,
                              int total_nodes, double alpha, int32_t* parent, int32_t* token,
                              int32_t* depth, uint32_t* anc, void* ws, size_t ws_bytes,
                              jt_stream_t stream) {
    JT_RANGE("jt_tree_build_mixed");
    if ((!draft_logits && N > 0) || !root_token || !tree_off || !parent || !token || !depth ||
        !anc || nseq < 1 || nseq > 65535 || N < 0 || N > JT_MAX_N || W < 1 || W > JT_MAX_W ||
        V < W || V > 0x7FFFFFFFll || total_nodes < nseq ||
        static_cast<long long>(nseq) * N > 65535 || !(alpha >= 0.0 && alpha <= 1.0))
        return JT_ERR_INVALID;
    if (!aligned(anc, 16)) return JT_ERR_INVALID;
    jt_status s = check_ws(ws, ws_bytes, build_ws(nseq, N, W, V, alpha != 0.0));
    if (s != JT_OK) return s;
    char* base = static_cast<char*>(ws);
    cudaError_t e = tree_build_launch(draft_logits, root_token, tree_off, nseq, total_nodes, N, W, V, alpha,
                                      parent, token, depth, anc, base + kWsHeader,
                                      reinterpret_cast<uint32_t*>(base), stream);
    return from_cuda(e);
}

jt_status jt_tree_build(const float* draft_logits, const int32_t* root_token,
                        const int32_t* tree_off, int nseq, int N, int W, int64_t V, int total_nodes,
                        int32_t* parent, int32_t* token, int32_t* depth, uint32_t* anc, void* ws,
                        size_t ws_bytes, jt_stream_t stream) {
    JT_RANGE("jt_tree_build");
    return jt_tree_build_mixed(draft_logits, root_token, tree_off, nseq, N, W, V, total_nodes, 0.0, parent,
                               token, depth, anc, ws, ws_bytes, stream);
}

jt_status jt_tree_expand_capped(const int32_t* tok, const double* lp, const int32_t* root_token,
                                const int32_t* tree_off, const int32_t* w_cap, const int32_t* n_cap,
                                int nseq, int N, int W, int total_nodes, int32_t* parent,
                                int32_t* token, int32_t* depth, uint32_t* anc, void* ws,
                                size_t ws_bytes, jt_stream_t stream) {
    JT_RANGE("jt_tree_expand_capped");
    if ((N > 0 && (!tok || !lp)) || !root_token || !tree_off || !parent || !token || !depth ||
        !anc || nseq < 1 || nseq > 65535 || N < 0 || N > JT_MAX_N || W < 1 || W > JT_MAX_W ||
        total_nodes < nseq || !aligned(anc, 16))
        return JT_ERR_INVALID;
    jt_status s = check_ws(ws, ws_bytes, kWsHeader);
    if (s != JT_OK) return s;
    char* base = static_cast<char*>(ws);
    cudaError_t e = tree_expand_launch(tok, lp, root_token, tree_off, w_cap, n_cap, nseq, total_nodes, N, W,
                                       parent, token, depth, anc, reinterpret_cast<uint32_t*>(base), stream);
    return from_cuda(e);
}

jt_status jt_tree_expand(const int32_t* tok, const double* lp, const int32_t* root_token,
                         const int32_t* tree_off, int nseq, int N, int W, int total_nodes,
                         int32_t* parent, int32_t* token, int32_t* depth, uint32_t* anc, void* ws,
                         size_t ws_bytes, jt_stream_t stream) {
    JT_RANGE("jt_tree_expand");
    return jt_tree_expand_capped(tok, lp, root_token, tree_off, nullptr, nullptr, nseq, N, W, total_nodes,
                                 parent, token, depth, anc, ws, ws_bytes, stream);
}

// Host checks of the policy's parameters (jt_tree_policy's rules); returns
// the per-request budget ceiling, or 0 when a parameter is out of range.
static int policy_params_ok(const jt_policy_params* p, int nseq, int N, int W) {
    if (!p || p->b_min < 1 || p->b_max < p->b_min || p->b_max > JT_MAX_TREE || p->node_cap < 0 ||
        p->w_min < 1 || p->w_min > W || p->n_min < 0 || p->n_min > N || p->n_slack < 0 ||
        p->n_slack > N || !(p->beta > 0.0) || !(p->beta <= 1.0) || p->log_conf != p->log_conf ||
        p->acc_thresh != p->acc_thresh)
        return 0;
    int c = p->b_max;
    if (p->node_cap > 0) {
        const int per = p->node_cap / nseq;
        c = per < p->b_min ? p->b_min : per;
        if (c > p->b_max) c = p->b_max;
    }
    return c;
}

jt_status jt_tree_policy(const double* lp, int nseq, int N, int W, const int32_t* accept_len,
                         const jt_policy_params* params, int32_t* budget_state, double* acc_ema,
                         int32_t* tree_off, int32_t* w_cap, int32_t* n_cap, void* ws,
                         size_t ws_bytes, jt_stream_t stream) {
    JT_RANGE("jt_tree_policy");
    if (!lp || !budget_state || !acc_ema || !tree_off || !w_cap || !n_cap || nseq < 1 ||
        nseq > 65535 || N < 1 || N > JT_MAX_N || W < 1 || W > JT_MAX_W ||
        policy_params_ok(params, nseq, N, W) == 0)
        return JT_ERR_INVALID;
    jt_status s = check_ws(ws, ws_bytes, kWsHeader);
    if (s != JT_OK) return s;
    cudaError_t e = tree_policy_launch(lp, nseq, N, W, accept_len, *params, budget_state, acc_ema, tree_off,
                                       w_cap, n_cap, static_cast<uint32_t*>(ws), stream);
    return from_cuda(e);
}

jt_status jt_tree_build_adaptive(const float* draft_logits, const int32_t* root_token, int nseq,
                                 int N, int W, int64_t V, int capacity, const int32_t* accept_len,
                                 const jt_policy_params* params, int32_t* budget_state,
                                 double* acc_ema, int32_t* tree_off, int32_t* w_cap,
                                 int32_t* n_cap, int32_t* parent, int32_t* token, int32_t* depth,
                                 uint32_t* anc, void* ws, size_t ws_bytes, jt_stream_t stream) {
    JT_RANGE("jt_tree_build_adaptive");
    if (!draft_logits || !root_token || !budget_state || !acc_ema || !tree_off || !w_cap || !n_cap ||
        !parent || !token || !depth || !anc || nseq < 1 || nseq > 65535 || N < 1 || N > JT_MAX_N ||
        W < 1 || W > JT_MAX_W || V < W || V > 0x7FFFFFFFll || static_cast<long long>(nseq) * N > 65535 ||
        !aligned(anc, 16))
        return JT_ERR_INVALID;
    const int ceil_b = policy_params_ok(params, nseq, N, W);
    if (ceil_b == 0 || static_cast<long long>(capacity) < static_cast<long long>(nseq) * ceil_b)
        return JT_ERR_INVALID;
    jt_status s = check_ws(ws, ws_bytes, build_ws(nseq, N, W, V));
    if (s != JT_OK) return s;
    char* base = static_cast<char*>(ws);
    cudaError_t e = tree_build_adaptive_launch(draft_logits, root_token, nseq, capacity, N, W, V, accept_len,
                                               *params, budget_state, acc_ema, tree_off, w_cap, n_cap, parent,
                                               token, depth, anc, base + kWsHeader,
                                               reinterpret_cast<uint32_t*>(base), stream);
    return from_cuda(e);
}

jt_status jt_tree_attn_paged(const void* q, const void* k_cache, const void* v_cache, int dtype,
                             const int32_t* block_table, int max_pages, int num_pages,
                             const int32_t* prefix_len, const int32_t* tree_off,
                             const uint32_t* anc, int nseq, int total_nodes, int max_tree, int Hq,
                             int Hkv, int D, int page_size, float scale, void* out, float* lse,
                             void* ws, size_t ws_bytes, jt_stream_t stream) {
    JT_RANGE("jt_tree_attn_paged");
    if (!q || !k_cache || !v_cache || !block_table || !prefix_len || !tree_off || !anc || !out ||
        nseq < 1 || nseq > 65535 || total_nodes < nseq || max_tree < 1 ||
        max_tree > JT_MAX_TREE || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_pages < 1 ||
        num_pages < 1 || page_size != JT_PAGE_SIZE || !isfinite(scale) ||
        (dtype != JT_DTYPE_BF16 && dtype != JT_DTYPE_F32))
        return JT_ERR_INVALID;
    const int G = Hq / Hkv;
    if (dtype == JT_DTYPE_BF16) {
        if (D != 64 && D != 128) return JT_ERR_UNSUPPORTED;
        if (G != 1 && G != 2 && G != 4 && G != 8 && G != 16) return JT_ERR_UNSUPPORTED;
        if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
            return JT_ERR_INVALID;
        if (Hkv > 65535) return JT_ERR_UNSUPPORTED;
    } else {
        if (D != 32 && D != 64 && D != 96 && D != 128) return JT_ERR_UNSUPPORTED;
    }
    const AttnPlan pl = attn_plan(nseq, Hkv, Hq, D, max_tree, max_pages, dtype);
    jt_status s = check_ws(ws, ws_bytes, attn_workspace_bytes(pl, total_nodes, Hq, D));
    if (s != JT_OK) return s;
    char* base = static_cast<char*>(ws);
    uint32_t* err = reinterpret_cast<uint32_t*>(base);
    cudaError_t e;
    if (dtype == JT_DTYPE_BF16)
        e = tree_attn_bf16_launch(q, k_cache, v_cache, block_table, max_pages, num_pages,
                                  prefix_len, tree_off, anc, nseq, total_nodes, Hq, Hkv, D, scale,
                                  out, lse, pl, base + kWsHeader, err, stream);
    else
        e = tree_attn_f32_launch(static_cast<const float*>(q), static_cast<const float*>(k_cache),
                                 static_cast<const float*>(v_cache), block_table, max_pages,
                                 num_pages, prefix_len, tree_off, anc, nseq, total_nodes, Hq, Hkv, D, scale,
                                 static_cast<float*>(out), lse, err, stream);
    return from_cuda(e);
}

jt_status jt_verify_accept(const float* target_logits, const int32_t* parent,
                           const int32_t* token, const int32_t* tree_off, int nseq, int N,
                           int64_t V, int total_nodes, int rule, double log_t,
                           int32_t* accept_len, int32_t* path, int32_t* bonus, void* ws,
                           size_t ws_bytes, jt_stream_t stream) {
    JT_RANGE("jt_verify_accept");
    if (!target_logits || !parent || !token || !tree_off || !accept_len || !path || !bonus ||
        nseq < 1 || nseq > 8192 || N < 0 || N > JT_MAX_TREE || V < 1 || V > 0x7FFFFFFFll ||
        total_nodes < nseq || (rule != JT_RULE_GREEDY && rule != JT_RULE_MARGIN) ||
        (rule == JT_RULE_MARGIN && !(log_t <= 0.0)))
        return JT_ERR_INVALID;
    jt_status s = check_ws(ws, ws_bytes, accept_workspace_bytes(nseq, total_nodes));
    if (s != JT_OK) return s;
    return from_cuda(verify_accept_launch(target_logits, parent, token, tree_off, nseq, N, V,
                                          total_nodes, rule, log_t, accept_len, path, bonus,
                                          static_cast<char*>(ws), stream));
}

jt_status jt_verify_accept_stochastic(const float* target_logits, const float* draft_logits,
                                      const int32_t* parent, const int32_t* token,
                                      const int32_t* tree_off, int nseq, int N, int64_t V,
                                      int total_nodes, const double* u_accept, const double* u_bonus,
                                      int32_t* accept_len, int32_t* path, int32_t* bonus, void* ws,
                                      size_t ws_bytes, jt_stream_t stream) {
    JT_RANGE("jt_verify_accept_stochastic");
    if (!target_logits || (!draft_logits && N > 0) || !parent || !token || !tree_off || !u_accept ||
        !u_bonus || !accept_len || !path || !bonus || nseq < 1 || nseq > 8192 || N < 0 ||
        N > JT_MAX_TREE || V < 1 || V > 0x7FFFFFFFll || total_nodes < nseq)
        return JT_ERR_INVALID;
    if (V > JT_STOCHASTIC_MAX_V) return JT_ERR_UNSUPPORTED;
    jt_status s = check_ws(ws, ws_bytes, accept_workspace_bytes(nseq, total_nodes));
    if (s != JT_OK) return s;
    return from_cuda(verify_stochastic_launch(target_logits, draft_logits, parent, token, tree_off, nseq, N, V,
                                              total_nodes, u_accept, u_bonus, accept_len, path, bonus,
                                              static_cast<char*>(ws), stream));
}

jt_status jt_qkv_append(const void* qkv, int dtype, int64_t row_stride, const void* q_weight,
                        const void* k_weight, float eps, const float* cos_sin, int max_pos,
                        int rot_dim, int interleaved, const int32_t* depth,
                        const int32_t* block_table, int max_pages, int num_pages,
                        const int32_t* prefix_len, const int32_t* tree_off, int nseq,
                        int total_nodes, int Hq, int Hkv, int D, int page_size, void* q_out,
                        void* k_cache, void* v_cache, void* ws, size_t ws_bytes,
                        jt_stream_t stream) {
    JT_RANGE("jt_qkv_append");
    if (total_nodes < 0 || nseq < 1 || nseq > 65535 || Hq < 0 || Hkv < 1 || D < 1 || max_pages < 1 ||
        num_pages < 1 || page_size != JT_PAGE_SIZE || rot_dim < 0 || rot_dim > D ||
        (interleaved != 0 && interleaved != 1) || !(eps >= 0.0f) || !isfinite(eps) ||
        (dtype != JT_DTYPE_BF16 && dtype != JT_DTYPE_F32))
        return JT_ERR_INVALID;
    const bool bf16 = dtype == JT_DTYPE_BF16;
    if (bf16 ? (D != 64 && D != 128) : (D != 32 && D != 64 && D != 96 && D != 128)) return JT_ERR_UNSUPPORTED;
    if (rot_dim % (bf16 ? 16 : 8) != 0) return JT_ERR_UNSUPPORTED;
    if (total_nodes == 0) return JT_OK;
    if (!qkv || !block_table || !prefix_len || !tree_off || !k_cache || !v_cache || (Hq > 0 && !q_out) ||
        (rot_dim > 0 && (!cos_sin || max_pos < 1)) ||
        row_stride < (static_cast<int64_t>(Hq) + 2 * static_cast<int64_t>(Hkv)) * D || row_stride % (bf16 ? 8 : 4) != 0)
        return JT_ERR_INVALID;
    if (!aligned(qkv, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(cos_sin, 16) ||
        !aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return JT_ERR_INVALID;
    jt_status s = check_ws(ws, ws_bytes, kWsHeader);
    if (s != JT_OK) return s;
    const int64_t esize = bf16 ? 2 : 4, pool = static_cast<int64_t>(num_pages) * JT_PAGE_SIZE * Hkv * D * esize;
    const int64_t in = (static_cast<int64_t>(total_nodes - 1) * row_stride + (Hq + 2ll * Hkv) * D) * esize;
    const int64_t qb = static_cast<int64_t>(total_nodes) * Hq * D * esize;
    if (overlap(k_cache, pool, v_cache, pool) || overlap(qkv, in, k_cache, pool) || overlap(qkv, in, v_cache, pool) ||
        overlap(q_out, qb, k_cache, pool) || overlap(q_out, qb, v_cache, pool) || overlap(q_out, qb, qkv, in))
        return JT_ERR_INVALID;
    AppendArgs a;
    a.qkv = qkv;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.cos_sin = cos_sin;
    a.depth = depth;
    a.block_table = block_table;
    a.prefix_len = prefix_len;
    a.tree_off = tree_off;
    a.q_out = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.row_stride = row_stride;
    a.dtype = dtype;
    a.max_pos = max_pos;
    a.rot_dim = rot_dim;
    a.interleaved = interleaved;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.nseq = nseq;
    a.total = total_nodes;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.eps = eps;
    return from_cuda(qkv_append_launch(a, static_cast<uint32_t*>(ws), stream));
}

jt_status jt_chunk_attn_paged(const void* q, const void* k_cache, const void* v_cache, int dtype,
                              const int32_t* block_table, int max_pages, int num_pages,
                              const int32_t* prefix_len, const int32_t* chunk_off, int nseq,
                              int total_tokens, int max_chunk, int Hq, int Hkv, int D,
                              int page_size, float scale, void* out, float* lse, void* ws,
                              size_t ws_bytes, jt_stream_t stream) {
    JT_RANGE("jt_chunk_attn_paged");
    if (total_tokens < 0 || nseq < 1 || nseq > 65535 || max_chunk < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 ||
        D < 1 || max_pages < 1 || num_pages < 1 || page_size != JT_PAGE_SIZE || !isfinite(scale) || !(scale > 0.0f) ||
        (dtype != JT_DTYPE_BF16 && dtype != JT_DTYPE_F32))
        return JT_ERR_INVALID;
    const bool bf16 = dtype == JT_DTYPE_BF16;
    const int G = Hq / Hkv;
    if (bf16 ? (D != 64 && D != 128) : (D != 32 && D != 64 && D != 96 && D != 128)) return JT_ERR_UNSUPPORTED;
    if (G > (bf16 ? 128 : 64)) return JT_ERR_UNSUPPORTED;
    if (!bf16 && static_cast<long long>(nseq) * Hkv * ((static_cast<long long>(max_chunk) + 64 / G - 1) / (64 / G)) >
                     0x7FFFFFFFll)
        return JT_ERR_UNSUPPORTED;
    if (total_tokens == 0) return JT_OK;
    if (!q || !k_cache || !v_cache || !block_table || !prefix_len || !chunk_off || !out || !aligned(q, 16) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
        return JT_ERR_INVALID;
    jt_status s = check_ws(ws, ws_bytes,
                           bf16 ? chunk_attn_bf16_workspace_bytes(D)
                                : chunk_attn_f32_need_bytes(nseq, Hq, Hkv, D, max_pages, max_chunk));
    if (s != JT_OK) return s;
    const int64_t bytes = static_cast<int64_t>(total_tokens) * Hq * D * (bf16 ? 2 : 4);
    // other CTAs may still read the queries, keys and values of a row written
    const int64_t pool = static_cast<int64_t>(num_pages) * JT_PAGE_SIZE * Hkv * D * (bf16 ? 2 : 4);
    const int64_t rows = lse ? static_cast<int64_t>(total_tokens) * Hq * 4 : 0;
    if (overlap(q, bytes, out, bytes) || overlap(out, bytes, k_cache, pool) || overlap(out, bytes, v_cache, pool) ||
        overlap(lse, rows, q, bytes) || overlap(lse, rows, out, bytes) || overlap(lse, rows, k_cache, pool) ||
        overlap(lse, rows, v_cache, pool))
        return JT_ERR_INVALID;
    ChunkArgs a;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.prefix_len = prefix_len;
    a.chunk_off = chunk_off;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.nseq = nseq;
    a.total = total_tokens;
    a.max_chunk = max_chunk;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    char* base = static_cast<char*>(ws);
    return from_cuda(bf16 ? chunk_attn_bf16_launch(a, base, stream) : chunk_attn_f32_launch(a, base, stream));
}

jt_status jt_kv_commit(void* k_cache, void* v_cache, int dtype, int layers, int64_t layer_stride,
                       const int32_t* block_table, int max_pages, int num_pages,
                       const int32_t* prefix_len, const int32_t* tree_off,
                       const int32_t* accept_len, const int32_t* path, int nseq, int N, int Hkv,
                       int D, int page_size, int32_t* new_prefix, void* ws, size_t ws_bytes,
                       jt_stream_t stream) {
    JT_RANGE("jt_kv_commit");
    if (!k_cache || !v_cache || !block_table || !prefix_len || !tree_off || !accept_len || !path || !new_prefix ||
        nseq < 1 || nseq > 65535 || N < 0 || N > JT_MAX_TREE || layers < 1 || layers > 65535 || max_pages < 1 ||
        num_pages < 1 || Hkv < 1 || D < 1 || page_size != JT_PAGE_SIZE ||
        (dtype != JT_DTYPE_BF16 && dtype != JT_DTYPE_F32))
        return JT_ERR_INVALID;
    const int64_t esize = dtype == JT_DTYPE_BF16 ? 2 : 4;
    const int64_t row = static_cast<int64_t>(Hkv) * D * esize;
    if (row % 16 != 0 || row > (1 << 24)) return JT_ERR_UNSUPPORTED;
    if (layers > 1 && (layer_stride < static_cast<int64_t>(num_pages) * JT_PAGE_SIZE * Hkv * D ||
                       layer_stride * esize % 16 != 0))
        return JT_ERR_INVALID;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return JT_ERR_INVALID;
    const int64_t n = static_cast<int64_t>(nseq) * static_cast<int64_t>(sizeof(int32_t));
    const bool in_place = new_prefix == prefix_len;
    if (!in_place && overlap(new_prefix, n, prefix_len, n)) return JT_ERR_INVALID;
    jt_status s = check_ws(ws, ws_bytes, in_place ? kv_commit_workspace_bytes(nseq) : kWsHeader);
    if (s != JT_OK) return s;
    // CTAs write new_prefix while others still read these (in place, all of them have been read by then)
    if (!in_place && (overlap(new_prefix, n, accept_len, n) || overlap(new_prefix, n, tree_off, n + 4) ||
                      overlap(new_prefix, n, path, n * (N + 1)) || overlap(new_prefix, n, block_table, n * max_pages)))
        return JT_ERR_INVALID;
    // two CTAs would move the same path
    if (layers_meet(k_cache, v_cache, static_cast<int64_t>(num_pages) * JT_PAGE_SIZE * row,
                    layers > 1 ? layer_stride * esize : 0, layers))
        return JT_ERR_INVALID;
    CommitArgs a;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.prefix_len = prefix_len;
    a.tree_off = tree_off;
    a.accept_len = accept_len;
    a.path = path;
    a.new_prefix = new_prefix;
    a.layer_stride = layers > 1 ? layer_stride * esize : 0;
    a.row_bytes = static_cast<int>(row);
    a.layers = layers;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.nseq = nseq;
    a.N = N;
    return from_cuda(kv_commit_launch(a, static_cast<char*>(ws), stream));
}

jt_status jt_call(int op, const void* args, size_t bytes) {
    struct Append {
        const void* qkv;
        int dtype;
        int64_t row_stride;
        const void* q_weight;
        const void* k_weight;
        float eps;
        const float* cos_sin;
        int max_pos, rot_dim, interleaved;
        const int32_t* depth;
        const int32_t* block_table;
        int max_pages, num_pages;
        const int32_t* prefix_len;
        const int32_t* tree_off;
        int nseq, total_nodes, Hq, Hkv, D, page_size;
        void* q_out;
        void* k_cache;
        void* v_cache;
        void* ws;
        size_t ws_bytes;
        jt_stream_t stream;
    };
    struct Chunk {
        const void* q;
        const void* k_cache;
        const void* v_cache;
        int dtype;
        const int32_t* block_table;
        int max_pages, num_pages;
        const int32_t* prefix_len;
        const int32_t* chunk_off;
        int nseq, total_tokens, max_chunk, Hq, Hkv, D, page_size;
        float scale;
        void* out;
        float* lse;
        void* ws;
        size_t ws_bytes;
        jt_stream_t stream;
    };
    struct Commit {
        void* k_cache;
        void* v_cache;
        int dtype, layers;
        int64_t layer_stride;
        const int32_t* block_table;
        int max_pages, num_pages;
        const int32_t* prefix_len;
        const int32_t* tree_off;
        const int32_t* accept_len;
        const int32_t* path;
        int nseq, N, Hkv, D, page_size;
        int32_t* new_prefix;
        void* ws;
        size_t ws_bytes;
        jt_stream_t stream;
    };
    if (!args) return JT_ERR_INVALID;
    if (op == JT_OP_QKV_APPEND && bytes == sizeof(Append)) {
        const Append& a = *static_cast<const Append*>(args);
        return jt_qkv_append(a.qkv, a.dtype, a.row_stride, a.q_weight, a.k_weight, a.eps, a.cos_sin, a.max_pos,
                             a.rot_dim, a.interleaved, a.depth, a.block_table, a.max_pages, a.num_pages, a.prefix_len,
                             a.tree_off, a.nseq, a.total_nodes, a.Hq, a.Hkv, a.D, a.page_size, a.q_out, a.k_cache,
                             a.v_cache, a.ws, a.ws_bytes, a.stream);
    }
    if (op == JT_OP_CHUNK_ATTN && bytes == sizeof(Chunk)) {
        const Chunk& a = *static_cast<const Chunk*>(args);
        return jt_chunk_attn_paged(a.q, a.k_cache, a.v_cache, a.dtype, a.block_table, a.max_pages, a.num_pages,
                                   a.prefix_len, a.chunk_off, a.nseq, a.total_tokens, a.max_chunk, a.Hq, a.Hkv, a.D,
                                   a.page_size, a.scale, a.out, a.lse, a.ws, a.ws_bytes, a.stream);
    }
    if (op == JT_OP_KV_COMMIT && bytes == sizeof(Commit)) {
        const Commit& a = *static_cast<const Commit*>(args);
        return jt_kv_commit(a.k_cache, a.v_cache, a.dtype, a.layers, a.layer_stride, a.block_table, a.max_pages,
                            a.num_pages, a.prefix_len, a.tree_off, a.accept_len, a.path, a.nseq, a.N, a.Hkv, a.D,
                            a.page_size, a.new_prefix, a.ws, a.ws_bytes, a.stream);
    }
    return JT_ERR_INVALID;
}

jt_status jt_check(void* ws, jt_stream_t stream) {
    JT_RANGE("jt_check");
    if (!ws) return JT_ERR_WORKSPACE;
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return JT_ERR_CUDA;
    uint32_t err = 0;
    e = cudaMemcpy(&err, ws, sizeof(err), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return JT_ERR_CUDA;
    if (err) {
        const uint32_t zero = 0;
        if (cudaMemcpy(ws, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess)
            return JT_ERR_CUDA;
    }
    if (err & DEVERR_TIMEOUT) return JT_ERR_TIMEOUT;
    if (err & DEVERR_INVALID) return JT_ERR_INVALID;
    return JT_OK;
}

}  // extern "C"
