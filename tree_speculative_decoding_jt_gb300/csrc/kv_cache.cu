// kv_cache.cu -- the writers of the paged KV cache: new tokens' keys and values
// (with the per-head norm and the position rotation on the way), and the move
// of an accepted path's keys and values behind the prefix.
#include <algorithm>

#include "jt_common.cuh"
#include "jt_internal.h"

namespace jt {
namespace kv {

// ---------------------------------------------------------------------------
// qkv_append: per token i of sequence b and head h of the packed projection
//     y = x * rsqrt(mean(x^2) + eps) * w         (q and k heads, with weights)
//     (a, b) -> (a cos - b sin, b cos + a sin)   (q and k heads, rotated pairs)
// fp32 throughout, one rounding; q goes to q_out, k and v to slot L_b + i.
//
// A head vector is shared by LPH lanes; a lane holds kPairs rotation pairs, as
// two 16-byte vectors: elements (j, j + rot/2) of the half-split layout or (2j,
// 2j + 1) of the interleaved one, and the plain rest in order.  So the rotation
// needs no exchange between lanes and the norm one sum over LPH.  A warp stays
// with one token: its angles sit in registers for all heads, four heads' loads
// are in flight per lane.  Bound: HBM bytes (one read, one write of every
// element) for many tokens, a chain of dependent loads (offsets, prefix, page,
// row) for one.  Measured (32/8 heads, D 128; data from HBM): 22610 tokens 100 us,
// 5.7 TB/s; 8 trees of 256 nodes 13.4 us, 3.8 TB/s (9.7 us where the 51 MB are in
// the L2 already); one token 2.3 us.
// ---------------------------------------------------------------------------
struct Append {
    const void* qkv;
    const void* q_weight;
    const void* k_weight;
    const float* cos_sin;
    const int32_t* depth;
    const int32_t* block_table;
    const int32_t* prefix_len;
    const int32_t* off;
    void* q_out;
    void* k_cache;
    void* v_cache;
    uint32_t* err;
    long long row_stride;
    int max_pos, rot, interleaved, max_pages, num_pages, nseq, total, Hq, Hkv, warps_per_token;
    float eps;
};

// Two 16-byte vectors of a lane as N rotation pairs (a[j], b[j]) in fp32, and
// back (rounded to the type): the halves of the vectors, or (kInter) neighbours.
template <typename T, bool kInter>
struct Pairs;
template <bool kInter>
struct Pairs<float, kInter> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4& u, const uint4& v, float (&a)[4], float (&b)[4]) {
        const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = __uint_as_float(w[kInter ? 2 * j : j]);
            b[j] = __uint_as_float(w[kInter ? 2 * j + 1 : 4 + j]);
        }
    }
    static __device__ __forceinline__ void pack(const float (&a)[4], const float (&b)[4], uint4& u, uint4& v) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[kInter ? 2 * j : j] = __float_as_uint(a[j]);
            w[kInter ? 2 * j + 1 : 4 + j] = __float_as_uint(b[j]);
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
        v = make_uint4(w[4], w[5], w[6], w[7]);
    }
};
template <bool kInter>
struct Pairs<__nv_bfloat16, kInter> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4& u, const uint4& v, float (&a)[8], float (&b)[8]) {
        const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xFFFF0000u);
            if (kInter)
                a[j] = lo, b[j] = hi;
            else if (j < 4)
                a[2 * j] = lo, a[2 * j + 1] = hi;
            else
                b[2 * j - 8] = lo, b[2 * j - 7] = hi;
        }
    }
    static __device__ __forceinline__ void pack(const float (&a)[8], const float (&b)[8], uint4& u, uint4& v) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = kInter    ? pack_bf16x2(a[j], b[j])
                   : j < 4 ? pack_bf16x2(a[(2 * j) & 7], a[(2 * j + 1) & 7])
                           : pack_bf16x2(b[(2 * j) & 7], b[(2 * j + 1) & 7]);
        u = make_uint4(w[0], w[1], w[2], w[3]);
        v = make_uint4(w[4], w[5], w[6], w[7]);
    }
};

// Packed fp32 pair arithmetic: half the instructions of the scalar forms.
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

// The last sequence whose offset is at most i (one warp; a few steps of 32).
__device__ __forceinline__ int find_seq(const int32_t* off, int nseq, int i, int lane) {
    int lo = 0, n = nseq;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool le = lane * step < n && off[lo + lane * step] <= i;
        const int k = 31 - __clz(__ballot_sync(0xFFFFFFFFu, le) | 1u);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

constexpr int kAppendThreads = 128;
constexpr int kUnroll = 4;  // heads in flight per lane group

template <typename T, int D, int LPH, bool kInter>
__global__ void __launch_bounds__(kAppendThreads) qkv_append_kernel(const Append p) {
    using P = Pairs<T, kInter>;
    constexpr int N = P::N;                   // pairs per lane
    constexpr int kActive = D / 2 / N;        // lanes of a head that hold elements
    constexpr int kHeads = 32 / LPH;          // heads per warp at a time
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long gw = static_cast<long long>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int i = static_cast<int>(gw / p.warps_per_token), part = static_cast<int>(gw % p.warps_per_token);
    if (i >= p.total) return;
    const int t = lane % LPH;
    const bool on = kActive == LPH || t < kActive;
    const int p0 = t * N;  // first of this lane's pairs
    const bool rotated = on && p0 < p.rot / 2;
    const bool split = rotated && !kInter;
    const int e0 = on ? (split ? p0 : 2 * p0) : 0, e1 = on ? (split ? p.rot / 2 + p0 : 2 * p0 + N) : 0;
    const T* row = static_cast<const T*>(p.qkv) + i * p.row_stride;
    const int H = p.Hq + 2 * p.Hkv;
    const int hstep = p.warps_per_token * kHeads;
    int h0 = part * kHeads + lane / LPH;
    uint4 va[kUnroll], vb[kUnroll];
    auto load = [&](int h) {
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
            va[q] = vb[q] = make_uint4(0u, 0u, 0u, 0u);
            if (on && h + q * hstep < H) {
                va[q] = __ldcs(reinterpret_cast<const uint4*>(row + static_cast<long long>(h + q * hstep) * D + e0));
                vb[q] = __ldcs(reinterpret_cast<const uint4*>(row + static_cast<long long>(h + q * hstep) * D + e1));
            }
        }
    };
    // The first heads are on their way while the chain offsets -> sequence ->
    // prefix -> page, angles is walked (rows behind the last token are in the
    // array too; they are dropped below).
    load(h0);
    if (i >= p.off[p.nseq]) return;
    const int b = find_seq(p.off, p.nseq, i, lane);
    const int o = p.off[b], B = p.off[b + 1] - o, L = p.prefix_len[b], local = i - o;
    const long long slot = static_cast<long long>(L) + local;
    const int step = p.depth ? p.depth[i] : local;
    const long long pos = static_cast<long long>(L) + step;
    bool ok = o >= 0 && local >= 0 && local < B && o <= p.total - B && L >= 0 &&
              static_cast<long long>(L) + B <= static_cast<long long>(p.max_pages) * JT_PAGE_SIZE &&
              (p.rot == 0 || (step >= 0 && pos < p.max_pos));
    int page = 0;
    if (ok) {
        page = p.block_table[static_cast<long long>(b) * p.max_pages + slot / JT_PAGE_SIZE];
        ok = page >= 0 && page < p.num_pages;
    }
    if (!ok) {
        if (lane == 0) raise_error(p.err, DEVERR_INVALID);
        return;
    }
    int kind = 0;  // the heads that the matrices are for: 1 q, 2 k
    float ca[N], sb[N], cb[N], sa[N];
    const float* angles = p.cos_sin + pos * p.rot + p0;
    const long long cache_row = (static_cast<long long>(page) * JT_PAGE_SIZE + slot % JT_PAGE_SIZE) * p.Hkv;
    while (__any_sync(0xFFFFFFFFu, h0 < H)) {
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
            const int h = h0 + q * hstep;
            if (!__any_sync(0xFFFFFFFFu, h < H)) break;
            const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
            const T* wt = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
            // The norm's weight and the rotation as one matrix per pair: a' = a
            // ca - b sb, b' = b cb + a sa, worked out once for the q and once
            // for the k heads of the token.
            if (on && !is_v && kind != (is_q ? 1 : 2)) {
                kind = is_q ? 1 : 2;
                float wa[N], wb[N];
#pragma unroll
                for (int j = 0; j < N; ++j) wa[j] = wb[j] = 1.0f;
                if (wt) {
                    const uint4 u = *reinterpret_cast<const uint4*>(wt + e0), v = *reinterpret_cast<const uint4*>(wt + e1);
                    P::unpack(u, v, wa, wb);
                }
#pragma unroll
                for (int j = 0; j < N; ++j) ca[j] = wa[j], cb[j] = wb[j], sa[j] = sb[j] = 0.0f;
                if (rotated) {
#pragma unroll
                    for (int j = 0; j < N; j += 4) {
                        const float4 c = *reinterpret_cast<const float4*>(angles + j);
                        const float4 sn = *reinterpret_cast<const float4*>(angles + p.rot / 2 + j);
                        const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            ca[j + k] = wa[j + k] * cv[k];
                            cb[j + k] = wb[j + k] * cv[k];
                            sa[j + k] = wa[j + k] * sv[k];
                            sb[j + k] = -wb[j + k] * sv[k];
                        }
                    }
                }
            }
            float ss = 0.0f;
            float fa[N], fb[N];
            P::unpack(va[q], vb[q], fa, fb);
            if (wt) {
                float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                for (int j = 0; j < N; j += 2) {
                    fma2(s0, s1, fa[j], fa[j + 1], fa[j], fa[j + 1], s0, s1);
                    fma2(s0, s1, fb[j], fb[j + 1], fb[j], fb[j + 1], s0, s1);
                }
                ss = s0 + s1;
            }
            if (p.q_weight || p.k_weight)
#pragma unroll
                for (int d = LPH / 2; d >= 1; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
            if (!on || h >= H) continue;
            T* dst = is_q ? static_cast<T*>(p.q_out) + (static_cast<long long>(i) * p.Hq + h) * D
                          : static_cast<T*>(is_v ? p.v_cache : p.k_cache) +
                                (cache_row + (is_v ? h - p.Hq - p.Hkv : h - p.Hq)) * D;
            if (!is_v && (wt || rotated)) {
                const float inv = wt ? rsqrtf(ss * (1.0f / D) + p.eps) : 1.0f;
#pragma unroll
                for (int j = 0; j < N; j += 2) {
                    float x0, x1, y0, y1;
                    mul2(x0, x1, fa[j], fa[j + 1], ca[j], ca[j + 1]);
                    mul2(y0, y1, fb[j], fb[j + 1], cb[j], cb[j + 1]);
                    if (rotated) {  // elsewhere 0 times an infinity would reach the neighbour
                        fma2(x0, x1, fb[j], fb[j + 1], sb[j], sb[j + 1], x0, x1);
                        fma2(y0, y1, fa[j], fa[j + 1], sa[j], sa[j + 1], y0, y1);
                    }
                    mul2(fa[j], fa[j + 1], x0, x1, inv, inv);
                    mul2(fb[j], fb[j + 1], y0, y1, inv, inv);
                }
                P::pack(fa, fb, va[q], vb[q]);
            }
            *reinterpret_cast<uint4*>(dst + e0) = va[q];
            *reinterpret_cast<uint4*>(dst + e1) = vb[q];
        }
        h0 += hstep * kUnroll;
        if (__any_sync(0xFFFFFFFFu, h0 < H)) load(h0);
    }
}

template <typename T, int D>
static cudaError_t append_launch(Append prm, cudaStream_t st) {
    constexpr int active = D / 2 / Pairs<T, false>::N;
    constexpr int LPH = active <= 4 ? 4 : active <= 8 ? 8 : 16;
    static_assert(active <= 16, "head dim");
    const int H = prm.Hq + 2 * prm.Hkv, per = 32 / LPH;
    // A token's heads go to as many warps as it takes to have about twelve warps
    // per SM at work.  Many tokens get one warp each: the token's offsets, page
    // and angles are looked up once, and its heads are read four per lane group
    // at a time (22610 tokens of 32/8 heads, D 128: 98 us with one warp a token,
    // 110 with two, 117 with three).  Few tokens get up to one lane group per
    // head (761 tokens of 12/4 heads, D 96, fp32, data in the L2: 6.2 us with one,
    // 4.7 with three).
    const long long fine = (H + per - 1) / per;
    prm.warps_per_token = static_cast<int>(
        std::max(1ll, std::min(fine, (12ll * device_sm_count() + prm.total - 1) / prm.total)));
    const long long warps = static_cast<long long>(prm.total) * prm.warps_per_token;
    const long long blocks = (warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    return launch_kernel_pdl(
        prm.interleaved ? qkv_append_kernel<T, D, LPH, true> : qkv_append_kernel<T, D, LPH, false>,
        dim3(static_cast<unsigned>(blocks)), dim3(kAppendThreads), 0, st, prm);
}

// ---------------------------------------------------------------------------
// kv_commit: for d = 1 .. accept_len[b], slot L_b + d <- slot L_b + path[b, d]
// in every layer, K and V; new_prefix[b] = L_b + accept_len[b] + 1.
//
// The path rises strictly, so path[d] >= d and a step's source is never a slot
// that an earlier step wrote unless it is its own target: walking d upwards in
// place is safe, and so is loading a batch of steps before storing it.  A slot's
// heads are one contiguous row; a thread moves one 16-byte column of it, with
// the row offsets of the whole path worked out once per CTA.  grid (nseq,
// layer-halves): a CTA takes every gridDim.y-th of the 2 * layers caches.
// Bound: HBM bytes of the moved rows; for one sequence the chain accept_len ->
// path -> page -> row.  Measured (36 layers, 8 heads, D 128): 32 sequences, 40 MB,
// 9.5 us from HBM, 4.2 TB/s (6.2 us where they are in the L2); one sequence 2.2 us.
// ---------------------------------------------------------------------------
struct Commit {
    char* k_cache;
    char* v_cache;
    const int32_t* block_table;
    const int32_t* prefix_len;
    const int32_t* off;
    const int32_t* accept_len;
    const int32_t* path;
    int32_t* new_prefix;
    int32_t* staged;        // [nseq]: new lengths, when new_prefix is prefix_len
    uint32_t* err;
    uint32_t* arrivals;     // workspace header word, 0 between calls
    long long layer_stride;
    int row_bytes, layers, max_pages, num_pages, nseq, N, in_place;
};

constexpr int kCommitThreads = 128;
constexpr int kCommitBatch = 8;

__global__ void __launch_bounds__(kCommitThreads) kv_commit_kernel(const Commit p) {
    __shared__ long long src[JT_MAX_TREE], dst[JT_MAX_TREE];
    __shared__ int last;
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x, tid = threadIdx.x;
    const int acc = p.accept_len[b], L = p.prefix_len[b], B = p.off[b + 1] - p.off[b];
    const int32_t* path = p.path + static_cast<long long>(b) * (p.N + 1);
    bool ok = acc >= 0 && acc <= p.N && B >= 1 && B <= JT_MAX_TREE && acc < B && L >= 0 &&
              static_cast<long long>(L) + B <=
                  min(static_cast<long long>(p.max_pages) * JT_PAGE_SIZE, 0x7FFFFF00ll);
    if (ok) {
        const int32_t* table = p.block_table + static_cast<long long>(b) * p.max_pages;
        for (int d = tid; d <= acc; d += kCommitThreads) {
            const int node = path[d], before = d > 0 ? path[d - 1] : -1;
            if (node <= before || node >= B || (d == 0 && node != 0)) {
                ok = false;
            } else if (d > 0) {
                const int sp = table[(L + node) / JT_PAGE_SIZE], dp = table[(L + d) / JT_PAGE_SIZE];
                if (sp < 0 || sp >= p.num_pages || dp < 0 || dp >= p.num_pages) ok = false;
                src[d - 1] = (static_cast<long long>(sp) * JT_PAGE_SIZE + (L + node) % JT_PAGE_SIZE) * p.row_bytes;
                dst[d - 1] = (static_cast<long long>(dp) * JT_PAGE_SIZE + (L + d) % JT_PAGE_SIZE) * p.row_bytes;
            }
        }
    }
    ok = __syncthreads_and(ok);
    if (blockIdx.y == 0 && tid == 0) {
        if (!ok) raise_error(p.err, DEVERR_INVALID);
        if (p.in_place)
            p.staged[b] = ok ? L + acc + 1 : L;
        else if (ok)
            p.new_prefix[b] = L + acc + 1;
    }
    if (p.in_place && tid == 0) {
        // Every CTA has read its old length by the time it arrives: the last to
        // arrive may overwrite them, and leaves the count at 0 for the next call.
        __threadfence();
        const uint32_t n = gridDim.x * gridDim.y;
        last = atomicAdd(p.arrivals, 1u) == n - 1u;
        if (last) *p.arrivals = 0u;
        __threadfence();
    }
    if (ok) {
        for (int c = blockIdx.y; c < 2 * p.layers; c += gridDim.y) {
            char* cache = (c & 1 ? p.v_cache : p.k_cache) + (c >> 1) * p.layer_stride;
            for (int col = tid * 16; col < p.row_bytes; col += kCommitThreads * 16) {
                for (int d0 = 0; d0 < acc; d0 += kCommitBatch) {
                    uint4 v[kCommitBatch];
#pragma unroll
                    for (int k = 0; k < kCommitBatch; ++k)
                        if (d0 + k < acc && src[d0 + k] != dst[d0 + k])
                            v[k] = *reinterpret_cast<const uint4*>(cache + src[d0 + k] + col);
#pragma unroll
                    for (int k = 0; k < kCommitBatch; ++k)
                        if (d0 + k < acc && src[d0 + k] != dst[d0 + k])
                            *reinterpret_cast<uint4*>(cache + dst[d0 + k] + col) = v[k];
                }
            }
        }
    }
    if (p.in_place) {
        __syncthreads();
        if (last)
            for (int i = tid; i < p.nseq; i += kCommitThreads)
                p.new_prefix[i] = *static_cast<volatile int32_t*>(p.staged + i);
    }
}

}  // namespace kv

cudaError_t qkv_append_launch(const AppendArgs& a, uint32_t* err, cudaStream_t st) {
    kv::Append p;
    p.qkv = a.qkv;
    p.q_weight = a.q_weight;
    p.k_weight = a.k_weight;
    p.cos_sin = a.cos_sin;
    p.depth = a.depth;
    p.block_table = a.block_table;
    p.prefix_len = a.prefix_len;
    p.off = a.tree_off;
    p.q_out = a.q_out;
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.err = err;
    p.row_stride = a.row_stride;
    p.max_pos = a.max_pos;
    p.rot = a.rot_dim;
    p.interleaved = a.interleaved;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.nseq = a.nseq;
    p.total = a.total;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.warps_per_token = 1;
    p.eps = a.eps;
    if (a.dtype == JT_DTYPE_BF16) {
        if (a.D == 64) return kv::append_launch<__nv_bfloat16, 64>(p, st);
        if (a.D == 128) return kv::append_launch<__nv_bfloat16, 128>(p, st);
        return cudaErrorInvalidValue;
    }
    switch (a.D) {
        case 32: return kv::append_launch<float, 32>(p, st);
        case 64: return kv::append_launch<float, 64>(p, st);
        case 96: return kv::append_launch<float, 96>(p, st);
        case 128: return kv::append_launch<float, 128>(p, st);
        default: return cudaErrorInvalidValue;
    }
}

size_t kv_commit_workspace_bytes(int nseq) { return kWsHeader + align_up(static_cast<size_t>(nseq) * sizeof(int32_t)); }

cudaError_t kv_commit_launch(const CommitArgs& a, char* ws, cudaStream_t st) {
    kv::Commit p;
    p.k_cache = static_cast<char*>(a.k_cache);
    p.v_cache = static_cast<char*>(a.v_cache);
    p.block_table = a.block_table;
    p.prefix_len = a.prefix_len;
    p.off = a.tree_off;
    p.accept_len = a.accept_len;
    p.path = a.path;
    p.new_prefix = a.new_prefix;
    p.staged = reinterpret_cast<int32_t*>(ws + kWsHeader);
    p.err = reinterpret_cast<uint32_t*>(ws);
    p.arrivals = &reinterpret_cast<WsHeader*>(ws)->arrivals;
    p.layer_stride = a.layer_stride;
    p.row_bytes = a.row_bytes;
    p.layers = a.layers;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.nseq = a.nseq;
    p.N = a.N;
    p.in_place = a.new_prefix == a.prefix_len;
    // about 16 CTAs per SM: beyond that a CTA takes several caches, so that its
    // path's offsets serve more than one
    const int halves = 2 * a.layers;
    const int ctas = std::max(1, std::min(halves, 16 * device_sm_count() / std::max(1, a.nseq)));
    return launch_kernel_pdl(kv::kv_commit_kernel, dim3(a.nseq, std::min(ctas, 65535)), dim3(kv::kCommitThreads), 0, st,
                             p);
}

}  // namespace jt
