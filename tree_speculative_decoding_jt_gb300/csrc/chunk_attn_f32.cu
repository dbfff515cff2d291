// chunk_attn_f32.cu -- causal attention of a ragged batch of new tokens over a
// paged fp32 KV cache on the CUDA cores (the tensor cores would round fp32
// operands to tf32).
//
// Same mathematics and layout as the bf16 path (chunk_attn.cu), everything in
// fp32.  A CTA holds 64 query rows (npt = 64 / G new tokens x the G query heads
// of one KV head) and walks 64-key tiles: S = Q K^T with 4 x 4 scores per
// thread from operands stored dim-major in shared memory, the online softmax on
// registers (16 threads share four rows), then O += P V with 4 rows x D / 16
// columns per thread.  The next K tile's loads are issued before the softmax
// and V arrives by cp.async during S, two CTAs per SM cover the rest.  With few
// units (a handful of single tokens) the keys of a unit are split over several
// CTAs and merged by chunk_f32_combine_kernel.  Bound: FMA issue (per SM 128
// FMA per clock) for chunks, and for single tokens the padding of G rows to 64.
#include <algorithm>

#include "jt_common.cuh"
#include "jt_internal.h"

namespace jt {
namespace chunk32 {

constexpr int kThreads = 256;
constexpr int kRows = 64;
constexpr int kKeys = 64;
constexpr int kPad = 68;  // floats per dim-major row of 64
constexpr int kMaxSplits = 32;

struct Params {
    const float* q;
    const float* k_cache;
    const float* v_cache;
    const int32_t* block_table;
    const int32_t* prefix_len;
    const int32_t* off;
    float* out;
    float* lse;
    float* part_o;    // [unit][split][64][D]
    float2* part_ml;  // [unit][split][64]
    uint32_t* err;
    int max_pages, num_pages, nseq, total, max_chunk, Hq, Hkv, G, npt, mtiles, splits;
    float scale;
};

struct SeqInfo {
    int L, B, off;
    bool ok;
};

__device__ __forceinline__ SeqInfo load_seq(const Params& p, int b) {
    SeqInfo s;
    s.off = p.off[b];
    s.B = p.off[b + 1] - s.off;
    s.L = p.prefix_len[b];
    s.ok = s.B >= 0 && s.B <= p.max_chunk && s.L >= 0 && s.off >= 0 && s.off <= p.total - s.B &&
           static_cast<long long>(s.L) + s.B <= min(static_cast<long long>(p.max_pages) * JT_PAGE_SIZE, 0x7FFFFF00ll);
    return s;
}

__device__ __forceinline__ void cp_async16(float* dst, const float* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <int D>
constexpr int smem_floats() {
    return D * kPad + (D > 64 ? D : 64) * kPad + kKeys * D;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) chunk_f32_kernel(const Params p) {
    constexpr int kV2 = D / 32;  // float2 columns of O per thread: 2 tx + 32 j
    extern __shared__ float smem[];
    float* Qs = smem;                              // [D][kPad]
    float* Ks = Qs + D * kPad;                     // [D][kPad]; then P as [key][kPad]
    float* Vs = Ks + (D > 64 ? D : 64) * kPad;     // [64][D]
    pdl_wait();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int u = blockIdx.x, mt = u % p.mtiles, g = u / p.mtiles % p.Hkv, b = u / (p.mtiles * p.Hkv);
    const SeqInfo s = load_seq(p, b);
    if (!s.ok) {
        if (tid == 0 && g == 0 && mt == 0 && blockIdx.y == 0) raise_error(p.err, DEVERR_INVALID);
        return;
    }
    const int tok0 = mt * p.npt;
    if (tok0 >= s.B) return;
    const int rows = min(s.B - tok0, p.npt) * p.G;
    const int end = s.L + min(s.B, tok0 + p.npt);  // keys that the tile's last token sees
    const int T = (end + kKeys - 1) / kKeys;
    const int tps = (T + p.splits - 1) / p.splits;
    const int t0 = blockIdx.y * tps, t1 = min(T, t0 + tps);
    if (t0 >= T) return;

    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), f = i % (D / 4);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < rows)
            v = *reinterpret_cast<const float4*>(
                p.q + (static_cast<long long>(s.off + tok0 + r / p.G) * p.Hq + g * p.G + r % p.G) * D + 4 * f);
        Qs[(4 * f + 0) * kPad + r] = v.x * p.scale;
        Qs[(4 * f + 1) * kPad + r] = v.y * p.scale;
        Qs[(4 * f + 2) * kPad + r] = v.z * p.scale;
        Qs[(4 * f + 3) * kPad + r] = v.w * p.scale;
    }

    const int key = tid >> 2, f0 = tid & 3;  // this thread's key of a tile, its first 16-byte piece
    float4 kreg[D / 16];
    bool bad_page = false;
    // offset of this thread's key of tile t in the cache, or -1 past the end
    auto key_base = [&](int t) -> long long {
        const int slot = t * kKeys + key;
        if (slot >= end) return -1;
        const long long page = p.block_table[static_cast<long long>(b) * p.max_pages + slot / JT_PAGE_SIZE];
        if (page < 0 || page >= p.num_pages) {
            bad_page = true;
            return -1;
        }
        return ((page * JT_PAGE_SIZE + slot % JT_PAGE_SIZE) * p.Hkv + g) * D;
    };
    auto load_k = [&](long long base) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            kreg[i] = base < 0 ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                               : *reinterpret_cast<const float4*>(p.k_cache + base + 4 * (f0 + 4 * i));
    };
    float m[4], l[4], acc[4][kV2][2];
    int limit[4];  // a row sees the slots below this
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
        limit[i] = s.L + tok0 + min(4 * ty + i, rows - 1) / p.G + 1;
#pragma unroll
        for (int j = 0; j < kV2; ++j) acc[i][j][0] = acc[i][j][1] = 0.0f;
    }
    long long base = key_base(t0);
    load_k(base);
    for (int t = t0; t < t1; ++t) {
        __syncthreads();  // the previous tile's P and V have been read
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const int d = 4 * (f0 + 4 * i);
            Ks[(d + 0) * kPad + key] = kreg[i].x;
            Ks[(d + 1) * kPad + key] = kreg[i].y;
            Ks[(d + 2) * kPad + key] = kreg[i].z;
            Ks[(d + 3) * kPad + key] = kreg[i].w;
        }
        float* vrow = Vs + key * D;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const int d = 4 * (f0 + 4 * i);
            if (base >= 0)
                cp_async16(vrow + d, p.v_cache + base + d);
            else
                *reinterpret_cast<float4*>(vrow + d) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        __syncthreads();
        float sc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[i][j] = 0.0f;
#pragma unroll 8
        for (int d = 0; d < D; ++d) {
            const float4 a = *reinterpret_cast<const float4*>(Qs + d * kPad + 4 * ty);
            const float4 c = *reinterpret_cast<const float4*>(Ks + d * kPad + 4 * tx);
            const float av[4] = {a.x, a.y, a.z, a.w}, cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[i][j] = fmaf(av[i], cv[j], sc[i][j]);
        }
        if (t + 1 < t1) {  // the next tile's keys are on their way during the softmax and P V
            base = key_base(t + 1);
            load_k(base);
        }
        const int slot0 = t * kKeys;
        const bool masked = slot0 + kKeys > s.L + tok0 + 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (masked && slot0 + 4 * tx + j >= limit[i]) sc[i][j] = -INFINITY;
                mx = fmaxf(mx, sc[i][j]);
            }
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            const float mn = fmaxf(m[i], mx);
            const float corr = m[i] == -INFINITY ? 0.0f : expf(m[i] - mn);
            m[i] = mn;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sc[i][j] = sc[i][j] == -INFINITY ? 0.0f : expf(sc[i][j] - mn);
                sum += sc[i][j];
            }
            l[i] = l[i] * corr + sum;  // this thread's keys only; summed over the 16 at the end
#pragma unroll
            for (int j = 0; j < kV2; ++j) {
                acc[i][j][0] *= corr;
                acc[i][j][1] *= corr;
            }
        }
        __syncthreads();  // the scores are in registers: P takes the keys' place
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float4*>(Ks + (4 * tx + j) * kPad + 4 * ty) =
                make_float4(sc[0][j], sc[1][j], sc[2][j], sc[3][j]);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        if (!masked) {
#pragma unroll 4
            for (int k = 0; k < kKeys; ++k) {
                const float4 a = *reinterpret_cast<const float4*>(Ks + k * kPad + 4 * ty);
                const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int j = 0; j < kV2; ++j) {
                    const float2 v = *reinterpret_cast<const float2*>(Vs + k * D + 2 * tx + 32 * j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[i][j][0] = fmaf(av[i], v.x, acc[i][j][0]);
                        acc[i][j][1] = fmaf(av[i], v.y, acc[i][j][1]);
                    }
                }
            }
        } else {
            // a key that a row does not see adds nothing even where its value is not finite
            for (int k = 0; k < kKeys; ++k) {
                const float4 a = *reinterpret_cast<const float4*>(Ks + k * kPad + 4 * ty);
                const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int j = 0; j < kV2; ++j) {
                    const float2 v = *reinterpret_cast<const float2*>(Vs + k * D + 2 * tx + 32 * j);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (slot0 + k < limit[i]) {
                            acc[i][j][0] = fmaf(av[i], v.x, acc[i][j][0]);
                            acc[i][j][1] = fmaf(av[i], v.y, acc[i][j][1]);
                        }
                }
            }
        }
    }
    if (bad_page) raise_error(p.err, DEVERR_INVALID);
    const bool partial = tps < T;
    const long long part = (static_cast<long long>(u) * p.splits + blockIdx.y) * kRows;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], o);
        const int r = 4 * ty + i;
        if (r >= rows) continue;
        if (partial) {
            if (tx == 0) p.part_ml[part + r] = make_float2(m[i], l[i]);
#pragma unroll
            for (int j = 0; j < kV2; ++j)
                *reinterpret_cast<float2*>(p.part_o + (part + r) * D + 2 * tx + 32 * j) =
                    make_float2(acc[i][j][0], acc[i][j][1]);
        } else {
            const long long rowid =
                static_cast<long long>(s.off + tok0 + r / p.G) * p.Hq + g * p.G + r % p.G;
            const float inv = 1.0f / l[i];
            if (tx == 0 && p.lse) p.lse[rowid] = m[i] + logf(l[i]);
#pragma unroll
            for (int j = 0; j < kV2; ++j)
                *reinterpret_cast<float2*>(p.out + rowid * D + 2 * tx + 32 * j) =
                    make_float2(acc[i][j][0] * inv, acc[i][j][1] * inv);
        }
    }
}

// One warp per query row of a split unit: lane k holds split k's (m, l).
template <int D>
__global__ void __launch_bounds__(kThreads) chunk_f32_combine_kernel(const Params p) {
    constexpr int kC = D / 32;
    pdl_wait();
    const int u = blockIdx.x, mt = u % p.mtiles, g = u / p.mtiles % p.Hkv, b = u / (p.mtiles * p.Hkv);
    const SeqInfo s = load_seq(p, b);
    const int tok0 = mt * p.npt;
    if (!s.ok || tok0 >= s.B) return;
    const int rows = min(s.B - tok0, p.npt) * p.G;
    const int T = (s.L + min(s.B, tok0 + p.npt) + kKeys - 1) / kKeys;
    const int tps = (T + p.splits - 1) / p.splits;
    const int n = (T + tps - 1) / tps;
    const int r = blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (n <= 1 || r >= rows) return;
    auto row = [&](int k) { return (static_cast<long long>(u) * p.splits + k) * kRows + r; };
    const float2 ml = lane < n ? p.part_ml[row(lane)] : make_float2(-INFINITY, 0.0f);
    float M = ml.x;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    const float w = ml.x == -INFINITY ? 0.0f : expf(ml.x - M);
    float l = w * ml.y;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    float acc[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = 0.0f;
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
        const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
        if (wk != 0.0f)
#pragma unroll
            for (int c = 0; c < kC; ++c) acc[c] = fmaf(wk, p.part_o[row(k) * D + lane + 32 * c], acc[c]);
    }
    const long long rowid = static_cast<long long>(s.off + tok0 + r / p.G) * p.Hq + g * p.G + r % p.G;
#pragma unroll
    for (int c = 0; c < kC; ++c) p.out[rowid * D + lane + 32 * c] = acc[c] / l;
    if (lane == 0 && p.lse) p.lse[rowid] = M + logf(l);
}

struct Plan {
    int npt, mtiles, splits;
    long long units;
};

// Keys are split when the units (a dense count: shorter chunks leave some of
// them empty) are fewer than eight rounds of the CTA slots, two per SM, at most
// one split per four key tiles.  A key tile takes a CTA about 5 us, so a ragged
// batch's longest unit sets the time: 4 sequences of 16 to 512 tokens over 128 to
// 1500 (8/2 heads, D 64) took 204 us with splits for less than one round only, and
// take 86 (21 TFLOP/s of the visible pairs).
static long long rounds() { return 16ll * std::max(1, device_sm_count()); }
static long long max_splits(int max_pages) {
    const long long tmax = (static_cast<long long>(max_pages) * JT_PAGE_SIZE + kKeys - 1) / kKeys;
    return std::min(tmax / 4, static_cast<long long>(kMaxSplits));
}
static Plan plan(int nseq, int Hq, int Hkv, int max_pages, int max_chunk) {
    Plan pl;
    pl.npt = std::max(1, kRows / (Hq / Hkv));
    pl.mtiles = (max_chunk - 1) / pl.npt + 1;  // max_chunk may be INT_MAX
    pl.units = static_cast<long long>(nseq) * Hkv * pl.mtiles;
    pl.splits = static_cast<int>(std::max(1ll, std::min(rounds() / std::max(1ll, pl.units), max_splits(max_pages))));
    return pl;
}

template <int D>
static cudaError_t launch(const ChunkArgs& a, char* ws, cudaStream_t st) {
    const Plan pl = plan(a.nseq, a.Hq, a.Hkv, a.max_pages, a.max_chunk);
    Params prm;
    prm.q = static_cast<const float*>(a.q);
    prm.k_cache = static_cast<const float*>(a.k_cache);
    prm.v_cache = static_cast<const float*>(a.v_cache);
    prm.block_table = a.block_table;
    prm.prefix_len = a.prefix_len;
    prm.off = a.chunk_off;
    prm.out = static_cast<float*>(a.out);
    prm.lse = a.lse;
    prm.part_ml = reinterpret_cast<float2*>(ws + kChunkFixedBytes);
    prm.part_o = reinterpret_cast<float*>(
        ws + kChunkFixedBytes + align_up(static_cast<size_t>(pl.units) * pl.splits * kRows * sizeof(float2)));
    prm.err = reinterpret_cast<uint32_t*>(ws);
    prm.max_pages = a.max_pages;
    prm.num_pages = a.num_pages;
    prm.nseq = a.nseq;
    prm.total = a.total;
    prm.max_chunk = a.max_chunk;
    prm.Hq = a.Hq;
    prm.Hkv = a.Hkv;
    prm.G = a.Hq / a.Hkv;
    prm.npt = pl.npt;
    prm.mtiles = pl.mtiles;
    prm.splits = pl.splits;
    prm.scale = a.scale;
    constexpr size_t smem = smem_floats<D>() * sizeof(float);
    static PerDeviceCache attr;
    const cudaError_t ea = static_cast<cudaError_t>(attr.get([] {
        return static_cast<int>(cudaFuncSetAttribute(chunk_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(smem_floats<D>() * sizeof(float))));
    }));
    if (ea != cudaSuccess) return ea;
    cudaError_t e = launch_kernel_pdl(chunk_f32_kernel<D>, dim3(static_cast<unsigned>(pl.units), pl.splits),
                                      dim3(kThreads), smem, st, prm);
    if (e != cudaSuccess || pl.splits == 1) return e;
    return launch_kernel_pdl(chunk_f32_combine_kernel<D>,
                             dim3(static_cast<unsigned>(pl.units), kRows / (kThreads / 32)), dim3(kThreads), 0, st,
                             prm);
}

}  // namespace chunk32

static size_t f32_bytes(long long splits, int D) {  // partial results of `splits` (unit, split) tiles
    const size_t rows = static_cast<size_t>(splits) * chunk32::kRows;
    return kChunkFixedBytes + align_up(rows * sizeof(float2)) + align_up(rows * D * sizeof(float));
}

size_t chunk_attn_f32_need_bytes(int nseq, int Hq, int Hkv, int D, int max_pages, int max_chunk) {
    const chunk32::Plan pl = chunk32::plan(nseq, Hq, Hkv, max_pages, max_chunk);
    return pl.splits == 1 ? kChunkFixedBytes : f32_bytes(pl.units * pl.splits, D);
}

// A call with fewer units splits them further, so its need can be the larger one.
// What is reported covers every call with at most these sequences, pages and
// chunk lengths: units * splits is at most rounds() and at most units * max_splits.
size_t chunk_attn_f32_workspace_bytes(int nseq, int Hq, int Hkv, int D, int max_pages, int max_chunk) {
    const long long per = chunk32::max_splits(max_pages);
    if (per < 2) return kChunkFixedBytes;
    const long long units = std::min(chunk32::plan(nseq, Hq, Hkv, max_pages, max_chunk).units, chunk32::rounds());
    return f32_bytes(std::min(units * per, chunk32::rounds()), D);
}

cudaError_t chunk_attn_f32_launch(const ChunkArgs& a, char* ws, cudaStream_t st) {
    switch (a.D) {
        case 32: return chunk32::launch<32>(a, ws, st);
        case 64: return chunk32::launch<64>(a, ws, st);
        case 96: return chunk32::launch<96>(a, ws, st);
        case 128: return chunk32::launch<128>(a, ws, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace jt
