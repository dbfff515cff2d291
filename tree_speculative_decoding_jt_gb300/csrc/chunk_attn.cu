// chunk_attn.cu -- causal attention of a ragged batch of new tokens over a
// paged bf16 KV cache on the sm_103a tensor cores (tcgen05 + TMEM + TMA).
//
// Mathematics.  Sequence b has L_b cached tokens and B_b new ones, whose keys
// and values already sit in the slots L_b .. L_b + B_b - 1.  New token i sees
// the slots 0 .. L_b + i:
//     out = sum_s exp(scale q.k_s - m) v_s / l,  l = sum_s exp(scale q.k_s - m),
// one pass over the keys with the running maximum m and sum l (fp32), P =
// exp(...) rounded once to bf16 for the second product (at most 2^-8 relative, as
// the inputs are; l sums the unrounded values), the output rounded once.  The
// product takes operands of one type, so P held finer would mean V in two parts and
// twice the MMAs; a prompt is bound by the chain that they are part of.
//
// Work.  A unit is (sequence b, KV head g, query-tile pair mp): two 128-row
// query tiles of npt = 128 / G new tokens x the G query heads of KV head g
// (stacked in the MMA's M dimension: they share K and V) against the 128-key
// tiles 0 .. T_u - 1 of the keys that the pair's last token sees.  A work slot
// is a pair of CTAs on two SMs (a cluster): CTA rank X takes query tile X, and
// one tcgen05.mma.cta_group::2 of M = 256 covers both.  Each CTA holds its half
// of every K tile (keys 64X..) and of every V tile (dims D/2 X..), so a unit's
// keys cross L2 once for 256 query rows.  All units' key tiles are laid end to
// end in (b, g, mp) order and cut into one equal range per work slot, planned
// on the device from prefix_len and chunk_off (sums over a head's units in
// closed form), so lengths never visit the host and every SM gets the same
// number of tiles.  A unit cut by a range boundary leaves fp32 partials; the
// slot that finishes its last piece merges them, summing in piece order.
//
// Warps per CTA (512 threads):
//   0-3 / 4-7  softmax of the tiles with even / odd number, one query row per
//              thread.  Warps w and w + 4 hold the same 32 rows, and each warp
//              has two tiles' time for one tile's softmax.  P of all tiles of a
//              row is relative to one maximum m: each warp keeps the m it knows
//              and its own part of the sum, and tells the other m after every
//              tile.  m is the first tile's maximum, rounded up to a whole number
//              of log2 units and raised only when a later score exceeds it by
//              2^32: P, O and l then stay far inside fp32, with no loss of relative
//              precision, a change of m scales by powers of two, and the partner's
//              m is not on the way of a tile's exponentials.  Warps whose rows are all past
//              the chunk's end (single tokens fill 1 to 16 of 256 rows) compute
//              nothing.
//   8-11       epilogue: O of a piece to the output or to its partial, and the
//              merges, while the softmax warps are at the next piece's tiles;
//   12 / 14    TMA producers of Q and K / of V, one box per 16-token page;
//   13 / 15    in the pair's leader, the MMA issuers of O += P V and of S = Q K^T:
//              one warp for both spends longer on its waits, issues and commits
//              than the MMAs take (1163 us where two take 1123: 8192 tokens on
//              8192, 32/8 heads, D 128); 13 also allocates TMEM.
// TMEM (512 columns): S0, S1, S2 (P of a tile overwrites the first half of its
// S) and O.  S runs up to three tiles ahead of O, across units; Q is double
// buffered.
//
// What bounds it, measured (32/8 heads, D 128 unless said; flops of the visible
// (token, key) pairs, bytes read and written once):
//   8192 tokens on 8192           1075-1155 us, 1.43-1.53 PFLOP/s: the chain score
//     -> softmax -> P -> output MMA of a tile over three S buffers (1650 cycles a
//     tile where its MMAs take 1080);
//   16 sequences, 1 to 512 tokens on 1024 to 8192   200-215 us, 0.92-1.0 PFLOP/s: the
//     same, 0.11 of the work past the chunks' ends, and some 2.5 us a piece;
//   32 single tokens on 32768     653-713 us, 6.0-6.6 TB/s: HBM;
//   1 token on 4096               19.5 us from HBM, 18.4 from the L2: latency (plan, 3
//     or 4 tiles, merge);
//   D 64, 5 chunks of up to 1500  107 us: exponentials and pieces
// (ranges: from GPU to GPU, and replayed back to back or call by call).
// A tile's row maximum taken by the TMEM load itself, P released in halves, the
// exponential as a polynomial, scores in halves of 64 keys, and the piece cut by a
// range's end done first (its merge then amid the others) were slower or equal.
#include <algorithm>

#include "jt_common.cuh"
#include "jt_internal.h"

namespace jt {
namespace chunk {

constexpr int kThreads = 512;
// Registers: 128 a thread at launch; the softmax and epilogue warps take what
// the others give up: 256 * 136 + 128 * 160 + 128 * 80 = 512 * 128.
constexpr int kLaunchRegs = 65536 / kThreads;
constexpr int kSoftmaxRegs = 136, kEpilogueRegs = 160, kOtherRegs = 80;
// setmaxnreg.inc may not go below the launch's count, .dec not above it, and
// what the warps take must not exceed what the block was launched with.
static_assert(kSoftmaxRegs >= kLaunchRegs && kEpilogueRegs >= kLaunchRegs && kOtherRegs <= kLaunchRegs);
static_assert(kSoftmaxRegs % 8 == 0 && kEpilogueRegs % 8 == 0 && kOtherRegs % 8 == 0);
static_assert(256 * kSoftmaxRegs + 128 * kEpilogueRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs);
constexpr int kTileN = 128;  // keys per KV tile
constexpr int kTileM = 128;  // query rows per query tile
constexpr float kRescaleLog2 = 32.0f;
// Pieces whose rows' maxima and sums may wait for the epilogue.  A softmax warp
// writes its entry of piece n once it is through its own tiles, and in a piece of
// one tile one of the two warps of a row has none.  Tiles alternate, so the last
// tile that it has seen is at least the one before n's last, no earlier than the
// last tile e of piece n - 1.  S of that tile waited for the PV three tiles before,
// which lies in piece n - 4 or later (a piece has at least one tile), and the first
// PV of piece n - 4 waited until the epilogue had read piece n - 5.  So a warp is at
// most four pieces ahead of what the epilogue has read: five entries.
constexpr int kRing = 5;

struct Params {
    const int32_t* block_table;
    const int32_t* prefix_len;
    const int32_t* off;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_cache;
    const __nv_bfloat16* v_cache;
    __nv_bfloat16* out;
    float* lse;
    float* part_o;    // [2 * slots][2][128][D]: partial O of the pieces of cut units
    float2* part_ml;  // [2 * slots][2][128]: their running max (log2 units) and sum
    unsigned long long* tickets;    // CTA arrivals over all calls (workspace header)
    unsigned long long* merge_cnt;  // [slots][2]: (call number << 32) | pieces done
    uint32_t* err;
    int max_pages, num_pages, nseq, total, max_chunk, Hq, Hkv, G, npt;
    float scale_log2;
};

template <int D>
struct Smem {
    static constexpr int kChunks = D / 64;                  // 64-dim (128-byte) column blocks of Q and K
    static constexpr int kQChunk = kTileM * 128;            // 128 query rows x 64 dims
    static constexpr int kQBytes = kChunks * kQChunk;
    static constexpr int kKChunk = 64 * 128;                // 64 keys x 64 dims
    static constexpr int kKHalf = kChunks * kKChunk;        // this CTA's 64 keys
    static constexpr int kVRow = D;                         // bytes of this CTA's D / 2 dims of one key
    static constexpr int kVHalf = kTileN * kVRow;
    static constexpr int kKStages = D == 128 ? 4 : 6;
    static constexpr int kVStages = D == 128 ? 4 : 6;
    static constexpr int kQ = 0;                            // two Q tiles
    static constexpr int kK = kQ + 2 * kQBytes;
    static constexpr int kV = kK + kKStages * kKHalf;
    static constexpr int kStage = kV + kVStages * kVHalf;   // epilogue staging, 2 KB per warp
    static constexpr int kBar = kStage + 4 * 2048;
    static constexpr int kM = kBar + 1024;                  // [tile / 2 mod 2][warpgroup][row]: (tile + 1, maximum)
    static constexpr int kX = kM + 4096;                    // [piece mod kRing][warpgroup][row]: (maximum, sum)
    static constexpr int kW = kX + kRing * 2048;            // the softmax and epilogue warps' walks
    static constexpr int kBytes = kW + 2048;
    static constexpr int kAlloc = kBytes + 1024;            // room to align the base to 1024
};

constexpr int kMaxStages = 6;

struct Bars {
    uint64_t q_full[2];             // leader: both CTAs' Q tiles have landed
    uint64_t q_empty[2];            // every QK of the piece has completed
    uint64_t k_full[kMaxStages];    // leader: both halves of the stage's K tile have landed
    uint64_t k_empty[kMaxStages];   // QK of the stage's tile has completed
    uint64_t v_full[kMaxStages];    // leader: both halves of the stage's V tile have landed
    uint64_t v_empty[kMaxStages];   // PV of the stage's tile has completed
    uint64_t v_own[kMaxStages];     // this CTA's half of a unit-final V tile has landed
    uint64_t s_full[3];             // S buffer holds QK of its latest tile
    uint64_t p_full[3];             // leader: P of the tile in the S buffer, from 8 softmax warps
    uint64_t o_done[3];             // one phase per PV of a tile t with t mod 3 == index
    uint64_t o_free;                // leader: the pair's 8 epilogue warps have read the piece's O
    uint64_t mma_final;             // every MMA of the pair has completed (both issuers)
    uint64_t x_bar[kRing][4];       // warps w, w + 4 have left a piece's maxima and sums for the epilogue
    uint64_t msync;                 // this CTA's 4 epilogue warps meet (merge of a cut unit)
    uint32_t tmem_base;
    int abort;
    int w_b, w_g, w_mp, w_t, w_quota, w_P;
    uint32_t call_id;
    int merge_flag;
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

// ---------------------------------------------------------------------------
// The work plan
// ---------------------------------------------------------------------------
struct SeqInfo {
    int L, B, off;
    int np;  // query-tile pairs (0: no new token, -1: contents out of range)
};

__device__ __forceinline__ SeqInfo load_seq(const Params& p, int b) {
    SeqInfo s;
    s.off = p.off[b];
    s.B = p.off[b + 1] - s.off;
    s.L = p.prefix_len[b];
    const bool ok = s.B >= 0 && s.B <= p.max_chunk && s.L >= 0 && s.off >= 0 && s.off <= p.total - s.B &&
                    static_cast<long long>(s.L) + s.B <=
                        min(static_cast<long long>(p.max_pages) * JT_PAGE_SIZE, 0x7FFFFF00ll);
    s.np = !ok ? -1 : (s.B + 2 * p.npt - 1) / (2 * p.npt);
    return s;
}

// Keys needed by pair mp: those its last token sees.
__device__ __forceinline__ int unit_end(const SeqInfo& s, int mp, int npt) {
    return s.L + min(s.B, (mp + 1) * 2 * npt);
}
__device__ __forceinline__ int unit_tiles(const SeqInfo& s, int mp, int npt) {
    return static_cast<int>((static_cast<unsigned>(unit_end(s, mp, npt)) + kTileN - 1u) / kTileN);
}

// sum_{i=0}^{n-1} floor((a i + b) / m), by the Euclidean reduction of (a, m).
__device__ __noinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
    long long ans = 0;
    for (;;) {
        if (a >= m) {
            ans += static_cast<long long>(n) * (n - 1) / 2 * (a / m);
            a %= m;
        }
        if (b >= m) {
            ans += static_cast<long long>(n) * (b / m);
            b %= m;
        }
        const uint32_t y = a * n + b;  // a, b < m <= 256: no overflow for n < 2^23
        if (y < m) return ans;
        n = y / m;
        b = y % m;
        const uint32_t t = m;
        m = a;
        a = t;
    }
}

// Key tiles of the first k units of one KV head, k < np (each of 2 npt tokens).
__device__ __forceinline__ long long prefix_tiles(const SeqInfo& s, int k, int npt) {
    if (k <= 0) return 0;
    return floor_sum(static_cast<uint32_t>(k), kTileN, 2u * npt, static_cast<uint32_t>(s.L) + kTileN - 1u + 2u * npt);
}
__device__ __forceinline__ long long head_tiles(const SeqInfo& s, int npt) {
    if (s.np <= 0) return 0;
    return prefix_tiles(s, s.np - 1, npt) + unit_tiles(s, s.np - 1, npt);
}

// One piece: key tiles [t0, t0 + nt) of unit (b, g, mp), which has T tiles.
// slot: the partial slot the piece writes, or -1 when it is the whole unit.
struct Piece {
    SeqInfo s;
    int b, g, mp, t0, nt, T, slot;
    int gpos;  // global tile index of the piece's first tile
};

// Walks the pieces of one work slot's range in order; every role runs its own.
struct Walker {
    SeqInfo s;
    int b, g, mp, t, remaining, piece, gpos, work;

    __device__ __forceinline__ void init(const Params& p, const Bars* bars, int work_slot) {
        b = bars->w_b;
        g = bars->w_g;
        mp = bars->w_mp;
        t = bars->w_t;
        remaining = bars->w_quota;
        work = work_slot;
        gpos = work * bars->w_P;
        piece = 0;
        if (remaining > 0) s = load_seq(p, b);
    }

    __device__ __forceinline__ bool next(const Params& p, Piece& pc) {
        if (remaining <= 0) return false;
        const int T = unit_tiles(s, mp, p.npt);
        const int nt = min(T - t, remaining);
        pc.s = s;
        pc.b = b;
        pc.g = g;
        pc.mp = mp;
        pc.t0 = t;
        pc.nt = nt;
        pc.T = T;
        pc.slot = (t == 0 && nt == T) ? -1 : 2 * work + (piece == 0 ? 0 : 1);
        pc.gpos = gpos;
        gpos += nt;
        remaining -= nt;
        t += nt;
        ++piece;
        if (t == T && remaining > 0) {  // on to the next unit in (b, g, mp) order
            t = 0;
            if (++mp >= s.np) {
                mp = 0;
                if (++g >= p.Hkv) {
                    g = 0;
                    do {
                        ++b;
                        s = load_seq(p, b);
                    } while (s.np <= 0 && b + 1 < p.nseq);
                }
            }
        }
        return true;
    }
};

struct WarpWalk {
    Walker w;
    Piece pc;
};
static_assert(12 * sizeof(WarpWalk) <= 2048, "walk block");

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Key tiles of one KV head with every unit's rounded up to a multiple of P.
__device__ __forceinline__ int padded_head_tiles(const SeqInfo& s, int npt, int P) {
    int t = 0;
    for (int mp = 0; mp < s.np; ++mp) t += (unit_tiles(s, mp, npt) + P - 1) / P * P;
    return t;
}

// The planner (one warp): the range of work slot `work` (of nwork) and the unit
// and tile that it starts at.  Ranges are equal shares P of all tiles; with few
// units (at most half the slots) every unit starts at a range's start instead, P
// being large enough for the units' last ranges to be cut short: a slot then
// has one piece, and no slot the ends of two units one after the other (one
// token over 4096, 8 KV heads: 24 -> 19 us).  rec: also report the sequences
// whose offsets or lengths are out of range.
__device__ void plan_slot(const Params& p, Bars* bars, int lane, int work, int nwork, bool rec) {
    SeqInfo mine;  // the sequence of this lane in the batch's last 32
    mine.np = 0;
    long long total = 0, units = 0;
    for (int base = 0; base < p.nseq; base += 32) {
        const int b = base + lane;
        long long t = 0, u = 0;
        if (b < p.nseq) {
            mine = load_seq(p, b);
            if (mine.np < 0) {
                if (rec) raise_error(p.err, DEVERR_INVALID);
            } else {
                t = p.Hkv * head_tiles(mine, p.npt);
                u = static_cast<long long>(p.Hkv) * mine.np;
            }
        } else {
            mine.np = 0;
        }
        total += warp_sum(t);
        units += warp_sum(u);
    }
    if (total > 0x7FFF0000ll) {  // beyond the int tile arithmetic: refuse the launch's work
        if (rec && lane == 0) raise_error(p.err, DEVERR_INVALID);
        total = 0;
    }
    const int T_total = static_cast<int>(total);
    int P = T_total > 0 ? (T_total + nwork - 1) / nwork : 0;
    bool aligned = false;
    if (T_total > 0 && 2 * units <= nwork) {
        // sum of ceil(T_u / P) <= T_total / P + units <= nwork
        const int share = nwork - static_cast<int>(units);
        const int Pa = (T_total + share - 1) / share;
        if (Pa <= P + 6) {  // the end of a piece costs a slot about six tiles' time
            P = Pa;
            aligned = true;
        }
    }
    const long long start = static_cast<long long>(work) * P;
    int found_b = -1, found_rel = 0;
    long long acc = 0;
    for (int base = 0; base < p.nseq && T_total > 0 && found_b < 0; base += 32) {
        const int b = base + lane;
        long long t = 0;
        if (b < p.nseq) {
            if (p.nseq > 32) mine = load_seq(p, b);
            if (mine.np > 0)
                t = p.Hkv * (aligned ? static_cast<long long>(padded_head_tiles(mine, p.npt, P)) : head_tiles(mine, p.npt));
        }
        long long incl = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += u;
        }
        const long long excl = acc + incl - t;
        const bool here = t > 0 && start >= excl && start < excl + t;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, here);
        if (m) {
            const int src = __ffs(m) - 1;
            found_b = base + src;
            found_rel = static_cast<int>(start - __shfl_sync(0xFFFFFFFFu, excl, src));
        }
        acc += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    int quota = 0, g = 0, mp = 0, t = 0;
    if (found_b >= 0) {
        SeqInfo s;
        if (p.nseq > 32) {
            s = load_seq(p, found_b);
        } else {
            s.L = __shfl_sync(0xFFFFFFFFu, mine.L, found_b);
            s.B = __shfl_sync(0xFFFFFFFFu, mine.B, found_b);
            s.off = __shfl_sync(0xFFFFFFFFu, mine.off, found_b);
            s.np = __shfl_sync(0xFFFFFFFFu, mine.np, found_b);
        }
        if (aligned) {
            const int ht = padded_head_tiles(s, p.npt, P);
            g = found_rel / ht;
            t = found_rel - g * ht;
            for (;; ++mp) {
                const int T = unit_tiles(s, mp, p.npt), padded = (T + P - 1) / P * P;
                if (t < padded) {
                    quota = min(P, T - t);
                    break;
                }
                t -= padded;
            }
        } else {
            const int ht = static_cast<int>(head_tiles(s, p.npt));
            g = found_rel / ht;
            const int r = found_rel - g * ht;
            int n = s.np;  // the last unit in [mp, mp + n) that starts at or before tile r
            while (n > 1) {
                const int step = (n + 31) / 32;
                const bool le = lane * step < n && prefix_tiles(s, mp + lane * step, p.npt) <= r;
                const unsigned m = __ballot_sync(0xFFFFFFFFu, le);
                const int k = 31 - __clz(m | 1u);
                mp += k * step;
                n = min(step, n - k * step);
            }
            t = r - static_cast<int>(prefix_tiles(s, mp, p.npt));
            quota = static_cast<int>(min(static_cast<long long>(P), T_total - start));
        }
    }
    if (lane == 0) {
        bars->w_b = found_b;
        bars->w_g = g;
        bars->w_mp = mp;
        bars->w_t = t;
        bars->w_quota = quota;
        bars->w_P = P;
    }
}

// The slots holding the pieces of the unit that starts at global tile U and
// has T tiles (range length P): c0 .. c0 + n - 1; partial slot of piece k.
struct CutUnit {
    int c0, n, slot0;
    __device__ __forceinline__ CutUnit(int U, int T, int P) {
        c0 = U / P;
        n = (U + T - 1) / P - c0 + 1;
        slot0 = 2 * c0 + (U == c0 * P ? 0 : 1);
    }
    __device__ __forceinline__ int slot(int k) const { return k == 0 ? slot0 : 2 * (c0 + k); }
};

// Call numbers for the merge counts: the first CTA of a call draws
// kTicketQuantum - (CTAs - 1) tickets from the workspace's counter and every
// other CTA one, so all CTAs of a call compute the same ticket /
// kTicketQuantum, and counts left by earlier calls never need clearing.
constexpr unsigned long long kTicketQuantum = 1ull << 24;

__device__ __forceinline__ uint32_t draw_call_id(unsigned long long* tickets, bool first, unsigned ctas) {
    const unsigned long long t = atomicAdd(tickets, first ? kTicketQuantum - (ctas - 1u) : 1ull);
    return static_cast<uint32_t>(t / kTicketQuantum) + 1u;
}

// ---------------------------------------------------------------------------
// softmax helpers: one query row (128 scores) per thread
// ---------------------------------------------------------------------------
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Three-input maximum (one instruction on sm_100 and later).
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Packed fp32 pair arithmetic: (d0, d1) = (a0, a1) * (b0, b1) + (c0, c1), and the sum.
__device__ __forceinline__ void ffma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0,
                                      float c1) {
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void fadd2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// The softmax's code is kept small (loops over a row's chunks, masks out of
// line): unrolled over the whole row with the masks in place, it pushed itself and
// the MMA warp's loop out of the instruction caches, and a tile took 2000 cycles
// where its MMAs need 1080.  A chunk of 32 columns loads while the one before is
// worked on.

// Scores at or past column `visible` of this thread's row -> -inf, in tensor
// memory (a unit's last tiles only).
__device__ __noinline__ void mask_row(uint32_t tS, int visible) {
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        uint32_t c[32];
        tmem_ld32(tS + 32 * q, c);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (32 * q + i >= visible) c[i] = __float_as_uint(-INFINITY);
        tmem_st32(tS + 32 * q, c);
    }
    tmem_wait_st();
}

__device__ __forceinline__ void max_chunk(const uint32_t (&c)[32], float (&m)[4]) {
#pragma unroll
    for (int i = 0; i < 32; i += 2)
        m[(i >> 1) & 3] = fmax3(m[(i >> 1) & 3], __uint_as_float(c[i]), __uint_as_float(c[i + 1]));
}

// Maximum of this thread's score row.
__device__ __forceinline__ float row_max(uint32_t tS) {
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    uint32_t c[32], d[32];
    tmem_ld32(tS, c);
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        tmem_wait_ld();
        tmem_ld32(tS + 64 * h + 32, d);
        max_chunk(c, m);
        tmem_wait_ld();
        if (h == 0) tmem_ld32(tS + 64, c);
        max_chunk(d, m);
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// One chunk's exponentials: packed to bf16 pairs into 16 columns at tP, summed.
__device__ __forceinline__ void exp_chunk(const uint32_t (&c)[32], uint32_t tP, float sl2, float m, float (&a)[4]) {
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float x0, x1;
        ffma2(x0, x1, __uint_as_float(c[2 * i]), __uint_as_float(c[2 * i + 1]), sl2, sl2, -m, -m);
        const float e0 = ex2_approx(x0);
        const float e1 = ex2_approx(x1);
        const int k = 2 * (i & 1);
        fadd2(a[k], a[k + 1], a[k], a[k + 1], e0, e1);
        pk[i] = pack_bf16x2(e0, e1);
    }
    tmem_st16(tP, pk);
}

// P = exp2(s * sl2 - m), packed to bf16 pairs into the first 64 columns of the
// S region (chunk q writes columns 16 q .. 16 q + 15, which chunks up to q have
// been read from); returns the sum of the unrounded values.
__device__ __forceinline__ float row_exp(uint32_t tS, float sl2, float m) {
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t c[32], d[32];
    tmem_ld32(tS, c);
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        tmem_wait_ld();
        tmem_ld32(tS + 64 * h + 32, d);
        exp_chunk(c, tS + 32 * h, sl2, m, a);
        tmem_wait_ld();
        if (h == 0) tmem_ld32(tS + 64, c);
        exp_chunk(d, tS + 32 * h + 16, sl2, m, a);
    }
    return (a[0] + a[1]) + (a[2] + a[3]);
}

// The partner warp's word for tile t, (t + 1, m) (bounded: false when it gives
// up, the error raised).
__device__ __forceinline__ bool partner_max(volatile unsigned long long* word, int t, float& m, uint32_t* err,
                                            volatile int* abort) {
    unsigned long long t0 = 0ull;
    for (uint32_t i = 1;; ++i) {
        const unsigned long long v = *word;
        m = __uint_as_float(static_cast<uint32_t>(v));
        if (__all_sync(0xFFFFFFFFu, static_cast<uint32_t>(v >> 32) == static_cast<uint32_t>(t) + 1u)) return true;
        if ((i & 63u) == 0u) {
            if (__any_sync(0xFFFFFFFFu, *abort != 0)) return false;
            const unsigned long long now = globaltimer_ns();
            if (t0 == 0ull) t0 = now;
            if (__any_sync(0xFFFFFFFFu, now - t0 > kWaitLimitNs)) {
                raise_error(err, DEVERR_TIMEOUT);
                *abort = 1;
                return false;
            }
        }
    }
}

// 32 * n columns of tensor memory times f (this thread's row): fp32, or bf16
// pairs.  Out of line: it runs when a row's maximum has grown by more than 2^32.
template <bool kPairs>
__device__ __noinline__ void scale_tmem(uint32_t taddr, int n, float f) {
    for (int q = 0; q < n; ++q) {
        uint32_t v[32];
        tmem_ld32(taddr + q * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c)
            v[c] = kPairs ? pack_bf16x2(__uint_as_float(v[c] << 16) * f, __uint_as_float(v[c] & 0xFFFF0000u) * f)
                          : __float_as_uint(__uint_as_float(v[c]) * f);
        tmem_st32(taddr + q * 32, v);
    }
    tmem_wait_st();
}

// Stage this warp's 32 rows' 16 * N-byte pieces (slot[N] = this thread's row)
// through shared memory (16-byte slots XOR-swizzled by row) and store each
// row's piece as whole lines: dst(rr) is where staged row rr goes (nullptr: skip).
template <int N, typename Dst>
__device__ __forceinline__ void stage_store(uint8_t* stage, int lane, const uint4 (&slot)[N], Dst dst) {
    uint4* my_row = reinterpret_cast<uint4*>(stage + lane * (16 * N));
#pragma unroll
    for (int c = 0; c < N; ++c) my_row[c ^ (lane & (N - 1))] = slot[c];
    __syncwarp();
    const int sub = lane & (N - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int rr = (32 / N) * i + lane / N;  // staged row this lane copies
        const uint4 val = reinterpret_cast<const uint4*>(stage + rr * (16 * N))[sub ^ (rr & (N - 1))];
        uint4* d = dst(rr);
        if (d) d[sub] = val;
    }
    __syncwarp();  // the next piece overwrites the stage
}

// ---------------------------------------------------------------------------
// Rows whose result is not finite.  A masked key has P = 0, but 0 times a
// value that is not finite is not 0: the tensor core lets an infinity or NaN in
// the values of a chunk's later token reach the rows before it in the same key
// tile.  A row that comes out not finite is computed again here, key by key over
// the keys that it sees (a warp per row): rare, and then right.
// ---------------------------------------------------------------------------
template <int D>
__device__ __noinline__ void redo_row(const Params& p, int b, int L, int g, int token, long long rowid, int lane) {
    constexpr int kPer = D / 32;
    float qv[kPer], acc[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) qv[k] = __bfloat162float(p.q[rowid * D + lane + 32 * k]);
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    constexpr int kBatch = 8;  // keys in flight, half a page
    for (int s0 = 0; s0 <= L + token; s0 += kBatch) {
        const long long page = p.block_table[static_cast<long long>(b) * p.max_pages + s0 / JT_PAGE_SIZE];
        const bool in_pool = page >= 0 && page < p.num_pages;  // the copies read zeros from a page outside
        const long long base = ((page * JT_PAGE_SIZE + s0 % JT_PAGE_SIZE) * p.Hkv + g) * D;
        const long long step = static_cast<long long>(p.Hkv) * D;
        const int n = min(kBatch, L + token + 1 - s0);
        float d[kBatch], v[kBatch][kPer];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            d[i] = 0.0f;
            const bool on = in_pool && i < n;
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                d[i] = fmaf(qv[k], on ? __bfloat162float(p.k_cache[base + i * step + lane + 32 * k]) : 0.0f, d[i]);
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                v[i][k] = on ? __bfloat162float(p.v_cache[base + i * step + lane + 32 * k]) : 0.0f;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
            for (int i = 0; i < kBatch; ++i) d[i] += __shfl_xor_sync(0xFFFFFFFFu, d[i], o);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (i >= n) break;
            const float s = d[i] * p.scale_log2;
            const float mn = fmaxf(m, s);
            const float corr = m == -INFINITY ? 0.0f : exp2f(m - mn);
            const float e = s == -INFINITY ? 0.0f : exp2f(s - mn);
            l = l * corr + e;
#pragma unroll
            for (int k = 0; k < kPer; ++k) acc[k] = fmaf(e, v[i][k], acc[k] * corr);
            m = mn;
        }
    }
    const float inv = 1.0f / l;
#pragma unroll
    for (int k = 0; k < kPer; ++k) p.out[rowid * D + lane + 32 * k] = __float2bfloat16(acc[k] * inv);
}

// Operand descriptors are stepped by adding the byte offset / 16 to the
// start-address field.  The whole MMA warp calls these; one elected lane issues.

// The pair's MMAs with the low words of their operands' descriptors in 32 bits
// (the start address steps; the high words are constants), which halves the
// address arithmetic between two MMAs.
__device__ __forceinline__ void mma_ss32(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts32(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// S = Q K^T over the pair: D / 16 MMAs of M = 256, N = 128, K = 16; then the
// commits that report S, the K stage and, past a piece's last tile, its Q.
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t tS, uint64_t dq, uint64_t dk, uint64_t* s_full, uint64_t* k_empty,
                                         uint64_t* q_empty) {
    using SL = Smem<D>;
    constexpr uint32_t idesc = idesc_bf16_f32(2 * kTileM, kTileN, false);
    if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t qo = ((kk >> 2) * SL::kQChunk + (kk & 3) * 32) >> 4;
            const uint32_t ko = ((kk >> 2) * SL::kKChunk + (kk & 3) * 32) >> 4;
            mma_ss32(tS, static_cast<uint32_t>(dq) + qo, static_cast<uint32_t>(dk) + ko, (1024u >> 4) | 1u << 14 | 2u << 29,
                     idesc, kk > 0 ? 1u : 0u);
        }
        mma_commit_pair(s_full);
        mma_commit_pair(k_empty);
        if (q_empty) mma_commit_pair(q_empty);
    }
    __syncwarp();
}

// O (+)= P V over the pair, P (bf16 pairs) in the first 64 columns of an S
// buffer: 8 MMAs of M = 256, N = D, K = 16; then the commits that report O (and
// with it the S buffer) and the V stage.
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t tO, uint32_t tP, uint64_t dv, bool accumulate, uint64_t* o_done,
                                         uint64_t* v_empty) {
    constexpr uint32_t idesc = idesc_bf16_f32(2 * kTileM, D, true);
    if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kTileN / 16; ++kk)
            mma_ts32(tO, tP + kk * 8, static_cast<uint32_t>(dv) + kk * ((16 * Smem<D>::kVRow) >> 4),
                     static_cast<uint32_t>(dv >> 32), idesc, (accumulate || kk > 0) ? 1u : 0u);
        mma_commit_pair(o_done);
        mma_commit_pair(v_empty);
    }
    __syncwarp();
}

__device__ __forceinline__ void commit_warp(uint64_t* bar) {
    if (elect_one()) mma_commit_pair(bar);
    __syncwarp();
}

// MN-major B operand (V): 128-byte rows take the 128-byte swizzle (64 dims per
// CTA), 64-byte rows the 64-byte one (32 dims per CTA); groups of 8 keys are
// contiguous.
template <int D>
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((Smem<D>::kVHalf >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>((8 * Smem<D>::kVRow) >> 4) << 32;
    d |= 1ull << 46;
    d |= (D == 128 ? 2ull : 4ull) << 61;
    return d;
}

// Page ids of 4 consecutive tiles (group g4) of a piece: lane l holds page
// l % 8 of tile 4 * g4 + l / 8 of the piece.
__device__ __forceinline__ int bt_group(const Params& p, const Piece& pc, int valid_end, int g4, int lane) {
    const int tile = 4 * g4 + (lane >> 3);
    const int slot = (pc.t0 + tile) * kTileN + (lane & 7) * JT_PAGE_SIZE;
    return (tile < pc.nt && slot < valid_end)
               ? p.block_table[static_cast<long long>(pc.b) * p.max_pages + slot / JT_PAGE_SIZE]
               : 0;
}

// A page id, or the first one past the pool for every id outside it: the copies
// then read zeros, and the K producer reports it.
__device__ __forceinline__ int page_in_pool(const Params& p, int pid) {
    return static_cast<int>(min(static_cast<uint32_t>(pid), static_cast<uint32_t>(p.num_pages)));
}

// Merge of a cut unit's pieces for this CTA's query tile x, by the 4 epilogue
// warps.  Per row M = max m_k, O = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k,
// in piece order whoever merges, so every call rounds the same way.  A piece
// without a visible key has l = 0 and an O that says nothing; one whose scores
// are all NaN has m = -inf and a NaN sum, which stays.  Both forms are small
// loops: a merge runs once or twice in a CTA's life, from a cold instruction
// cache (16 sequences of 1 to 512 tokens on 1024 to 8192, 32/8 heads, D 128: 216
// us with rows and pieces unrolled, 199 so).
template <int kC>
__device__ __forceinline__ void load_cols(const float* src, float (&v)[kC]) {
    if constexpr (kC == 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(src));
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(src));
        v[0] = f.x, v[1] = f.y;
    }
}
// The row's columns to dst as bf16; whether some are not finite (warp-uniform).
template <int kC>
__device__ __forceinline__ bool store_cols(__nv_bfloat16* dst, const float (&acc)[kC], float inv) {
    float o[kC], probe = 0.0f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        o[c] = acc[c] * inv;
        probe += o[c] * 0.0f;
    }
    if (dst) {
        if constexpr (kC == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
        else
            *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0], o[1]);
    }
    return __any_sync(0xFFFFFFFFu, probe != 0.0f);
}

// More rows than pieces (prompts): a warp takes up to 32 rows, 8 of them at a
// time; lane i keeps the weights of its row i.
template <int D>
__device__ __noinline__ void merge_many(const Params& p, const Piece& pc, const CutUnit cu, int x, int rows, int swarp,
                                        int lane) {
    constexpr int kC = D / 32;               // columns per lane
    const int q = (rows + 31) / 32 * 8;      // rows per warp
    const int base = swarp * q, n = min(rows - base, q);
    if (n <= 0) return;
    const int r = min(base + lane, rows - 1);  // this lane's row
    const int token = (2 * pc.mp + x) * p.npt + r / p.G;
    const long long rowid = static_cast<long long>(pc.s.off + token) * p.Hq + pc.g * p.G + r % p.G;
    constexpr long long stride = 2ll * kTileM;  // rows between partial slots
    const float2* ml = p.part_ml + x * kTileM + r;
    float M = -INFINITY, l = 0.0f;
#pragma unroll 2
    for (int k = 0; k < cu.n; ++k) M = fmaxf(M, __ldcg(ml + cu.slot(k) * stride).x);
#pragma unroll 2
    for (int k = 0; k < cu.n; ++k) {
        const float2 a = __ldcg(ml + cu.slot(k) * stride);
        l += a.y == 0.0f ? 0.0f : exp2f(a.x - M) * a.y;
    }
    const float inv = 1.0f / l;
    if (p.lse && lane < n) p.lse[rowid] = (M + log2f(l)) * 0.6931471805599453f;
    unsigned bad = 0u;
#pragma unroll 1
    for (int r0 = 0; r0 < n; r0 += 8) {
        const float* src = p.part_o + (x * kTileM + base + r0) * D + lane * kC;
        float acc[8][kC];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < kC; ++c) acc[i][c] = 0.0f;
#pragma unroll 1
        for (int k = 0; k < cu.n; ++k) {
            const long long at = cu.slot(k) * stride;
            const float2 a = __ldcg(ml + at);
            float v[8][kC];
#pragma unroll
            for (int i = 0; i < 8; ++i) load_cols<kC>(src + at * D + i * D, v[i]);
            const float w = a.y == 0.0f ? 0.0f : exp2f(a.x - M);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float wi = __shfl_sync(0xFFFFFFFFu, w, r0 + i);
                if (wi != 0.0f)
#pragma unroll
                    for (int c = 0; c < kC; ++c) acc[i][c] = fmaf(wi, v[i][c], acc[i][c]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const long long id = __shfl_sync(0xFFFFFFFFu, rowid, r0 + i);
            const bool nf = store_cols<kC>(r0 + i < n ? p.out + id * D + lane * kC : nullptr, acc[i],
                                           __shfl_sync(0xFFFFFFFFu, inv, r0 + i));
            if (nf && r0 + i < n) bad |= 1u << (r0 + i);
        }
    }
    bad &= __ballot_sync(0xFFFFFFFFu, l == l);
    while (bad) {
        const int i = __ffs(bad) - 1;
        bad &= bad - 1;
        __syncwarp();
        redo_row<D>(p, pc.b, pc.s.L, pc.g, __shfl_sync(0xFFFFFFFFu, token, i), __shfl_sync(0xFFFFFFFFu, rowid, i), lane);
    }
}

// More pieces than rows (single tokens): a warp takes one row at a time, 32
// pieces' weights in its lanes and 16 pieces' O in flight.
template <int D>
__device__ __noinline__ void merge_few(const Params& p, const Piece& pc, const CutUnit cu, int x, int rows, int swarp,
                                       int lane) {
    constexpr int kC = D / 32, kBatch = 16;
    constexpr long long stride = 2ll * kTileM;
#pragma unroll 1
    for (int r = swarp; r < rows; r += 4) {
        const long long xr = x * kTileM + r;
        const int token = (2 * pc.mp + x) * p.npt + r / p.G;
        const long long rowid = static_cast<long long>(pc.s.off + token) * p.Hq + pc.g * p.G + r % p.G;
        float M = -INFINITY, l = 0.0f, acc[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) acc[c] = 0.0f;
#pragma unroll 1
        for (int k0 = 0; k0 < cu.n; k0 += 32) {
            const float2 a = k0 + lane < cu.n ? __ldcg(p.part_ml + cu.slot(k0 + lane) * stride + xr)
                                              : make_float2(-INFINITY, 0.0f);
            float w = 0.0f;
#pragma unroll 1
            for (int kk = k0; kk < min(cu.n, k0 + 32); kk += kBatch) {
                float v[kBatch][kC];
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    load_cols<kC>(p.part_o + (cu.slot(min(kk + k, cu.n - 1)) * stride + xr) * D + lane * kC, v[k]);
                if (kk == k0) {
                    float mx = a.x, sum;
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                    mx = fmaxf(mx, M);
                    const float old = l == 0.0f ? 0.0f : exp2f(M - mx);  // what earlier pieces are worth now
                    M = mx;
                    w = a.y == 0.0f ? 0.0f : exp2f(a.x - mx);
                    sum = w * a.y;
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    l = l * old + sum;
#pragma unroll
                    for (int c = 0; c < kC; ++c) acc[c] *= old;
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const float wk = __shfl_sync(0xFFFFFFFFu, w, (kk - k0 + k) & 31);
                    if (wk != 0.0f)  // past the last piece, too
#pragma unroll
                        for (int c = 0; c < kC; ++c) acc[c] = fmaf(wk, v[k][c], acc[c]);
                }
            }
        }
        const bool nf = store_cols<kC>(p.out + rowid * D + lane * kC, acc, 1.0f / l);
        if (lane == 0 && p.lse) p.lse[rowid] = (M + log2f(l)) * 0.6931471805599453f;
        if (nf && l == l) {
            __syncwarp();
            redo_row<D>(p, pc.b, pc.s.L, pc.g, token, rowid, lane);
        }
    }
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Params p) {
    using SL = Smem<D>;
    constexpr int KS = SL::kKStages, VS = SL::kVStages;
    constexpr int kHalfCols = D / 2;  // dims of V per CTA
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Bars* bars = reinterpret_cast<Bars*>(smem + SL::kBar);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();  // 0: the leader, which issues the pair's MMAs
    const int work = static_cast<int>(blockIdx.x >> 1), nwork = static_cast<int>(gridDim.x >> 1);
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->q_full[s], 1);
            mbar_init(&bars->q_empty[s], 1);
        }
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&bars->k_full[s], 1);
            mbar_init(&bars->k_empty[s], 1);
            mbar_init(&bars->v_full[s], 1);
            mbar_init(&bars->v_empty[s], 1);
            mbar_init(&bars->v_own[s], 1);
        }
        for (int x = 0; x < 3; ++x) {
            mbar_init(&bars->s_full[x], 1);
            mbar_init(&bars->p_full[x], 8);
            mbar_init(&bars->o_done[x], 1);
        }
        mbar_init(&bars->o_free, 8);
        mbar_init(&bars->mma_final, 2);
        for (int i = 0; i < kRing; ++i)
            for (int w = 0; w < 4; ++w) mbar_init(&bars->x_bar[i][w], 2);
        mbar_init(&bars->msync, 4);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 12 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 13) tmem_alloc_pair(&bars->tmem_base, 512);
    // The V ring starts as zeros, and the rows of a unit-final tile's last page
    // past the needed slots are zeroed once it has landed: rows that no copy of
    // the present tile wrote are then always finite (P is 0 there, but 0 * NaN
    // would not be).
    for (int i = tid; i < VS * SL::kVHalf / 16; i += kThreads)
        reinterpret_cast<uint4*>(smem + SL::kV)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    reinterpret_cast<uint64_t*>(smem + SL::kM)[tid] = 0ull;  // kThreads words: no tile yet
    cluster_sync();  // both CTAs' barriers exist before any copy, commit or arrive crosses the pair
    pdl_wait();      // no global memory is read before the previous kernel's writes are visible
    if (warp == 12) plan_slot(p, bars, lane, work, nwork, work == 0 && rank == 0);
    if (tid == 0) bars->call_id = draw_call_id(p.tickets, work == 0 && rank == 0, gridDim.x);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    volatile int* abort = &bars->abort;
    const int quota = bars->w_quota;  // the same in both CTAs: one plan per work slot

    uint8_t* sQ = smem + SL::kQ;
    uint8_t* sK = smem + SL::kK;
    uint8_t* sV = smem + SL::kV;
    const int npt = p.npt;

    if (quota > 0 && warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 12) {
            // ------------------------------------------------------- TMA: Q, K
            Walker w;
            w.init(p, bars, work);
            Piece pc;
            int jj = 0, npc = 0;
            bool ok = true;
            while (ok && !*abort && w.next(p, pc)) {
                const int valid_end = unit_end(pc.s, pc.mp, npt);
                const int qs = npc & 1;
                // this CTA's Q tile (the peer's may lie past the chunk: its rows are never written out)
                if (npc >= 2 && !mbar_wait_warp(&bars->q_empty[qs], ((npc >> 1) - 1) & 1, p.err, abort)) break;
                if (lane == 0) {
                    if (rank == 0) mbar_arrive_expect_tx(&bars->q_full[qs], 2 * SL::kChunks * npt * p.G * 128);
                    for (int c = 0; c < SL::kChunks; ++c)
                        tma_load_3d_pair(sQ + qs * SL::kQBytes + c * SL::kQChunk, &tm_q, cluster_map(&bars->q_full[qs], 0),
                                         c * 64, pc.g * p.G, pc.s.off + (2 * pc.mp + static_cast<int>(rank)) * npt);
                }
                ++npc;
                int bt_cur = bt_group(p, pc, valid_end, 0, lane);
                int bt_nxt = bt_group(p, pc, valid_end, 1, lane);
                int bt_nn = bt_group(p, pc, valid_end, 2, lane);
                for (int j = 0; j < pc.nt; ++j, ++jj) {
                    const int st = jj % KS;
                    if (j > 0 && (j & 3) == 0) {
                        bt_cur = bt_nxt;
                        bt_nxt = bt_nn;
                        bt_nn = bt_group(p, pc, valid_end, (j >> 2) + 2, lane);
                    }
                    const int nvalid = min(kTileN, valid_end - (pc.t0 + j) * kTileN);
                    const int npg = (nvalid + JT_PAGE_SIZE - 1) / JT_PAGE_SIZE;
                    const int pid = page_in_pool(p, __shfl_sync(0xFFFFFFFFu, bt_cur, ((j & 3) << 3) + (lane & 7)));
                    if (lane < npg && pid == p.num_pages) raise_error(p.err, DEVERR_INVALID);
                    // this CTA's 64 keys (pages 4X..4X+3 of the tile); the slot frees once QK of tile jj - KS is done
                    if (jj >= KS && !mbar_wait_warp(&bars->k_empty[st], ((jj / KS) & 1) ^ 1, p.err, abort)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0 && rank == 0)
                        mbar_arrive_expect_tx(&bars->k_full[st], npg * SL::kChunks * (JT_PAGE_SIZE * 128));
                    __syncwarp();
                    if (lane < npg && (lane >> 2) == static_cast<int>(rank)) {
                        const uint32_t lead = cluster_map(&bars->k_full[st], 0);
                        for (int c = 0; c < SL::kChunks; ++c)
                            tma_load_4d_pair(sK + st * SL::kKHalf + c * SL::kKChunk + (lane & 3) * (JT_PAGE_SIZE * 128),
                                             &tm_k, lead, c * 64, pc.g, 0, pid);
                    }
                }
            }
            // on abort the leader lets the copies it counted land before the pair exits
            if (*abort && rank == 0) {
                for (int j = max(0, jj - KS); j < jj; ++j)
                    mbar_wait(&bars->k_full[j % KS], (j / KS) & 1, p.err, nullptr);
                for (int n = max(0, npc - 2); n < npc; ++n) mbar_wait(&bars->q_full[n & 1], (n >> 1) & 1, p.err, nullptr);
            }
        } else if (warp == 14) {
            // ---------------------------------------------------------- TMA: V
            Walker w;
            w.init(p, bars, work);
            Piece pc;
            int jj = 0;
            int fin = 0;  // unit-final tiles so far
            bool ok = true;
            while (ok && !*abort && w.next(p, pc)) {
                const int valid_end = unit_end(pc.s, pc.mp, npt);
                int bt_cur = bt_group(p, pc, valid_end, 0, lane);
                int bt_nxt = bt_group(p, pc, valid_end, 1, lane);
                int bt_nn = bt_group(p, pc, valid_end, 2, lane);
                for (int j = 0; j < pc.nt; ++j, ++jj) {
                    const int st = jj % VS;
                    if (j > 0 && (j & 3) == 0) {
                        bt_cur = bt_nxt;
                        bt_nxt = bt_nn;
                        bt_nn = bt_group(p, pc, valid_end, (j >> 2) + 2, lane);
                    }
                    const int nvalid = min(kTileN, valid_end - (pc.t0 + j) * kTileN);
                    const int npg = (nvalid + JT_PAGE_SIZE - 1) / JT_PAGE_SIZE;
                    const int pid = page_in_pool(p, __shfl_sync(0xFFFFFFFFu, bt_cur, ((j & 3) << 3) + (lane & 7)));
                    // this CTA's D / 2 dims of every key; the slot frees once PV of tile jj - VS is done
                    if (jj >= VS && !mbar_wait_warp(&bars->v_empty[st], ((jj / VS) & 1) ^ 1, p.err, abort)) {
                        ok = false;
                        break;
                    }
                    uint8_t* vt = sV + st * SL::kVHalf;
                    const int c0 = static_cast<int>(rank) * kHalfCols;
                    if (pc.t0 + j != pc.T - 1) {
                        if (lane == 0 && rank == 0)
                            mbar_arrive_expect_tx(&bars->v_full[st], 2 * npg * (JT_PAGE_SIZE * SL::kVRow));
                        __syncwarp();
                        if (lane < npg)
                            tma_load_4d_pair(vt + lane * (JT_PAGE_SIZE * SL::kVRow), &tm_v,
                                             cluster_map(&bars->v_full[st], 0), c0, pc.g, 0, pid);
                    } else {
                        // a unit's final tile: each CTA lands its half on its own
                        // barrier; a softmax warp zeroes the rows past the last
                        // needed slot before it releases the tile's P.  The
                        // leader's v_full phase of this tile completes empty
                        if (lane == 0) {
                            if (rank == 0) mbar_arrive(&bars->v_full[st]);
                            mbar_arrive_expect_tx(&bars->v_own[fin % VS], npg * (JT_PAGE_SIZE * SL::kVRow));
                        }
                        __syncwarp();
                        if (lane < npg)
                            tma_load_4d(vt + lane * (JT_PAGE_SIZE * SL::kVRow), &tm_v, &bars->v_own[fin % VS], c0, pc.g, 0, pid);
                        ++fin;
                    }
                }
            }
            if (*abort) {
                for (int f = max(0, fin - VS); f < fin; ++f)
                    mbar_wait(&bars->v_own[f % VS], (f / VS) & 1, p.err, nullptr);
                if (rank == 0)
                    for (int j = max(0, jj - VS); j < jj; ++j)
                        mbar_wait(&bars->v_full[j % VS], (j / VS) & 1, p.err, nullptr);
            }
        } else if (rank == 0 && warp == 15) {
            // ------------------------------------------------ MMA: S = Q K^T
            const uint64_t dq0 = smem_desc_sw128(smem_u32(sQ), 16, 1024);
            const uint64_t dk0 = smem_desc_sw128(smem_u32(sK), 16, 1024);
            Walker w;
            w.init(p, bars, work);
            Piece pc;
            int qs = 0, st = 0, b = 0;              // Q slot, K stage and S buffer of the tile
            uint32_t qpar = 0, kpar = 0, opar = 1;  // their phase parities (S buffer: PV of its last tile)
            int fresh = 3;                          // S buffers that no tile has used
            bool ok = true;
            while (ok && w.next(p, pc)) {
                ok = mbar_wait_warp(&bars->q_full[qs], qpar, p.err, abort);
                const uint64_t dq = dq0 + qs * (SL::kQBytes >> 4);
                for (int left = pc.nt; ok && left > 0; --left) {
                    ok = mbar_wait_warp(&bars->k_full[st], kpar, p.err, abort);
                    // S(t mod 3) is free once PV(t - 3) has read the P in it
                    if (fresh > 0)
                        --fresh;
                    else
                        ok = ok && mbar_wait_warp(&bars->o_done[b], opar, p.err, abort);
                    if (!ok) break;
                    tc_fence_after();
                    issue_qk<D>(tmem + 128 * b, dq, dk0 + st * (SL::kKHalf >> 4), &bars->s_full[b], &bars->k_empty[st],
                                left == 1 ? &bars->q_empty[qs] : nullptr);
                    if (++st == KS) st = 0, kpar ^= 1;
                    if (++b == 3) b = 0, opar ^= 1;
                }
                qs ^= 1;
                if (qs == 0) qpar ^= 1;
            }
            commit_warp(&bars->mma_final);
        } else if (rank == 0 && warp == 13) {
            // ------------------------------------------------ MMA: O += P V
            const uint64_t dv0 = v_desc<D>(smem_u32(sV));
            Walker w;
            w.init(p, bars, work);
            Piece pc;
            int st = 0, b = 0;                      // V stage and S buffer of the tile
            uint32_t vpar = 0, ppar = 0, fpar = 1;
            bool ok = true, first = true;
            while (ok && w.next(p, pc)) {
                // the previous piece's O has been read out
                if (!first) ok = mbar_wait_warp(&bars->o_free, fpar, p.err, abort);
                first = false;
                fpar ^= 1;
                for (int j = 0; ok && j < pc.nt; ++j) {
                    ok = mbar_wait_warp(&bars->v_full[st], vpar, p.err, abort) &&
                         mbar_wait_warp(&bars->p_full[b], ppar, p.err, abort);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv<D>(tmem + 384, tmem + 128 * b, dv0 + st * (SL::kVHalf >> 4), j > 0, &bars->o_done[b],
                                &bars->v_empty[st]);
                    if (++st == VS) st = 0, vpar ^= 1;
                    if (++b == 3) b = 0, ppar ^= 1;
                }
            }
            commit_warp(&bars->mma_final);
        }
    } else if (quota > 0 && warp < 8) {
        // ------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int x = static_cast<int>(rank);
        const int wg = warp >> 2, w4 = warp & 3;
        const int r = tid & 127;  // query row = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(w4 * 32) << 16;
        const uint32_t tO = tmem + 384 + lane_off;
        const float sl2 = p.scale_log2;
        // The two warps of a row tell each other its m after every tile, lane
        // to lane in one 8-byte word.  A warp writes the word of tile t + 4 over
        // that of tile t, which its partner has read by then: each waits for the
        // other's word of the tile before in every tile.
        volatile unsigned long long* words = reinterpret_cast<volatile unsigned long long*>(smem + SL::kM) + r;
        auto word_of = [&](int t) { return words + ((t >> 1 & 1) * 2 + (t & 1)) * 128; };
        auto tell_partner = [&](int t, float m) {
            *word_of(t) = static_cast<unsigned long long>(t + 1) << 32 | __float_as_uint(m);
        };
        float2* xch = reinterpret_cast<float2*>(smem + SL::kX) + wg * 128 + r;
        const uint32_t lead_p = cluster_map(&bars->p_full[0], 0);
        WarpWalk* ws = reinterpret_cast<WarpWalk*>(smem + SL::kW) + warp;
        if (lane == 0) ws->w.init(p, bars, work);
        int cnt = 0, npc = 0, fin = 0;      // tiles, pieces and unit-final tiles so far
        bool ok = true;
        while (ok) {
            __syncwarp();
            int more = 0;
            if (lane == 0) more = ws->w.next(p, ws->pc) ? 1 : 0;
            more = __shfl_sync(0xFFFFFFFFu, more, 0);
            if (!more) break;
            const Piece& pc = ws->pc;
            const int tok0 = (2 * pc.mp + x) * npt;
            const int token = tok0 + r / p.G;
            const bool valid_row = r < npt * p.G && token < pc.s.B;
            const bool warp_on = __any_sync(0xFFFFFFFFu, valid_row);
            const int nt = pc.nt;
            const int visible0 = pc.s.L + token + 1 - pc.t0 * kTileN;  // keys of the row from the piece's first on
            const int jdiag = (pc.s.L + tok0 + 1) / kTileN - pc.t0;    // tiles before it need no mask
            const int jfin = pc.T - 1 - pc.t0;                         // the unit's final tile
            float m_run = -INFINITY, l_run = 0.0f;
            for (int j = (cnt + wg) & 1; j < nt; j += 2) {
                const int t = cnt + j, b = t % 3;
                if (!mbar_wait_warp(&bars->s_full[b], (t / 3) & 1, p.err, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // Warps without rows keep step all the same: a warp waits only
                // for its own tiles' S, and the partner's words tell it that the
                // phases in between have passed.
                float m_o = -INFINITY;  // the partner's m after the tile before: what O is scaled by
                if (warp_on) {
                    const uint32_t tS = tmem + 128 * b + lane_off;
                    if (j >= jdiag) mask_row(tS, visible0 - j * kTileN);
                    const float mx_s = row_max(tS) * sl2;
                    const float m_before = m_run;
                    if (j < 2 && t > 0) {
                        // j = 1: the row's first maximum; j = 0: the word to be
                        // written next may still be unread before this
                        if (!partner_max(word_of(t - 1), t - 1, m_o, p.err, abort)) {
                            ok = false;
                            break;
                        }
                        if (j == 1) m_run = m_o;
                    }
                    // a whole number of log2 units: a change of m then scales P and O
                    // by a power of two, and P is rounded once whatever m was then
                    if (mx_s > m_run + kRescaleLog2 || m_run == -INFINITY) m_run = ceilf(fmaxf(m_run, mx_s));
                    if (j == 0) tell_partner(t, m_run);  // early: the partner's first tile waits for it
                    // P = exp2(s*scale*log2e - m), written over S (bf16 pairs)
                    float sum = row_exp(tS, sl2, m_run == -INFINITY ? 0.0f : m_run);
                    if (j > 0) {
                        if (j > 1 && !partner_max(word_of(t - 1), t - 1, m_o, p.err, abort)) {
                            ok = false;
                            break;
                        }
                        if (__any_sync(0xFFFFFFFFu, valid_row && m_o != m_run)) {
                            const bool raise = m_run > m_o && m_o != -INFINITY;  // this tile raises m: O follows
                            const bool lag = m_o > m_run;                        // the partner has raised it: P follows
                            tmem_wait_st();
                            if (__any_sync(0xFFFFFFFFu, valid_row && raise)) {
                                // O holds PV(t - 1) before it is rescaled
                                if (!mbar_wait_warp(&bars->o_done[(t - 1) % 3], ((t - 1) / 3) & 1, p.err, abort)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                                scale_tmem<false>(tO, D / 32, raise ? ex2_approx(m_o - m_run) : 1.0f);
                            }
                            const float f = lag ? (m_run == -INFINITY ? 0.0f : ex2_approx(m_run - m_o)) : 1.0f;
                            scale_tmem<true>(tS, 2, f);
                            sum *= f;
                            if (lag) m_run = m_o;
                        }
                        tell_partner(t, m_run);
                    }
                    if (m_before != m_run) l_run = l_run == 0.0f ? 0.0f : l_run * ex2_approx(m_before - m_run);
                    l_run += sum;
                    tmem_wait_st();
                } else {
                    if (t > 0 && !partner_max(word_of(t - 1), t - 1, m_o, p.err, abort)) {
                        ok = false;
                        break;
                    }
                    tell_partner(t, -INFINITY);
                }
                if (j == jfin && w4 == 0) {
                    // the unit's final tile: zero the rows of its last page past the last needed slot
                    if (!mbar_wait_warp(&bars->v_own[fin % VS], (fin / VS) & 1, p.err, abort)) {
                        ok = false;
                        break;
                    }
                    const int nvalid = unit_end(pc.s, pc.mp, npt) - (pc.t0 + j) * kTileN;
                    const int end = (nvalid + JT_PAGE_SIZE - 1) / JT_PAGE_SIZE * JT_PAGE_SIZE;
                    for (int i = lane; i < (end - nvalid) * (SL::kVRow / 16); i += 32)
                        reinterpret_cast<uint4*>(sV + (t % VS) * SL::kVHalf + nvalid * SL::kVRow)[i] =
                            make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(lead_p + 8 * b);
            }
            if (!ok) break;
            cnt += nt;
            fin += jfin < nt ? 1 : 0;
            // The rows' maxima and sums go to the epilogue, which has read the
            // entry's previous piece (see kRing).
            xch[(npc % kRing) * 256] = make_float2(m_run, l_run);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->x_bar[npc % kRing][w4]);
            ++npc;
        }
    } else if (quota > 0) {
        // ------------------------------------------------------ epilogue
        // one query row per thread, while the softmax warps go on to the next piece
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
        const int x = static_cast<int>(rank);
        const int w4 = warp & 3;
        const int r = tid & 127;
        const uint32_t tO = tmem + 384 + (static_cast<uint32_t>(w4 * 32) << 16);
        uint8_t* stage = smem + SL::kStage + w4 * 2048;
        const float2* xch = reinterpret_cast<const float2*>(smem + SL::kX) + r;
        const uint32_t lead_free = cluster_map(&bars->o_free, 0);
        WarpWalk* ws = reinterpret_cast<WarpWalk*>(smem + SL::kW) + warp;
        if (lane == 0) ws->w.init(p, bars, work);
        int last = -1, npc = 0;  // the piece's last tile; pieces so far
        auto meet4 = [&](int i) -> bool {   // meeting i of a merge (a merge meets twice: parity i)
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->msync);
            return mbar_wait_warp(&bars->msync, static_cast<uint32_t>(i), p.err, abort);
        };
        bool ok = true;
        while (ok) {
            __syncwarp();
            int more = 0;
            if (lane == 0) more = ws->w.next(p, ws->pc) ? 1 : 0;
            more = __shfl_sync(0xFFFFFFFFu, more, 0);
            if (!more) break;
            const Piece& pc = ws->pc;
            last += pc.nt;
            const int tok0 = (2 * pc.mp + x) * npt;
            const int token = tok0 + r / p.G;
            const bool valid_row = r < npt * p.G && token < pc.s.B;
            const bool warp_on = __any_sync(0xFFFFFFFFu, valid_row);
            const bool tile_on = tok0 < pc.s.B;  // this CTA's query tile exists
            const bool partial = pc.slot >= 0;
            const long long rowid = static_cast<long long>(pc.s.off + token) * p.Hq + pc.g * p.G + r % p.G;
            // both softmax warps of the rows are through the piece (so S of its last tile has been seen)
            if (!mbar_wait_warp(&bars->x_bar[npc % kRing][w4], (npc / kRing) & 1, p.err, abort)) break;
            const float2 xa = xch[(npc % kRing) * 256], xb = xch[(npc % kRing) * 256 + 128];
            ++npc;
            const float m_tot = fmaxf(xa.x, xb.x);
            // (a sum is 0 without a key, and NaN beside m = -inf where every score was NaN: it stays NaN)
            const float l_tot = (xa.y == 0.0f ? 0.0f : xa.y * ex2_approx(xa.x - m_tot)) +
                                (xb.y == 0.0f ? 0.0f : xb.y * ex2_approx(xb.x - m_tot));
            if (ws->w.remaining <= 0) pdl_trigger();
            if (!mbar_wait_warp(&bars->o_done[last % 3], (last / 3) & 1, p.err, abort)) break;
            tc_fence_after();
            if (warp_on && partial) {
                const long long prow = (static_cast<long long>(pc.slot) * 2 + x) * kTileM + r;
                float* dst = p.part_o + prow * D;
#pragma unroll 1
                for (int h = 0; h < D / 32; ++h) {
                    uint32_t v[32];
                    tmem_ld32(tO + 32 * h, v);
                    tmem_wait_ld();
                    if (valid_row)
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            reinterpret_cast<uint4*>(dst + 32 * h)[c] =
                                make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
                }
                if (valid_row) p.part_ml[prow] = make_float2(m_tot, l_tot);
            }
            const float inv = 1.0f / l_tot;
            float probe = 0.0f;
            uint32_t packed[D / 2];
            if (warp_on && !partial) {
#pragma unroll
                for (int h = 0; h < D / 32; ++h) {
                    uint32_t v[32];
                    tmem_ld32(tO + 32 * h, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float a = __uint_as_float(v[2 * c]) * inv, b = __uint_as_float(v[2 * c + 1]) * inv;
                        probe += a * 0.0f + b * 0.0f;
                        packed[16 * h + c] = pack_bf16x2(a, b);
                    }
                }
            }
            // O has been read: the next piece's first PV may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(lead_free);
            if (warp_on && !partial) {
#pragma unroll
                for (int h = 0; h < D / 32; ++h) {
                    uint4 slot[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        slot[c] = make_uint4(packed[16 * h + 4 * c], packed[16 * h + 4 * c + 1],
                                             packed[16 * h + 4 * c + 2], packed[16 * h + 4 * c + 3]);
                    stage_store<4>(stage, lane, slot, [&](int rr) {
                        const long long rid = __shfl_sync(0xFFFFFFFFu, rowid, rr);
                        const bool rvalid = __shfl_sync(0xFFFFFFFFu, valid_row, rr);
                        return rvalid ? reinterpret_cast<uint4*>(p.out + rid * D + 32 * h) : nullptr;
                    });
                }
                if (valid_row && p.lse) p.lse[rowid] = (m_tot + log2f(l_tot)) * 0.6931471805599453f;
                unsigned bad = __ballot_sync(0xFFFFFFFFu, valid_row && probe != 0.0f && l_tot == l_tot);
                while (bad) {
                    const int rr = __ffs(bad) - 1;
                    bad &= bad - 1;
                    __syncwarp();
                    redo_row<D>(p, pc.b, pc.s.L, pc.g, __shfl_sync(0xFFFFFFFFu, token, rr),
                                        __shfl_sync(0xFFFFFFFFu, rowid, rr), lane);
                }
            }
            if (partial && tile_on) {
                // count this piece done; the slot that completes the unit merges every piece's rows
                const CutUnit cu(pc.gpos - pc.t0, pc.T, bars->w_P);
                if (!meet4(0)) break;  // the warps' partial rows are written
                if (w4 == 0 && lane == 0) {
                    __threadfence();  // and visible GPU-wide before the count
                    const uint32_t cid = bars->call_id;
                    unsigned long long* ctr = p.merge_cnt + 2 * cu.c0 + x;
                    unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(ctr), assumed, nv;
                    do {  // a count from an earlier call restarts at this call's first piece
                        assumed = old;
                        nv = ((assumed >> 32) == cid) ? assumed + 1ull
                                                      : ((static_cast<unsigned long long>(cid) << 32) | 1ull);
                        old = atomicCAS(ctr, assumed, nv);
                    } while (old != assumed);
                    bars->merge_flag = static_cast<int>(nv & 0xFFFFFFFFull) == cu.n;
                    __threadfence();  // the other pieces' rows are read after this count
                }
                if (!meet4(1)) break;
                if (bars->merge_flag) {
                    const int rows = min(pc.s.B - tok0, npt) * p.G;
                    if (rows > cu.n)
                        merge_many<D>(p, pc, cu, x, rows, w4, lane);
                    else
                        merge_few<D>(p, pc, cu, x, rows, w4, lane);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    // both CTAs: every MMA of the pair has completed before TMEM is released
    if (warp == 13 && quota > 0) mbar_wait_warp(&bars->mma_final, 0, p.err, nullptr);
    cluster_sync();  // no copy, arrive or MMA of the pair targets either CTA any more
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
typedef CUresult (*PFN_encodeTiled_t)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                      const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                      CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static PFN_encodeTiled_t encode_fn() {
    static const PFN_encodeTiled_t fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool got = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                                          &q) == cudaSuccess &&
                         q == cudaDriverEntryPointSuccess;
        return got ? reinterpret_cast<PFN_encodeTiled_t>(ptr) : nullptr;
    }();
    return fn;
}

// The merge counts sit between the header and a fixed offset, whatever the
// head dim and dtype of the calls that share a workspace.
constexpr int kMaxSlots = static_cast<int>((kChunkFixedBytes - kWsHeader) / 16);

// Work slots on the current device: the clusters of two CTAs that can be
// resident at once (one CTA per SM).
template <int D>
static int work_slots() {
    static PerDeviceCache cache;
    const int n = cache.get([] {
        const int fallback = std::max(1, device_sm_count() / 2);
        if (cudaFuncSetAttribute(chunk_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kAlloc) !=
            cudaSuccess) {
            (void)cudaGetLastError();
            return fallback;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * fallback);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Smem<D>::kAlloc;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, chunk_attn_kernel<D>, &cfg) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            return fallback;
        }
        return n;
    });
    return std::min(n, kMaxSlots);
}

static size_t ml_bytes(int slots) { return align_up(static_cast<size_t>(2) * slots * 2 * kTileM * sizeof(float2)); }

template <int D>
static cudaError_t launch(const ChunkArgs& a, char* ws, cudaStream_t st) {
    PFN_encodeTiled_t enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const int slots = work_slots<D>();
    const int G = a.Hq / a.Hkv, npt = kTileM / G;
    const cuuint64_t eD = D, eHq = a.Hq, eHkv = a.Hkv;
    const cuuint32_t es[4] = {1, 1, 1, 1};
    CUtensorMap tq, tk, tv;
    {
        const cuuint64_t dims[3] = {eD, eHq, static_cast<cuuint64_t>(a.total)};
        const cuuint64_t strides[2] = {eD * 2, eHq * eD * 2};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(npt)};
        if (enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t dims[4] = {eD, eHkv, JT_PAGE_SIZE, static_cast<cuuint64_t>(a.num_pages)};
        const cuuint64_t strides[3] = {eD * 2, eHkv * eD * 2, JT_PAGE_SIZE * eHkv * eD * 2};
        const cuuint32_t kbox[4] = {64, 1, JT_PAGE_SIZE, 1};
        const cuuint32_t vbox[4] = {D / 2, 1, JT_PAGE_SIZE, 1};
        if (enc(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.k_cache), dims, strides, kbox, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
            enc(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.v_cache), dims, strides, vbox, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    Params prm;
    prm.block_table = a.block_table;
    prm.prefix_len = a.prefix_len;
    prm.off = a.chunk_off;
    prm.q = static_cast<const __nv_bfloat16*>(a.q);
    prm.k_cache = static_cast<const __nv_bfloat16*>(a.k_cache);
    prm.v_cache = static_cast<const __nv_bfloat16*>(a.v_cache);
    prm.out = static_cast<__nv_bfloat16*>(a.out);
    prm.lse = a.lse;
    char* w = ws + kWsHeader;
    prm.merge_cnt = reinterpret_cast<unsigned long long*>(w);
    w += kChunkFixedBytes - kWsHeader;
    prm.part_ml = reinterpret_cast<float2*>(w);
    w += ml_bytes(slots);
    prm.part_o = reinterpret_cast<float*>(w);
    prm.tickets = &reinterpret_cast<WsHeader*>(ws)->tickets;
    prm.err = reinterpret_cast<uint32_t*>(ws);
    prm.max_pages = a.max_pages;
    prm.num_pages = a.num_pages;
    prm.nseq = a.nseq;
    prm.total = a.total;
    prm.max_chunk = a.max_chunk;
    prm.Hq = a.Hq;
    prm.Hkv = a.Hkv;
    prm.G = G;
    prm.npt = npt;
    prm.scale_log2 = a.scale * 1.4426950408889634f;
    static PerDeviceCache attr;  // the shared-memory opt-in is per device
    const cudaError_t ea = static_cast<cudaError_t>(attr.get([] {
        return static_cast<int>(cudaFuncSetAttribute(chunk_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     Smem<D>::kAlloc));
    }));
    if (ea != cudaSuccess) return ea;
    return launch_kernel_pdl(chunk_attn_kernel<D>, dim3(2 * slots), dim3(kThreads), Smem<D>::kAlloc, st, tq, tk, tv,
                             prm);
}

}  // namespace chunk

size_t chunk_attn_bf16_workspace_bytes(int D) {
    if (D != 64 && D != 128) return kChunkFixedBytes;
    const int slots = D == 128 ? chunk::work_slots<128>() : chunk::work_slots<64>();
    return kChunkFixedBytes + chunk::ml_bytes(slots) +
           align_up(static_cast<size_t>(2) * slots * 2 * chunk::kTileM * D * sizeof(float));
}

cudaError_t chunk_attn_bf16_launch(const ChunkArgs& a, char* ws, cudaStream_t st) {
    if (a.D == 128) return chunk::launch<128>(a, ws, st);
    if (a.D == 64) return chunk::launch<64>(a, ws, st);
    return cudaErrorInvalidValue;
}

}  // namespace jt
