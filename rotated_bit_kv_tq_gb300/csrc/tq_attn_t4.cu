// tq_attn_t4.cu -- single-token attention over turbo4 K and V caches on the 5th-generation
// tensor cores, with 8-bit operands.
//
// The mathematics is tq_attn.cu's (rotated domain, split keys, online softmax).  turbo4's
// levels are e4m3 numbers up to one scale: one byte lookup turns four codes into four exact
// operands (0.9 integer instructions per value), and tcgen05.mma kind::f8f6f4 takes them from
// shared memory as they are.  (mma.sync has an e4m3 form too, but sm_103a runs it as conversions
// and fp16 products: 0.19 per ns and SM.  On mma.sync with fp16 operands the conversions and
// fragment handling came to 3.5 instructions per value.)
//
// What fp32 held (the query, the weights p |v|) is cut into e4m3 pieces, piece i holding the
// remainder of those before it times 16^i, in rows of their own:
//   scores  S[(block, token), (block', piece, head)] = C_k[(block, token), coord] . Q~^T
//           M = 128 rows are 32 tokens of four 128-value blocks, N = the pieces of four blocks'
//           queries; a row uses its own block's columns only (three quarters of the product are
//           not looked at: the tensor cores have that to spare)
//   values  O_block[coord, (piece, head)] += C_v^T[coord, token] . P^T, one M = 128, K = 32 product
//           per block
// Four pieces keep 16 bits of the query, three keep 12 bits of the weights (fp16 keeps 11).
// Heads come in sets of four per KV head (SETS = 2 for five to eight).
//
// Weights: e4m3 spans 18 binades and |v| is unbounded, so the running shift m of the softmax is
// the maximum of s + log2 |v| instead of that of s (up to kLag): 64 p |v| = 64 |v| 2^(s - m) is
// then at most 256 and the third piece reaches 2^-24 below the largest contribution.
//
// Roles of a CTA (one per SM, 27 warps), per tile of 32 tokens x 8 blocks:
//  - warp 25 copies the rows into a ring of two tiles with TMA bulk copies (rows of eight blocks,
//    528 bytes; the page numbers of 16 tiles are looked up at once);
//  - warps 8-15 (K) and 16-23 (V), one thread per (block, token): read 64 bytes of codes, write 128
//    operand bytes in the no-swizzle canonical layouts (K: coordinates along K; V: coordinates
//    contiguous along M), double-buffered.  Rows of other widths come straight from global
//    memory, one tile ahead in registers (DIRECT);
//  - warps 24 (scores) and 26 (values) issue the products, the whole warp running the loop and one
//    lane issuing, so that descriptors stay in uniform registers; completions arrive through
//    tcgen05.commit;
//  - warps 0-7, one per block, one thread per token: read S from tensor memory, add the pieces,
//    scale by |k|, mask, shift, write the weights' pieces, and rescale O in tensor memory when a
//    maximum moved (every warp the 32 coordinates of its tensor-memory quarter, after a barrier
//    that publishes the factors).
// At head_dim 256 a head's two blocks are two warps, which exchange their halves of the scores.
//
// Work: the tokens of all sequences are laid end to end (each padded by kSegPad, about what
// starting and ending a segment costs) and cut into equal chunks, one per CTA, so a batch of
// unequal lengths leaves no SM idle; a CTA walks through the segments of its chunk.  Rows of more
// than eight blocks are cut in slices of eight, a CTA for each.  Rows that cannot be addressed
// are masked.
//
// Partial results: one sequence whose rows fit one slice is one cooperative launch that merges
// its own partials (merge_grid below); otherwise every segment writes one partial row, merged by
// attn_t4_merge_kernel.  Every wait is bounded.
#include <cmath>

#include "tq_attn_mma_kernel.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

constexpr int kT4 = TQ_TURBO4;
constexpr int kTile = 32;             // tokens per tile
constexpr int kSlice = 8;             // blocks of a row that one CTA takes
constexpr int kSliceRow = kSlice * block_bytes(TQ_TURBO4);   // 528
// A segment's fixed cost in rows.  64, 128, 256, 512: 83, 75, 68, 67 us for 33 sequences of 0-8,191
// rows under 40 heads; 27.0, 25.9, 27.1, 30.2 us for 64 sequences of 512 rows under 32.
constexpr int kSegPad = 256;
constexpr int kMinChunk = 32;         // rows per CTA, one sequence
constexpr int kMinChunkBatch = 128;   // padded rows per CTA, batch
constexpr int kSoftWarps = 8, kDecWarps = 8;      // softmax; K decode, V decode
constexpr int kWarpK = kSoftWarps, kWarpV = kWarpK + kDecWarps, kWarpMma = kWarpV + kDecWarps, kWarpTma = kWarpMma + 1;
constexpr int kWarpPv = kWarpTma + 1;
constexpr int kT4Warps = kWarpPv + 1, kT4Threads = 32 * kT4Warps;
constexpr int kRing = 2;              // ring tiles
constexpr int kNormSlots = 4;         // tiles whose norms are kept: K decode runs up to three ahead of the softmax
// The shift moves only when a maximum passes it by more than kLag (log2): O in tensor memory is
// then rarely rewritten (without the lag some head of the eight blocks moved in almost every
// tile of a long context's first quarter, 1,000 clocks each).  Weights are scaled by 2^kWeightUp, so
// that with the lag they stay below 2^8 (e4m3 ends at 448).
constexpr float kLag = 2.0f, kWeightUp = 6.0f;
constexpr float kDown = 0.0625f;      // a piece's scale against the one before it
constexpr uint32_t kDrainPolls = 1u << 24;

struct T4Params {
    CacheView kc, vc;
    const __half *q;
    const __half *k_new, *v_new;
    const int32_t *seq_lens;
    float *part;          // batch: fp32 rows [segment][Hq][part_stride]; one sequence: tagged words
    int2 *seg;            // batch: [n_seqs] first and last chunk of each sequence
    float score_scale;    // softmax scale * log2(e) / sqrt(128) * kE4m3Step4
    int32_t max_len, n_seqs, n_q_heads, group;
    int32_t bpr;          // blocks per row
    int32_t n_chunks;     // chunks the tokens are cut into (CTAs = chunks x slices)
    uint32_t wait_limit;
    OutPtr out;
    uint64_t *bar;        // one sequence: the grid-merge area
    uint32_t grid_wait_limit;
    int32_t withhold_tiles;
};

// ------------------------------------------------------------------ PTX helpers
// kind::f8f6f4, e4m3 operands, fp32 accumulators, M = 128, N = n
constexpr uint32_t idesc_f8(int n, bool a_mn, bool b_mn) {
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n"
                 ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t e4m3_of_half2(uint32_t h2) {   // two bytes in bits 0-15
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(h2));
    return d;
}
__device__ __forceinline__ uint32_t h2fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// The remainder h - piece, times 16: exact in fp16 (h has 11 bits, its e4m3 rounding the top 4).
__device__ __forceinline__ uint32_t rest16(uint32_t h, uint32_t piece) {
    return h2fma(e4m3_to_half2(piece), 0xCC00CC00u, h2mul(h, 0x4C004C00u));
}
// Bounded wait on a phase.  After a wait has run out (or another role's has) all later ones return
// at once; the roles then run through their loops and meet at the barriers.
__device__ __forceinline__ void t4_wait(uint64_t *bar, uint32_t parity, uint32_t limit, volatile int *gave_up) {
    const uint32_t a = smem_u32(bar);
    if (mbar_try_wait(a, parity)) return;
#pragma unroll 1
    for (uint32_t it = 1; it < limit; ++it) {
        if (mbar_try_wait(a, parity)) return;
        if (*gave_up) return;
    }
    record_error(TQ_ERR_DEVICE_TIMEOUT);
    *gave_up = 1;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 9, 256;" ::: "memory"); }
// The two warps of a head_dim-256 head.
__device__ __forceinline__ void pair_sync(int warp) { asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory"); }

// ------------------------------------------------------------------ chunks and segments
__device__ __forceinline__ int clamped_len(const T4Params &p, int len) {
    if (len < 0 || len > p.max_len) {
        record_error(TQ_ERR_OUT_OF_RANGE);
        len = len < 0 ? 0 : p.max_len;
    }
    return len;
}

// Calls f(seq, len, lo, hi) for every segment of this CTA's chunk, by whole warps, in order.
template <typename F>
__device__ __forceinline__ void for_segments(const T4Params &p, int64_t c, int64_t n_chunks, F f) {
    const int lane = threadIdx.x & 31;
    if (p.n_seqs == 1) {
        const int len = clamped_len(p, p.seq_lens[0]);
        const int chunk = max(kMinChunk, (int)((len + n_chunks - 1) / n_chunks));
        const int64_t lo = c * chunk;
        f(0, len, (int)min64(lo, len), (int)min64(lo + chunk, len), int64_t(0), (int64_t)chunk);
        return;
    }
    int64_t total = 0;
    for (int i = lane; i < p.n_seqs; i += 32) {
        const int len = p.seq_lens[i];
        const int l = len < 0 ? 0 : min(len, p.max_len);
        total += l > 0 ? (int64_t)l + kSegPad : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int64_t chunk = max64(kMinChunkBatch, (total + n_chunks - 1) / n_chunks);
    const int64_t c0 = c * chunk, c1 = c0 + chunk;
    int64_t before = 0;
    for (int base = 0; base < p.n_seqs && before < c1; base += 32) {
        const int i = base + lane;
        int len = 0;
        if (i < p.n_seqs) {
            len = p.seq_lens[i];
            if (len < 0 || len > p.max_len) {
                if (c == 0 && threadIdx.x < 32) record_error(TQ_ERR_OUT_OF_RANGE);
                len = len < 0 ? 0 : p.max_len;
            }
        }
        int64_t x = len > 0 ? (int64_t)len + kSegPad : 0;
        const int64_t mine = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const int64_t s = before + x - mine;   // this sequence's first padded row
        unsigned todo = __ballot_sync(0xffffffffu, len > 0 && s < c1 && s + len > c0);
        while (todo) {
            const int b = __ffs(todo) - 1;
            todo &= todo - 1;
            const int ln = __shfl_sync(0xffffffffu, len, b);
            const int64_t sb = __shfl_sync(0xffffffffu, s, b);
            f(base + b, ln, (int)max64(c0 - sb, 0), (int)min64(c1 - sb, ln), sb, chunk);
        }
        before += __shfl_sync(0xffffffffu, x, 31);
    }
}

// One contiguous run of rows: where it starts, and how many of its rows the cache holds.
struct Run {
    const uint8_t *src;
    int rows;
};
__device__ __forceinline__ Run row_run(const CacheView &cv, int seq, int64_t pos, int n) {
    Run r = {nullptr, 0};
    if (n <= 0) return r;
    if (seq >= cv.n_seqs) {
        record_error(TQ_ERR_OUT_OF_RANGE);
        return r;
    }
    if (cv.page_tokens == 0) {
        r.rows = (int)max64(0, min64(n, cv.capacity - pos));
        r.src = cv.base + (seq * cv.capacity + pos) * (int64_t)cv.row_bytes;
        if (r.rows < n) record_error(TQ_ERR_OUT_OF_RANGE);
        return r;
    }
    const int pi = (int)(pos / cv.page_tokens), off = (int)(pos - (int64_t)pi * cv.page_tokens);
    const int64_t page = pi < cv.max_pages ? cv.page_table[(int64_t)seq * cv.max_pages + pi] : -1;
    if (page < 0 || page >= cv.n_pages) {
        record_error(TQ_ERR_OUT_OF_RANGE);
        return r;
    }
    r.rows = n;
    r.src = cv.base + (page * cv.page_tokens + off) * (int64_t)cv.row_bytes;
    return r;
}


// ------------------------------------------------------------------ shared memory
// Operand tiles in the no-swizzle canonical layouts (8 x 16-byte core matrices):
//   Q  [group of 4 blocks][(block, set, piece, head) row][coord], coords along K
//   K  [buffer][group][(block, token) row][coord], coords along K
//   V  [buffer][block][token][coord], coords contiguous (M)
//   P  [block][set][token][(piece, head)], 16 bytes per token (N contiguous)
// The K area holds the segment's output rows after the loop.
template <int NB, int SETS, bool DIRECT>
struct T4Smem {
    static constexpr int kKBuf = SETS == 1 ? 2 : 1;    // K operand buffers (what fits)
    static constexpr int kSBuf = SETS == 1 ? 2 : 1;    // score buffers in tensor memory
    static constexpr int kHeads = 4 * SETS;
    static constexpr int kQGroup = SETS * 8192, kKGroup = 16384, kVBlock = 4096, kPBlock = SETS * 512;
    static constexpr int q = 0;
    static constexpr int k = q + 2 * kQGroup;
    static constexpr int v = k + kKBuf * 2 * kKGroup;
    static constexpr int p = v + 2 * kSlice * kVBlock;
    static constexpr int ring = p + kSlice * kPBlock;
    static constexpr int norms = ring + (DIRECT ? 0 : kRing * 2 * kTile * kSliceRow);    // [slot][K/V][block][token] fp16
    static constexpr int newrow = norms + kNormSlots * 2 * kSlice * kTile * 2;           // [K/V] one row of 8 blocks
    static constexpr int qs = newrow + 2 * kSliceRow;                                     // [block][head] query scales
    static constexpr int al = qs + kSlice * kHeads * 4;                                   // [parity][block][head] factors
    static constexpr int moved = al + 2 * kSlice * kHeads * 4;                            // [parity][block] a factor is not 1
    static constexpr int ml = moved + 2 * kSlice;                               // [block][head] (m, l)
    static constexpr int pair = ml + kSlice * kHeads * 8;                                 // [block][token] scores, NB = 2
    static constexpr int bars = pair + (NB == 2 ? kSlice * kTile * kHeads * 4 : 0);
    static constexpr int total = bars + 256;
    static_assert(ring % 16 == 0 && norms % 16 == 0 && newrow % 16 == 0 && pair % 16 == 0 && bars % 16 == 0, "aligned areas");
    static_assert(total + 1024 <= (int)kSmemBudget, "one CTA per SM");
};
// The barriers and small words at `bars`.
struct T4Bars {
    uint64_t full[kRing];      // ring tile landed (K lane and V lane of warp 25)
    uint64_t ring_free[kRing]; // ring tile read (16 decode warps)
    uint64_t kfull[2], kfree[2];   // K operand written (8 warps) / read by the score products (commit)
    uint64_t vfull[2], pvdone[2];  // V operand written (8 warps) / value products done (commit)
    uint64_t sfull[2], sfree[2];   // scores ready (commit) / read (8 warps)
    uint64_t pfull;                // weights written, O rescaled (8 warps)
    uint64_t drain;                // every product done (commit), before tensor memory is released
    uint64_t epoch;
    uint32_t ring_mask[2][kRing];      // rows of a ring tile that the cache holds
    uint32_t mask[kNormSlots];         // rows of a tile that both caches hold, for the softmax
    uint32_t tmem;
    int gave_up;
};
static_assert(sizeof(T4Bars) <= 256, "bars area");

// 64 bytes of codes at a row's natural alignment.
__device__ __forceinline__ void load_codes(const uint8_t *s, int align, uint32_t (&c)[16]) {
    if (align % 16 == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 u = reinterpret_cast<const uint4 *>(s)[i];
            c[4 * i] = u.x, c[4 * i + 1] = u.y, c[4 * i + 2] = u.z, c[4 * i + 3] = u.w;
        }
    } else if (align % 8 == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint2 u = reinterpret_cast<const uint2 *>(s)[i];
            c[2 * i] = u.x, c[2 * i + 1] = u.y;
        }
    } else if (align % 4 == 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) c[i] = reinterpret_cast<const uint32_t *>(s)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            c[i] = reinterpret_cast<const uint16_t *>(s)[2 * i] | (uint32_t)reinterpret_cast<const uint16_t *>(s)[2 * i + 1] << 16;
    }
}

// ------------------------------------------------------------------ grid merge
// One sequence: every CTA stores its partial rows, turned back to the model's basis, as 64-bit
// words (value, tag), and its (m, l) per head likewise (an empty chunk stores m = -inf, l = 0 and
// no values); the tag is a hash of the epoch word at the start of the workspace.  Each CTA (or warp)
// then merges the (head, coordinates 4 l + c of one block) slices assigned to it, re-reading until
// every word carries this call's tag: a word is written and read whole, so a matching tag means a
// current value.  The first CTA advances the epoch once its first slice has the (m, l) of every
// CTA: every CTA has read the epoch by then.  A workspace whose epoch word
// lacks the initialisation mark first passes a barrier of per-CTA flags.  All waits are bounded.
template <int NTHREADS>
__device__ __forceinline__ void merge_grid(const T4Params &p, uint8_t *scratch, uint64_t E, bool marked,
                                           uint32_t e, uint32_t tag, int D, int n_rows) {
    constexpr int kWarps = NTHREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int PS = part_stride(D), Hq = p.n_q_heads;
    const int64_t rw = (int64_t)Hq * PS;
    const int n_ctas = gridDim.x, me = blockIdx.x;
    int *s_ok = reinterpret_cast<int *>(scratch);
    float *s_red = reinterpret_cast<float *>(scratch) + 32;    // [2][kWarps]
    float *s_w = s_red + 2 * kWarps;                           // [kGridMergeMaxCtas]
    float *s_acc = s_w + kGridMergeMaxCtas;                    // [kWarps][32]
    const uint64_t *part = reinterpret_cast<const uint64_t *>(p.part);
    if (!marked) {
        if (warp == 0) {
            const uint64_t token = (E + 1) * 0x9E3779B97F4A7C15ull;
            if (lane == 0) {
                __threadfence();
                st_relaxed_u64(p.bar + 1 + me, token);
            }
            bool all = false;
            for (uint32_t it = 0; it < p.grid_wait_limit && !all; ++it) {
                bool mine = true;
                for (int c = lane; c < n_ctas; c += 32) mine &= ld_relaxed_u64(p.bar + 1 + c) == token;
                all = __all_sync(0xffffffffu, mine);
            }
            __threadfence();
            if (lane == 0) *s_ok = all ? 1 : 0;
        }
        __syncthreads();
        if (!*s_ok) {
            if (tid == 0) record_error(TQ_ERR_DEVICE_TIMEOUT);
            if (me == 0 && tid == 0) st_relaxed_u64(p.bar, ((uint64_t)kEpochMark << 32) | (e + 1u));
            return;
        }
    }
    constexpr int kRows = (kGridMergeMaxCtas + kWarps - 1) / kWarps;
    const int SL = D / 32, n_items = Hq * SL;
    bool advanced = false;
    // Few CTAs have many slices each: a warp merges one by itself then, a lane holding each CTA's
    // (m, l).  32 heads over 64, 257, 1,000 rows (2, 9, 32 CTAs): 11.3, 12.1, 11.8 us; by whole CTAs
    // 49.6, 19.3, 11.8.
    if (n_ctas <= 32) {
        constexpr int kFly = 8;   // rows in flight
        for (int item = me * kWarps + warp; item < n_items; item += n_ctas * kWarps) {
            const int sl = item % SL, hh = item / SL;
            const uint64_t *base = part + (int64_t)hh * PS;
            uint64_t wm = 0, wl = 0;
            bool done = false;
            for (uint32_t it = 0; it < p.grid_wait_limit && !done; ++it) {
                bool mine = true;
                if (lane < n_ctas) {
                    wm = ld_relaxed_u64(base + lane * rw + D);
                    wl = ld_relaxed_u64(base + lane * rw + D + 1);
                    mine = (uint32_t)(wm >> 32) == tag && (uint32_t)(wl >> 32) == tag;
                }
                done = __all_sync(0xffffffffu, mine);
            }
            if (done && item == 0 && lane == 0) {   // warp 0 of CTA 0: every CTA has read the epoch
                st_relaxed_u64(p.bar, ((uint64_t)kEpochMark << 32) | (e + 1u));
                advanced = true;
            }
            const float m = lane < n_ctas ? __uint_as_float((uint32_t)wm) : -INFINITY;
            const float l = lane < n_ctas ? __uint_as_float((uint32_t)wl) : 0.f;
            float M = m;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            const float w = m == -INFINITY ? 0.f : __expf(m - M);
            float L = w * l;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
            float acc = 0.f;
            for (int r0 = 0; r0 < n_rows && done; r0 += kFly) {
                float ov[kFly];
                done = false;
                for (uint32_t it = 0; it < p.grid_wait_limit && !done; ++it) {
                    bool mine = true;
#pragma unroll
                    for (int k = 0; k < kFly; ++k) {
                        const int r = r0 + k;
                        const uint64_t wv = r < n_rows ? ld_relaxed_u64(base + r * rw + 32 * sl + lane) : (uint64_t)tag << 32;
                        mine &= (uint32_t)(wv >> 32) == tag;
                        ov[k] = __uint_as_float((uint32_t)wv);
                    }
                    done = __all_sync(0xffffffffu, mine);
                }
#pragma unroll
                for (int k = 0; k < kFly; ++k) {
                    const float wr = __shfl_sync(0xffffffffu, w, (r0 + k) & 31);
                    if (r0 + k < n_rows) acc = fmaf(wr, ov[k], acc);
                }
            }
            if (!done) {
                if (lane == 0) record_error(TQ_ERR_DEVICE_TIMEOUT);
                break;
            }
            const float inv = L != 0.f ? kInvSqrt128 / L : 0.f;   // a NaN sum stays one
            store_out(p.out, (int64_t)hh * D + kBlock * (sl >> 2) + 4 * lane + (sl & 3), acc * inv);
        }
        if (me == 0 && tid == 0 && !advanced) st_relaxed_u64(p.bar, ((uint64_t)kEpochMark << 32) | (e + 1u));
        return;
    }
    for (int item = me; item < n_items; item += n_ctas) {
        const int sl = item % SL, hh = item / SL;
        const uint64_t *base = part + (int64_t)hh * PS;
        float ov[kRows];
        float2 ml = make_float2(-INFINITY, 0.f);
        bool done = false;
        for (uint32_t it = 0; it < p.grid_wait_limit && !done; ++it) {
            bool mine = true;
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int r = warp + kWarps * k;
                const uint64_t wv = r < n_rows ? ld_relaxed_u64(base + r * rw + 32 * sl + lane) : (uint64_t)tag << 32;
                mine &= (uint32_t)(wv >> 32) == tag;
                ov[k] = __uint_as_float((uint32_t)wv);
            }
            if (tid < n_ctas) {
                const uint64_t wm = ld_relaxed_u64(base + tid * rw + D);
                const uint64_t wl = ld_relaxed_u64(base + tid * rw + D + 1);
                mine &= (uint32_t)(wm >> 32) == tag && (uint32_t)(wl >> 32) == tag;
                ml = make_float2(__uint_as_float((uint32_t)wm), __uint_as_float((uint32_t)wl));
            }
            done = __syncthreads_and(mine) != 0;
        }
        if (!done) {
            if (tid == 0) record_error(TQ_ERR_DEVICE_TIMEOUT);
            break;
        }
        if (me == 0 && tid == 0 && !advanced) {
            st_relaxed_u64(p.bar, ((uint64_t)kEpochMark << 32) | (e + 1u));
            advanced = true;
        }
        float mx = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0) s_red[warp] = mx;
        __syncthreads();
        float M = s_red[0];
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_red[w]);
        const float wr = ml.x == -INFINITY ? 0.f : __expf(ml.x - M);
        if (tid < n_ctas) s_w[tid] = wr;
        float lw = wr * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
        if (lane == 0) s_red[kWarps + warp] = lw;
        __syncthreads();
        float acc = 0.f;
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int r = warp + kWarps * k;
            if (r < n_rows) acc = fmaf(s_w[r], ov[k], acc);
        }
        s_acc[warp * 32 + lane] = acc;
        __syncthreads();
        if (warp == 0) {
            float L = 0.f, o = 0.f;
            for (int w = 0; w < kWarps; ++w) {
                L += s_red[kWarps + w];
                o += s_acc[w * 32 + lane];
            }
            const float inv = L != 0.f ? kInvSqrt128 / L : 0.f;   // a NaN sum stays one
            store_out(p.out, (int64_t)hh * D + kBlock * (sl >> 2) + 4 * lane + (sl & 3), o * inv);
        }
        __syncthreads();   // the scratch is reused by the next item
    }
    if (me == 0 && tid == 0 && !advanced) st_relaxed_u64(p.bar, ((uint64_t)kEpochMark << 32) | (e + 1u));
}

// ------------------------------------------------------------------ the kernel
template <int NB, int SETS, bool APPEND, bool DIRECT>
__global__ void __launch_bounds__(kT4Threads, 1) attn_t4_kernel(const __grid_constant__ T4Params p) {
    using L = T4Smem<NB, SETS, DIRECT>;
    constexpr int D = NB * kBlock, PS = part_stride(D), kHeads = L::kHeads, kKBuf = L::kKBuf, kSBuf = L::kSBuf;
    constexpr uint32_t kTmemCols = 512, kTmemO = 256;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    T4Bars &B = *reinterpret_cast<T4Bars *>(smem + L::bars);
    volatile int *gave_up = &B.gave_up;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = p.group, Hq = p.n_q_heads, bpr = p.bpr;
    const int n_slices = (bpr + kSlice - 1) / kSlice;
    const int slice = (int)blockIdx.x % n_slices;
    const int64_t chunk_id = blockIdx.x / n_slices;
    const int blk_base = slice * kSlice, nblk = min(kSlice, bpr - blk_base);   // this CTA's blocks of a row
    const int head_base = blk_base / NB * G;                                   // and their first query head
    float *qs = reinterpret_cast<float *>(smem + L::qs);
    float *al = reinterpret_cast<float *>(smem + L::al);
    uint8_t *moved = smem + L::moved;
    float2 *ml = reinterpret_cast<float2 *>(smem + L::ml);
    uint16_t *norms = reinterpret_cast<uint16_t *>(smem + L::norms);
    auto norm_at = [&](int slot, int c, int blk) { return norms + ((slot * 2 + c) * kSlice + blk) * kTile; };

    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            tc_bar_init(smem_u32(&B.full[i]), 2);
            tc_bar_init(smem_u32(&B.ring_free[i]), 2 * kDecWarps);
        }
        for (int i = 0; i < 2; ++i) {
            tc_bar_init(smem_u32(&B.kfull[i]), kDecWarps);
            tc_bar_init(smem_u32(&B.kfree[i]), 1);
            tc_bar_init(smem_u32(&B.vfull[i]), kDecWarps);
            tc_bar_init(smem_u32(&B.pvdone[i]), 1);
            tc_bar_init(smem_u32(&B.sfull[i]), 1);
            tc_bar_init(smem_u32(&B.sfree[i]), kSoftWarps);
        }
        tc_bar_init(smem_u32(&B.pfull), kSoftWarps);
        tc_bar_init(smem_u32(&B.drain), 2);
        B.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        // first reads into L2 while the kernel before this one ends
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.seq_lens));
        if (p.n_seqs == 1) {
            l2_prefetch(p.q, (uint32_t)(Hq * D * 2));
            if (APPEND) {
                l2_prefetch(p.k_new, (uint32_t)(bpr * kBlock * 2));
                l2_prefetch(p.v_new, (uint32_t)(bpr * kBlock * 2));
            }
        }
    }
    if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&B.tmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem;
    pdl_wait();
    pdl_launch_dependents();

    uint64_t epoch_word = 0;
    if (p.bar && tid == 0) epoch_word = ld_relaxed_u64(p.bar);
    if (p.withhold_tiles && DIRECT && tid == 0) {   // injected fault, no tile copies to withhold
        record_error(TQ_ERR_DEVICE_TIMEOUT);
        *gave_up = 1;
    }
    int n_rows = 0;   // one sequence: chunks that hold rows
    int it = 0;       // tiles of the segments before
    for_segments(p, chunk_id, p.n_chunks, [&](int seq, int len, int lo, int hi, int64_t sbase, int64_t chunk) {
        const int span = hi - lo, n_tiles = (span + kTile - 1) / kTile;
        const bool owner = APPEND && span > 0 && hi == len;   // the chunk holds the new row
        // ================= warp 25: the rows of tiles from .. to - 1; lanes 2k and 2k + 1 form the
        // copies of the k-th tile of a batch, for K and for V
        auto copy_tiles = [&](int from, int to) {
            const int c = lane & 1;
            const CacheView &cv = c ? p.vc : p.kc;
            for (int t0 = from; t0 < to; t0 += 16) {
                const int i = t0 + (lane >> 1);
                Run a = {nullptr, 0}, b = {nullptr, 0};
                int na = 0;
                uint32_t mask = 0;
                if (i < to) {
                    const int64_t pos = (int64_t)lo + i * kTile;
                    int rows = min(kTile, span - i * kTile);
                    const bool with_new = owner && i == n_tiles - 1;
                    if (with_new) --rows;   // the new row comes from this CTA
                    na = rows;
                    if (cv.page_tokens) na = (int)min64(rows, cv.page_tokens - pos % cv.page_tokens);
                    a = row_run(cv, seq, pos, na);
                    b = row_run(cv, seq, pos + na, rows - na);
                    mask = (a.rows ? 0xffffffffu >> (32 - a.rows) : 0u) | (b.rows ? (0xffffffffu >> (32 - b.rows)) << na : 0u) |
                           (with_new ? 1u << rows : 0u);
                }
                for (int k = 0; k < 16 && t0 + k < to; ++k) {
                    const int u = it + t0 + k, s = u % kRing;
                    if (u >= kRing) t4_wait(&B.ring_free[s], (uint32_t)((u / kRing - 1) & 1), p.wait_limit, gave_up);
                    __syncwarp();
                    if (*gave_up) return;
                    if (lane >> 1 == k) {
                        const uint32_t bar = smem_u32(&B.full[s]);
                        uint8_t *dst = smem + L::ring + (s * 2 + c) * (kTile * kSliceRow);
                        const uint32_t ba = (uint32_t)(a.rows * kSliceRow), bb = (uint32_t)(b.rows * kSliceRow);
                        B.ring_mask[c][s] = mask;
                        asm volatile("mbarrier.expect_tx.shared.b64 [%0], %1;\n" ::"r"(bar), "r"(ba + bb) : "memory");
                        if (ba) bulk_g2s(smem_u32(dst), a.src, ba, bar);
                        if (bb) bulk_g2s(smem_u32(dst + (size_t)na * kSliceRow), b.src, bb, bar);
                        mbar_arrive(bar);
                    }
                }
            }
        };
        // the first tiles before the queries are ready (the ring is empty between segments)
        const int n_first = min(n_tiles, kRing);
        if (!DIRECT && warp == kWarpTma && !p.withhold_tiles) copy_tiles(0, n_first);
        // ================= decode warps: the queries' pieces, and the new row's blocks
        if (warp >= kWarpK && warp < kWarpMma && span > 0) {
            const int dw = warp - kWarpK;
            constexpr int kDw = 2 * kDecWarps;
            const int items = nblk * kHeads;
            for (int i0 = dw; i0 < items; i0 += 2 * kDw) {
                uint2 raw[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = i0 + k * kDw, blk = i / kHeads, h = i - blk * kHeads;
                    raw[k] = i < items && h < G
                                 ? *reinterpret_cast<const uint2 *>(p.q + (((int64_t)seq * Hq + head_base + blk / NB * G + h) * NB + blk % NB) * kBlock + 4 * lane)
                                 : make_uint2(0u, 0u);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = i0 + k * kDw, blk = i / kHeads, h = i - blk * kHeads;
                    if (i >= items) break;
                    const float2 f01 = __half22float2(*reinterpret_cast<const __half2 *>(&raw[k].x));
                    const float2 f23 = __half22float2(*reinterpret_cast<const __half2 *>(&raw[k].y));
                    float v[4] = {f01.x, f01.y, f23.x, f23.y};
                    apply_signs4(v, p.kc, 4 * lane);
                    warp_fwht4(v, lane);
                    float mx = 0.f;
                    bool bad = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] *= p.score_scale;
                        mx = fmaxf(mx, fabsf(v[e]));
                        bad |= !(fabsf(v[e]) < INFINITY);
                    }
                    mx = warp_max(mx);
                    bad = __any_sync(0xffffffffu, bad);
                    // largest magnitude into [128, 256): a power of two, undone through qs
                    const int up = min(134 - (int)(__float_as_uint(mx) >> 23), 120);
                    const float sc = __uint_as_float((uint32_t)(127 + up) << 23);
                    if (lane == 0) qs[blk * kHeads + h] = bad ? NAN : __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = bad ? 0.f : v[e] * sc;
                    const int n0 = ((blk & 3) * SETS + (h >> 2)) * 16 + (h & 3);
                    uint8_t *dst = smem + L::q + (blk >> 2) * L::kQGroup + (lane >> 2) * 128 + 4 * (lane & 3);
#pragma unroll
                    for (int pi = 0; pi < 4; ++pi) {
                        uint16_t a, b;
                        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(v[1]), "f"(v[0]));
                        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(v[3]), "f"(v[2]));
                        const int n = n0 + 4 * pi;
                        *reinterpret_cast<uint32_t *>(dst + (n >> 3) * 1024 + (n & 7) * 16) = (uint32_t)a | (uint32_t)b << 16;
                        const uint32_t ha = e4m3_to_half2(a), hb = e4m3_to_half2(b);
                        const float2 fa = __half22float2(*reinterpret_cast<const __half2 *>(&ha));
                        const float2 fb = __half22float2(*reinterpret_cast<const __half2 *>(&hb));
                        v[0] = (v[0] - fa.x) * 16.f;
                        v[1] = (v[1] - fa.y) * 16.f;
                        v[2] = (v[2] - fb.x) * 16.f;
                        v[3] = (v[3] - fb.y) * 16.f;
                    }
                }
            }
            if (owner) {   // append: encode the new K and V rows, one warp per block
                for (int bi = dw; bi < 2 * nblk; bi += kDw) {
                    const int c = bi >= nblk ? 1 : 0, jb = bi - c * nblk;
                    const CacheView &cv = c ? p.vc : p.kc;
                    const uint2 raw = warp_block_load((c ? p.v_new : p.k_new) + ((int64_t)seq * bpr + blk_base + jb) * kBlock, lane);
                    uint8_t *row = nullptr;
                    if (lane == 0) row = row_ptr(cv, seq, len - 1);
                    row = reinterpret_cast<uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(row), 0));
                    const WarpBlock wb = warp_encode_raw<kT4>(raw, cv, lane);
                    if (row) warp_store_block<kT4>(row, blk_base + jb, bpr, wb, lane);
                    warp_store_block<kT4>(smem + L::newrow + c * kSliceRow, jb, kSlice, wb, lane);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the query operand
        }
        __syncthreads();

        if (warp < kSoftWarps) {
            // ================= softmax: warp = block, lane = token
            const int quad = warp & 3, grp = warp >> 2;
            const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
            const bool active = warp < nblk;
            float m_run[kHeads], off[kHeads], l_run[kHeads], qsc[kHeads];
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                m_run[h] = -INFINITY;
                off[h] = 0.f;   // kWeightUp - m_run once there is a maximum
                l_run[h] = 0.f;
                qsc[h] = active && span > 0 ? qs[warp * kHeads + h] : 0.f;
            }
            for (int i = 0; i < n_tiles; ++i) {
                const int u = it + i, sb = u % kSBuf, slot = u % kNormSlots;
                t4_wait(&B.sfull[sb], (uint32_t)((u / kSBuf) & 1), p.wait_limit, gave_up);
                tc_fence_after();
                float s[kHeads];
                const float kn = __half2float(__ushort_as_half(norm_at(slot, 0, warp)[lane]));
#pragma unroll
                for (int set = 0; set < SETS; ++set) {
                    float r[16];
                    tc_ld16(tmem + lane_base + (uint32_t)(128 * SETS * sb + 64 * SETS * grp + 16 * (SETS * quad + set)), r);
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        s[4 * set + h] = fmaf(fmaf(fmaf(r[12 + h], kDown, r[8 + h]), kDown, r[4 + h]), kDown, r[h]) * (kn * qsc[4 * set + h]);
                }
                const uint32_t mask = B.mask[slot];
                const bool on = active && ((mask >> lane) & 1);
                const float vn = on ? __half2float(__ushort_as_half(norm_at(slot, 1, warp)[lane])) : 0.f;
                float w = fmaxf(vn, 5.9604645e-8f);   // 2^-24: no fp16 norm but 0 lies below it
                if (NB == 2 && on) w = fmaxf(w, __half2float(__ushort_as_half(norm_at(slot, 1, warp ^ 1)[lane])));
                tc_fence_before();
                __syncwarp();
                if (lane == 0) tc_arrive(smem_u32(&B.sfree[sb]));
                if (NB == 2) {   // the other block's share of the scores
                    float4 *x = reinterpret_cast<float4 *>(smem + L::pair);
#pragma unroll
                    for (int set = 0; set < SETS; ++set)
                        x[(warp * SETS + set) * kTile + lane] = make_float4(s[4 * set], s[4 * set + 1], s[4 * set + 2], s[4 * set + 3]);
                    pair_sync(warp);
#pragma unroll
                    for (int set = 0; set < SETS; ++set) {
                        const float4 o = x[((warp ^ 1) * SETS + set) * kTile + lane];
                        s[4 * set] += o.x;
                        s[4 * set + 1] += o.y;
                        s[4 * set + 2] += o.z;
                        s[4 * set + 3] += o.w;
                    }
                }
                const float lw = lg2(w);
                float ph[kHeads], mxh[kHeads];
                bool move = false;
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    s[h] = on ? s[h] : -INFINITY;
                    const float mx = warp_max(s[h] + lw);
                    mxh[h] = mx;
                    move |= mx > m_run[h] + kLag;   // (also the first maximum: m_run is -inf)
                }
                if (move) {   // publish the factors of O
#pragma unroll
                    for (int h = 0; h < kHeads; ++h) {
                        float alpha = 1.f;
                        if (mxh[h] > m_run[h] + kLag) {
                            alpha = ex2(m_run[h] - mxh[h]);
                            m_run[h] = mxh[h];
                            off[h] = kWeightUp - mxh[h];
                            l_run[h] *= alpha;
                        }
                        if (lane == 0) al[((u & 1) * kSlice + warp) * kHeads + h] = alpha;
                    }
                }
                if (lane == 0) moved[(u & 1) * kSlice + warp] = move;
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    ph[h] = ex2(s[h] + off[h]);
                    l_run[h] += ph[h];
                }
                // 64 p |v| of this token, cut in three pieces: 16 bytes (piece, head) per set
                uint4 pieces[SETS];
#pragma unroll
                for (int set = 0; set < SETS; ++set) {
                    const uint32_t ha = pack_half2(ph[4 * set] * vn, ph[4 * set + 1] * vn);
                    const uint32_t hb = pack_half2(ph[4 * set + 2] * vn, ph[4 * set + 3] * vn);
                    const uint32_t a0 = e4m3_of_half2(ha), b0 = e4m3_of_half2(hb);
                    const uint32_t ra = rest16(ha, a0), rb = rest16(hb, b0);
                    const uint32_t a1 = e4m3_of_half2(ra), b1 = e4m3_of_half2(rb);
                    const uint32_t a2 = e4m3_of_half2(rest16(ra, a1)), b2 = e4m3_of_half2(rest16(rb, b1));
                    pieces[set] = make_uint4(prmt(a0, b0, 0x5410), prmt(a1, b1, 0x5410), prmt(a2, b2, 0x5410), 0u);
                }
                // the last tile's value products are done: O is still, the weights' buffer is free
                if (i > 0) t4_wait(&B.pvdone[(u - 1) & 1], (uint32_t)(((u - 1) >> 1) & 1), p.wait_limit, gave_up);
                if (active) {
#pragma unroll
                    for (int set = 0; set < SETS; ++set)
                        *reinterpret_cast<uint4 *>(smem + L::p + warp * L::kPBlock + set * 512 + lane * 16) = pieces[set];
                }
                softmax_sync();   // every block's factors are published
                const uint2 mv = *reinterpret_cast<const uint2 *>(moved + (u & 1) * kSlice);
                const uint32_t mine = grp ? mv.y : mv.x;
                if (i > 0 && mine) {
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        if (!((mine >> (8 * k)) & 1)) continue;
                        const int blk = 4 * grp + k;
                        const float *a = al + ((u & 1) * kSlice + blk) * kHeads;
#pragma unroll
                        for (int set = 0; set < SETS; ++set) {
                            const float4 f = *reinterpret_cast<const float4 *>(a + 4 * set);
                            const uint32_t at = tmem + lane_base + kTmemO + (uint32_t)(16 * (SETS * blk + set));
                            float r[16];
                            uint32_t o[16];
                            tc_ld16(at, r);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(r[e] * ((e & 3) == 0 ? f.x : (e & 3) == 1 ? f.y : (e & 3) == 2 ? f.z : f.w));
                            tc_st16(at, o);
                        }
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) tc_arrive(smem_u32(&B.pfull));
            }
            // ---- the segment's sums: O of this quarter's 32 coordinates, m and l
            if (n_tiles > 0) {
                const int u = it + n_tiles - 1;
                t4_wait(&B.pvdone[u & 1], (uint32_t)((u >> 1) & 1), p.wait_limit, gave_up);
            }
            tc_fence_after();
            const bool good = n_tiles > 0 && !*gave_up;
            float *rows = reinterpret_cast<float *>(smem + L::k);
#pragma unroll 1
            for (int blk = 4 * grp; blk < min(4 * grp + 4, nblk); ++blk) {
#pragma unroll
                for (int set = 0; set < SETS; ++set) {
                    float r[16];
                    tc_ld16(tmem + lane_base + kTmemO + (uint32_t)(16 * (SETS * blk + set)), r);
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        if (4 * set + h < G)
                            rows[(blk / NB * G + 4 * set + h) * D + blk % NB * kBlock + 32 * quad + lane] =
                                good ? fmaf(fmaf(r[8 + h], kDown, r[4 + h]), kDown, r[h]) * kE4m3Step4 : 0.f;
                }
            }
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], o);
                if (lane == 0) ml[warp * kHeads + h] = good ? make_float2(m_run[h] == -INFINITY ? -INFINITY : m_run[h] * kLn2, l_run[h]) : make_float2(-INFINITY, 0.f);
            }
            tc_fence_before();
        } else if (warp < kWarpMma) {
            // ================= decode: thread = (block, token) of K or of V
            const int c = warp >= kWarpV ? 1 : 0, blk = (warp - kWarpK) & (kDecWarps - 1);
            const bool active = blk < nblk;
            const CacheView &cv = c ? p.vc : p.kc;
            const int R = cv.row_bytes, codes_at = (blk_base + blk) * kCodeBytes4, norm_off = bpr * kCodeBytes4 + 2 * (blk_base + blk);
            // the K warps hand both caches' norms and the tile's mask to the softmax
            uint32_t nx[16];      // DIRECT: the next tile's codes, norms and presence
            uint32_t nx_norm = 0;
            bool nx_on = false;
            auto load = [&](int i) {
                const int64_t t = (int64_t)i * kTile + lane;
                nx_on = false;
                nx_norm = 0;
                if (active && t < span) {
                    if (owner && lo + t == len - 1) {
                        nx_on = true;
                        const uint8_t *s = smem + L::newrow + c * kSliceRow;
                        load_codes(s + blk * kCodeBytes4, 16, nx);
                        if (c == 0) nx_norm = *reinterpret_cast<const uint16_t *>(s + kSlice * kCodeBytes4 + 2 * blk) |
                                              (uint32_t)*reinterpret_cast<const uint16_t *>(s + kSliceRow + kSlice * kCodeBytes4 + 2 * blk) << 16;
                    } else {
                        const Run r = row_run(cv, seq, lo + t, 1);
                        if (r.rows) {
                            nx_on = true;
                            load_codes(r.src + codes_at, R, nx);
                        }
                        if (c == 0 && r.rows) {
                            const Run rv = row_run(p.vc, seq, lo + t, 1);
                            nx_on = rv.rows != 0;
                            if (nx_on) nx_norm = *reinterpret_cast<const uint16_t *>(r.src + norm_off) |
                                                 (uint32_t)*reinterpret_cast<const uint16_t *>(rv.src + norm_off) << 16;
                        }
                    }
                }
            };
            if (DIRECT) {
#pragma unroll
                for (int e = 0; e < 16; ++e) nx[e] = 0;
                if (n_tiles > 0) load(0);
            }
            for (int i = 0; i < n_tiles; ++i) {
                const int u = it + i, slot = u % kNormSlots;
                uint32_t w[16];
                uint32_t norm;
                if (DIRECT) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = nx[e];
                    norm = nx_norm;
                    const unsigned on = __ballot_sync(0xffffffffu, nx_on);
                    if (i + 1 < n_tiles) load(i + 1);
                    if (c == 0) {
                        if (u >= kKBuf) t4_wait(&B.kfree[u % kKBuf], (uint32_t)((u / kKBuf - 1) & 1), p.wait_limit, gave_up);
                    } else if (u >= 2) {
                        t4_wait(&B.pvdone[u & 1], (uint32_t)(((u >> 1) - 1) & 1), p.wait_limit, gave_up);
                    }
                    if (c == 0 && blk == 0 && lane == 0) B.mask[slot] = on;
                } else {
                    const int s = u % kRing;
                    t4_wait(&B.full[s], (uint32_t)((u / kRing) & 1), p.wait_limit, gave_up);
                    const uint8_t *row = owner && lo + i * kTile + lane == len - 1 ? smem + L::newrow + c * kSliceRow
                                                                                 : smem + L::ring + (s * 2 + c) * (kTile * kSliceRow) + lane * kSliceRow;
                    load_codes(row + blk * kCodeBytes4, 16, w);
                    norm = 0;
                    uint32_t mask = 0;
                    if (c == 0) {   // K and V rows of a token lie one cache apart in the ring and in the new row
                        const uint8_t *vrow = row + (row >= smem + L::ring && row < smem + L::norms ? kTile * kSliceRow : kSliceRow);
                        norm = *reinterpret_cast<const uint16_t *>(row + kSlice * kCodeBytes4 + 2 * blk) |
                               (uint32_t)*reinterpret_cast<const uint16_t *>(vrow + kSlice * kCodeBytes4 + 2 * blk) << 16;
                        mask = B.ring_mask[0][s] & B.ring_mask[1][s];
                    }
                    // (the values are in registers before the tile is given back)
                    asm volatile("" ::"r"(w[0]), "r"(w[4]), "r"(w[8]), "r"(w[12]), "r"(norm), "r"(mask) : "memory");
                    __syncwarp();
                    if (lane == 0) tc_arrive(smem_u32(&B.ring_free[s]));
                    if (c == 0) {
                        if (u >= kKBuf) t4_wait(&B.kfree[u % kKBuf], (uint32_t)((u / kKBuf - 1) & 1), p.wait_limit, gave_up);
                    } else if (u >= 2) {
                        t4_wait(&B.pvdone[u & 1], (uint32_t)(((u >> 1) - 1) & 1), p.wait_limit, gave_up);
                    }
                    if (c == 0 && blk == 0 && lane == 0) B.mask[slot] = mask;
                }
                if (c == 0) {
                    norm_at(slot, 0, blk)[lane] = (uint16_t)norm;
                    norm_at(slot, 1, blk)[lane] = (uint16_t)(norm >> 16);
                }
                const int row = 32 * (blk & 3) + lane;   // of the group's K operand
                uint8_t *dst = c ? smem + L::v + ((u & 1) * kSlice + blk) * L::kVBlock + (lane >> 3) * 1024 + (lane & 7) * 16
                                 : smem + L::k + ((u % kKBuf) * 2 + (blk >> 2)) * L::kKGroup + (row >> 3) * 1024 + (row & 7) * 16;
                if (active) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {   // 16 coordinates
                        uint32_t o0, o1, o2, o3;
                        e4m3x8(w[2 * e], o0, o1);
                        e4m3x8(w[2 * e + 1], o2, o3);
                        *reinterpret_cast<uint4 *>(dst + 128 * e) = make_uint4(o0, o1, o2, o3);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) tc_arrive(smem_u32(c ? &B.vfull[u & 1] : &B.kfull[u % kKBuf]));
            }
        } else if (warp == kWarpTma) {
            if (!DIRECT && !p.withhold_tiles) copy_tiles(n_first, n_tiles);
        } else if (warp == kWarpMma) {
            // ================= score products
            constexpr uint32_t idesc_s = idesc_f8(64 * SETS, false, false);
            const uint32_t base = smem_u32(smem);
            const uint64_t dk = sdesc(base + L::k, 128, 1024), dq = sdesc(base + L::q, 128, 1024);
            for (int i = 0; i < n_tiles; ++i) {
                const int u = it + i;
                t4_wait(&B.kfull[u % kKBuf], (uint32_t)((u / kKBuf) & 1), p.wait_limit, gave_up);
                if (u >= kSBuf) t4_wait(&B.sfree[u % kSBuf], (uint32_t)((u / kSBuf - 1) & 1), p.wait_limit, gave_up);
                __syncwarp();
                tc_fence_after();
                const uint64_t da = dk + (uint64_t)((u % kKBuf) * 2 * (L::kKGroup >> 4));
                const uint32_t d = tmem + (uint32_t)(128 * SETS * (u % kSBuf));
                if (elect_one()) {
#pragma unroll
                    for (int grp = 0; grp < 2; ++grp)
                        if (4 * grp < nblk)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)   // 32 coordinates
                                mma_f8(d + 64u * SETS * grp, da + (uint64_t)(grp * (L::kKGroup >> 4) + 16 * ks),
                                       dq + (uint64_t)(grp * (L::kQGroup >> 4) + 16 * ks), idesc_s, ks > 0);
                    tc_commit(smem_u32(&B.sfull[u % kSBuf]));
                    tc_commit(smem_u32(&B.kfree[u % kKBuf]));
                }
                __syncwarp();
            }
        } else {
            // ================= value products
            constexpr uint32_t idesc_pv = idesc_f8(16 * SETS, true, true);
            const uint32_t base = smem_u32(smem);
            const uint64_t dv = sdesc(base + L::v, 1024, 128), dp = sdesc(base + L::p, 128, 512);
            for (int i = 0; i < n_tiles; ++i) {
                const int u = it + i;
                t4_wait(&B.vfull[u & 1], (uint32_t)((u >> 1) & 1), p.wait_limit, gave_up);
                t4_wait(&B.pfull, (uint32_t)(u & 1), p.wait_limit, gave_up);
                __syncwarp();
                tc_fence_after();
                const uint64_t da = dv + (uint64_t)((u & 1) * kSlice * (L::kVBlock >> 4));
                if (elect_one()) {
                    const uint32_t more = i > 0;
#pragma unroll
                    for (int blk = 0; blk < kSlice; ++blk)
                        if (blk < nblk)
                            mma_f8(tmem + kTmemO + (uint32_t)(16 * SETS * blk), da + (uint64_t)(blk * (L::kVBlock >> 4)),
                                   dp + (uint64_t)(blk * (L::kPBlock >> 4)), idesc_pv, more);
                    tc_commit(smem_u32(&B.pvdone[u & 1]));
                }
                __syncwarp();
            }
        }
        __syncthreads();
        tc_fence_after();
        // ================= the segment's rows leave
        const float *rows = reinterpret_cast<const float *>(smem + L::k);
        const int n_out = nblk / NB * G * NB;   // (head, block) rows of 128
        if (p.bar) {
            if (tid == 0) B.epoch = epoch_word;
            __syncthreads();
            const uint64_t E = B.epoch;
            const uint32_t e0 = (uint32_t)(E >> 32) == kEpochMark ? (uint32_t)E : 0u;
            const uint32_t tag = (e0 + 1u) * 0x9E3779B9u;
            n_rows = (int)min64(p.n_chunks, ((int64_t)len + chunk - 1) / chunk);
            uint64_t *dst = reinterpret_cast<uint64_t *>(p.part) + chunk_id * Hq * PS;
            for (int i = warp; i < n_out && span > 0; i += kT4Warps) {
                const int h = i / NB, b = i - h * NB;
                const float4 x = *reinterpret_cast<const float4 *>(rows + h * D + b * kBlock + 4 * lane);
                float v[4] = {x.x, x.y, x.z, x.w};
                warp_fwht4(v, lane);
                apply_signs4(v, p.vc, 4 * lane);
                // coordinate 4 lane + c at word 32 c + lane: every store is one 256-byte run
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    st_relaxed_u64(dst + (int64_t)h * PS + b * kBlock + 32 * c + lane, tagged(v[c], tag));
            }
            for (int h = tid; h < Hq; h += kT4Threads) {
                const float2 a = ml[h / G * NB * kHeads + h % G];
                st_relaxed_u64(dst + (int64_t)h * PS + D, tagged(a.x, tag));
                st_relaxed_u64(dst + (int64_t)h * PS + D + 1, tagged(a.y, tag));
            }
        } else {
            float *dst = p.part + ((chunk_id + seq) * Hq + head_base) * PS;
            for (int i = warp; i < n_out && span > 0; i += kT4Warps) {
                const int h = i / NB, b = i - h * NB;
                *reinterpret_cast<float4 *>(dst + (int64_t)h * PS + b * kBlock + 4 * lane) =
                    *reinterpret_cast<const float4 *>(rows + h * D + b * kBlock + 4 * lane);
            }
            for (int h = tid; h < nblk / NB * G && span > 0; h += kT4Threads)
                *reinterpret_cast<float2 *>(dst + (int64_t)h * PS + D) = ml[h / G * NB * kHeads + h % G];
            if (tid == 0 && slice == 0 && lo == 0)
                p.seg[seq] = make_int2((int)(sbase / chunk), (int)((sbase + len - 1) / chunk));
        }
        it += n_tiles;
        __syncthreads();   // the rows have been read: the operand areas are free for the next segment
    });
    if ((warp == kWarpMma || warp == kWarpPv) && elect_one()) {   // every product has completed before the memory goes
        tc_commit(smem_u32(&B.drain));
        for (uint32_t n = 0; n < kDrainPolls && !tc_test(smem_u32(&B.drain), 0); ++n) {}
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    if (p.bar) {
        const uint64_t E = B.epoch;
        const bool marked = (uint32_t)(E >> 32) == kEpochMark;
        const uint32_t e = marked ? (uint32_t)E : 0u;
        merge_grid<kT4Threads>(p, smem, E, marked, e, (e + 1u) * 0x9E3779B9u, D, n_rows);
    }
}

// Batch: merge the partial rows of one (head, sequence, block).  A warp takes every fourth row,
// eight loads in flight; the warps meet in shared memory and warp 0 undoes the rotation.
constexpr int kMergeWarps = 4, kMergeInFlight = 8;

__global__ void __launch_bounds__(32 * kMergeWarps) attn_t4_merge_kernel(const __grid_constant__ T4Params p, int D) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ float red_m[kMergeWarps], red_l[kMergeWarps];
    __shared__ float4 red_o[kMergeWarps][32];
    const int h = blockIdx.x, seq = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t at = ((int64_t)seq * p.n_q_heads + h) * D + b * kBlock + 4 * lane;
    if (min(p.seq_lens[seq], p.max_len) <= 0) {   // no chunk holds rows of it
        if (warp == 0) store_out4(p.out, at, 0.f, 0.f, 0.f, 0.f);
        return;
    }
    const int2 seg = p.seg[seq];
    const int64_t rw = (int64_t)p.n_q_heads * part_stride(D);
    const float *base = p.part + ((int64_t)(seg.x + seq) * p.n_q_heads + h) * part_stride(D);
    const int R = seg.y - seg.x + 1;
    float M = -INFINITY, ls = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r0 = warp; r0 < R; r0 += kMergeWarps * kMergeInFlight) {
        float2 ml[kMergeInFlight];
        float4 v[kMergeInFlight];
#pragma unroll
        for (int u = 0; u < kMergeInFlight; ++u) {
            const int r = r0 + kMergeWarps * u;
            ml[u] = make_float2(-INFINITY, 0.f);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < R) {
                ml[u] = *reinterpret_cast<const float2 *>(base + r * rw + D);
                v[u] = *reinterpret_cast<const float4 *>(base + r * rw + b * kBlock + 4 * lane);
            }
        }
        float mc = M;
#pragma unroll
        for (int u = 0; u < kMergeInFlight; ++u) mc = fmaxf(mc, ml[u].x);
        const float sc = M == -INFINITY ? 0.f : __expf(M - mc);
        M = mc;
        ls *= sc;
        acc.x *= sc;
        acc.y *= sc;
        acc.z *= sc;
        acc.w *= sc;
#pragma unroll
        for (int u = 0; u < kMergeInFlight; ++u) {
            const float w = ml[u].x == -INFINITY ? 0.f : __expf(ml[u].x - M);
            ls = fmaf(w, ml[u].y, ls);
            acc.x = fmaf(w, v[u].x, acc.x);
            acc.y = fmaf(w, v[u].y, acc.y);
            acc.z = fmaf(w, v[u].z, acc.z);
            acc.w = fmaf(w, v[u].w, acc.w);
        }
    }
    red_o[warp][lane] = acc;
    if (lane == 0) {
        red_m[warp] = M;
        red_l[warp] = ls;
    }
    __syncthreads();
    if (warp != 0) return;
    float mx = red_m[0], lsum = 0.f;
#pragma unroll
    for (int w = 1; w < kMergeWarps; ++w) mx = fmaxf(mx, red_m[w]);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
        const float wt = red_m[w] == -INFINITY ? 0.f : __expf(red_m[w] - mx);
        const float4 a = red_o[w][lane];
        o[0] = fmaf(wt, a.x, o[0]);
        o[1] = fmaf(wt, a.y, o[1]);
        o[2] = fmaf(wt, a.z, o[2]);
        o[3] = fmaf(wt, a.w, o[3]);
        lsum = fmaf(wt, red_l[w], lsum);
    }
    const float inv = lsum != 0.f ? kInvSqrt128 / lsum : 0.f;
    warp_fwht4(o, lane);
    apply_signs4(o, p.vc, 4 * lane);
    store_out4(p.out, at, o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
}

// ------------------------------------------------------------------ host side
template <int NB, int SETS, bool APPEND, bool DIRECT>
tq_status launch_t4_t(const T4Params &p, unsigned n_ctas, cudaStream_t stream) {
    constexpr size_t smem = T4Smem<NB, SETS, DIRECT>::total + 1024;
    const auto kernel = attn_t4_kernel<NB, SETS, APPEND, DIRECT>;
    const tq_status st = kernel_setup(reinterpret_cast<const void *>(kernel), (int)smem, kT4Threads, nullptr);
    if (st != TQ_OK) return st;
    PdlConfig lc(dim3(n_ctas), dim3(kT4Threads), smem, stream);
    if (p.bar) {
        lc.attrs[1].id = cudaLaunchAttributeCooperative;
        lc.attrs[1].val.cooperative = 1;
        lc.cfg.numAttrs = 2;
    }
    return check_cuda(cudaLaunchKernelEx(&lc.cfg, kernel, p));
}

template <int NB, int SETS>
tq_status launch_t4_nb(const T4Params &p, unsigned n_ctas, cudaStream_t stream) {
    if (p.bpr == kSlice)   // rows of eight blocks: 528 bytes, TMA copies
        return p.k_new ? launch_t4_t<NB, SETS, true, false>(p, n_ctas, stream) : launch_t4_t<NB, SETS, false, false>(p, n_ctas, stream);
    return p.k_new ? launch_t4_t<NB, SETS, true, true>(p, n_ctas, stream) : launch_t4_t<NB, SETS, false, true>(p, n_ctas, stream);
}

// Batch: one partial row per segment.  A segment ends where a chunk or a sequence ends, so the
// segment of chunk c and sequence s is number c + s: at most n_seqs + n_chunks rows.
size_t t4_rows_bytes(int n_seqs, int n_q_heads, int head_dim, int sm_count) {
    return sizeof(float) * (size_t)(n_seqs + sm_count) * n_q_heads * part_stride(head_dim);
}

}  // namespace

bool attn_t4_supported(const tq_cache &k, const tq_cache &v, int n_q_heads) {
    const int nb = k.head_dim / kBlock;
    return k.type == TQ_TURBO4 && v.type == TQ_TURBO4 && nb >= 1 && nb <= 2 && n_q_heads / k.n_kv_heads <= 8;
}

bool attn_t4_merges_itself(const tq_cache &k, int n_seqs, int n_splits) {
    return k.n_kv_heads * (k.head_dim / kBlock) <= kSlice && grid_merge_fits(n_seqs, n_splits);
}

size_t attn_t4_workspace_bytes(int n_seqs, int n_q_heads, int head_dim, int sm_count) {
    return kGridBarrierBytes + t4_rows_bytes(n_seqs, n_q_heads, head_dim, sm_count) + sizeof(int2) * (size_t)n_seqs;
}

tq_status launch_attn_t4(const tq_cache &k, const tq_cache &v, const void *q, int n_seqs, int n_q_heads,
                         const int32_t *seq_lens, int64_t max_seq_len, float scale, OutPtr out, void *ws,
                         int n_splits, const void *k_new, const void *v_new, cudaStream_t stream) {
    const int nb = k.head_dim / kBlock, sms = device_sm_count();
    T4Params p;
    p.kc = make_view(k);
    p.vc = make_view(v);
    p.q = static_cast<const __half *>(q);
    p.k_new = static_cast<const __half *>(k_new);
    p.v_new = static_cast<const __half *>(v_new);
    p.seq_lens = seq_lens;
    p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kGridBarrierBytes);
    p.seg = reinterpret_cast<int2 *>(reinterpret_cast<uint8_t *>(p.part) +
                                     t4_rows_bytes(n_seqs, n_q_heads, k.head_dim, sms));
    p.score_scale = scale * kLog2e * kInvSqrt128 * kE4m3Step4;
    p.max_len = (int32_t)max_seq_len;
    p.n_seqs = n_seqs;
    p.n_q_heads = n_q_heads;
    p.group = n_q_heads / k.n_kv_heads;
    p.bpr = k.n_kv_heads * nb;
    p.wait_limit = kWaitLimit;
    p.grid_wait_limit = kGridWaitLimit;
    p.withhold_tiles = 0;
    if (take_injected_timeout()) {
        p.wait_limit = kInjectedWaitLimit;
        p.withhold_tiles = 1;
    }
    p.out = out;
    const bool grid = attn_t4_merges_itself(k, n_seqs, n_splits);
    p.bar = grid ? static_cast<uint64_t *>(ws) : nullptr;
    const int slices = (p.bpr + kSlice - 1) / kSlice;
    p.n_chunks = grid ? n_splits : std::max(1, sms / slices);
    const unsigned n_ctas = (unsigned)(p.n_chunks * slices);
    const bool two = p.group > 4;
    tq_status st = nb == 1 ? (two ? launch_t4_nb<1, 2>(p, n_ctas, stream) : launch_t4_nb<1, 1>(p, n_ctas, stream))
                           : (two ? launch_t4_nb<2, 2>(p, n_ctas, stream) : launch_t4_nb<2, 1>(p, n_ctas, stream));
    if (st != TQ_OK || grid) return st;
    PdlConfig lc(dim3((unsigned)n_q_heads, (unsigned)n_seqs, (unsigned)nb), dim3(32 * kMergeWarps), 0, stream);
    return check_cuda(cudaLaunchKernelEx(&lc.cfg, attn_t4_merge_kernel, p, (int)k.head_dim));
}

}  // namespace tq
