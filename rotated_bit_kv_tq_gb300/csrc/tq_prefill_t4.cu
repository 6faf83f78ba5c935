// tq_prefill_t4.cu -- causal prompt-chunk attention over a turbo4 K cache and a turbo4 V cache,
// head_dim 128, on the 5th-generation tensor cores.
//
// Query token j of the chunk sits at position pos0 + j and attends to rows 0 .. pos0 + j.  With
// Q~ = H D q, key codes c_t and norms k_t, v_t (every constant factor folded into one scale):
//     s_t = k_t (Q~ . c_t),   p_t = 2^(s_t - m),   o = D' H (sum_t p_t v_t c'_t) / (sum_t p_t).
// A CTA owns 128 (token, head) rows of one KV head and walks over tiles of 128 keys.
//
//  - Warps 0-3 take the even tiles, warps 4-7 the odd ones, and each of the two groups has its own
//    running maximum, sum and output accumulator.  Nothing passes between them until the end, so
//    one group's softmax runs while the other waits for its products.  (Measured before the later steps, at 518 us: all eight
//    warps on one tile, exchanging row maxima for every tile, 531 us; two groups of eight warps
//    590 us.)
//  - Warps 8-11 (K) and 12-15 (V), one thread per key: stage the tile's codes (cp.async, four
//    lanes per key so that a request covers whole 32-byte sectors) and expand them once to fp16.
//  - Warp 16 issues the MMAs: S = Q~ C^T with Q~ as an fp16 pair hi + lo, and O += P V.
//
// The precision of P V.  v_t c' has more bits than fp16 holds, and so has p_t; rounding both
// costs two errors of up to 2^-11.  The V tile holds u_t c' instead, u_t the power of two at or
// below v_t (at most 2^12): exact in fp16 and no more than 49,152.  P takes the rest,
// p_t (v_t / u_t), rounded once: p_t <= 2^8 (below) and v_t / u_t < 32.  The row sum takes p_t in
// fp32.  Against 64 bits the fp16 outputs of 1,024 queries over 15,360 rows are
// 2.4e-4 of their size off, where rounding alone takes 2.1e-4; with both factors rounded they
// were 3.2e-4 off.
//
// Tensor memory: S0 [0,128), S1 [128,256), O0 [256,384), O1 [384,512).  A tile's weights overwrite
// the second half of its scores as those are read.
//
// The rotation Q~ = H D q is a product as well: the signs of D go into a +-1 matrix, and the
// sums of fp16 queries are exact up to the fp32 accumulator's rounding.
//
// What bounds it: 1,024 queries of 32 heads over 15,360 rows of 8 KV heads take 467 us (39 % of the
// tensor cores' cycles, 49 % of the issue slots), in two waves of which the second fills 104 of
// 152 SMs.  A tile takes 3,400 clocks, of which the MMAs need 1,536 (the score MMAs twice, for
// the query's low parts) and what they read from shared memory 1,280; the tiles written, the
// staged codes and the norms take another 1,000 of shared memory's time.  A group's chain for one
// tile is 1,400 clocks of score MMAs, 3,500 of softmax and 1,700 until its next scores can start.
#include <cmath>

#include "tq_prefill_tc.cuh"

namespace tq {
namespace {

constexpr int kP4Tmem = 512;
constexpr uint32_t kP4O = 256;
constexpr uint32_t kP4P = 64;          // the weights' first column within their tile's scores
constexpr int kP4MaxSplit = 4;         // CTAs that share a query block, as a cluster
constexpr float kP4Lag = 8.f;           // log2 units by which a score may pass the row's reference

// Buffer b of a double-buffered resource serves tiles b, b + 2, ...: tile i waits for phase i >> 1.
enum {
    kP4BarRaw = 0,      // queries and rotation matrix in shared memory (256 arrivals)
    kP4BarRot = 1,      // rotated (commit)
    kP4BarQ = 2,        // rotated queries written back as operands (256 arrivals)
    kP4BarKFull = 3,    // [2] K tile, its norms and the V ratios (one arrival per warp)
    kP4BarVFull = 5,    // [2] V tile (one arrival per warp)
    kP4BarSFull = 7,    // [2] scores ready, K tile free (commit)
    kP4BarPFull = 9,    // [2] weights written, O rescaled (one arrival per warp)
    kP4BarPvDone = 11,  // [2] the tile's P V done: its V tile, scores and weights free (commit)
    kP4BarDrain = 13,   // every MMA of the CTA done (commit)
    kP4BarCount = 14
};

struct P4Smem {
    // [0] Q~ high parts, [1] low parts, [row][coord] K-major; before that [0] the rotation
    // matrix and [1] the queries as they came; after the last MMA the epilogue's exchange area
    alignas(1024) uint8_t q[2][32768];
    alignas(1024) uint8_t k[2][32768];     // K tiles [key][coord], K-major; at the end the output rows
    alignas(1024) uint8_t v[2][32768];     // V tiles [key][coord], coords contiguous (MN-major)
    alignas(16) uint8_t raw[2][kTcKeys * 64];   // staged codes of one tile (K, V)
    // K norms and v_t / u_t of four tiles: a buffer is written for tile i + 4 after the scores of
    // tile i + 2, which are issued after the P V of tile i
    float kn[4][kTcKeys], vr[4][kTcKeys];
    float ml[2][2][kTcRows];               // [group][maximum, sum][row]
    float row_ml[kTcRows][2];              // the row's, over both groups
    alignas(8) uint64_t bar[kP4BarCount];
    uint32_t tmem;
};

// Staged codes: chunk c (16 bytes) of key k, rotated so that 8 consecutive keys' accesses to one
// chunk cover the banks once.
__device__ __forceinline__ uint32_t code_chunk(int key, int c) {
    return (uint32_t)(key * 64 + ((c ^ ((key >> 1) & 3)) << 4));
}

// The rows of one cache at positions pos, pos + 128, ...  The page of a position is loaded one
// tile ahead of its use.
struct RowWalk {
    int64_t pos, n_keys;
    int32_t pi, off, dq, dr, page;
    bool seq_ok;
    __device__ __forceinline__ RowWalk(const CacheView &c, int32_t seq, int64_t first, int64_t n)
        : pos(first), n_keys(n), pi(0), off(0), dq(0), dr(0), page(-1) {
        seq_ok = seq >= 0 && seq < c.n_seqs;
        if (c.page_tokens) {
            pi = first >> 31 ? (int32_t)(first / c.page_tokens) : (int32_t)((uint32_t)first / (uint32_t)c.page_tokens);
            off = (int32_t)(first - (int64_t)pi * c.page_tokens);
            dq = kTcKeys / c.page_tokens;
            dr = kTcKeys % c.page_tokens;
        }
        load_page(c, seq);
    }
    __device__ __forceinline__ void load_page(const CacheView &c, int32_t seq) {
        if (c.page_tokens)
            page = seq_ok && pos < n_keys && pi < c.max_pages ? c.page_table[(int64_t)seq * c.max_pages + pi] : -1;
    }
    __device__ __forceinline__ const uint8_t *row(const CacheView &c, int32_t seq) const {
        if (pos >= n_keys) return nullptr;
        int64_t r;
        bool ok = seq_ok;
        if (c.page_tokens) {
            ok = ok && page >= 0 && page < c.n_pages;
            r = (int64_t)page * c.page_tokens + off;
        } else {
            ok = ok && pos < c.capacity;
            r = (int64_t)seq * c.capacity + pos;
        }
        if (!ok) {
            record_error(TQ_ERR_OUT_OF_RANGE);
            return nullptr;
        }
        return c.base + r * c.row_bytes;
    }
    __device__ __forceinline__ void next(const CacheView &c, int32_t seq) {
        pos += kTcKeys;
        pi += dq;
        off += dr;
        if (c.page_tokens && off >= c.page_tokens) {
            off -= c.page_tokens;
            ++pi;
        }
        load_page(c, seq);
    }
};

// One producer group, one thread per key: stage and expand every tile of its cache.  A warp
// stages the rows of its own 32 keys, so it needs no barrier beyond its own.
template <bool IS_V>
__device__ __forceinline__ void p4_produce(const TcParams &p, P4Smem &sm, int g, int64_t n_keys, int tile0,
                                           int n_tiles, int pt, volatile int *abort_v) {
    const CacheView &cv = IS_V ? p.vc : p.kc;
    const bool chunked = IS_V ? p.chunked_v : p.chunked_k;
    const int lane = pt & 31, w0 = pt & ~31;
    uint8_t *raw = sm.raw[IS_V ? 1 : 0];
    const int wait_bar = IS_V ? kP4BarPvDone : kP4BarSFull, full_bar = IS_V ? kP4BarVFull : kP4BarKFull;
    const int64_t first = (int64_t)tile0 * kTcKeys + pt;
    RowWalk walk(cv, p.seq, first, n_keys), vwalk(p.vc, p.seq, first, IS_V ? 0 : n_keys);
    uint32_t nrm = 0, vnrm = 0;   // norm bits of the staged tile: this cache's, V's (K only)
    auto stage = [&]() {
        const uint8_t *row = walk.row(cv, p.seq);
        if (chunked) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = w0 + 8 * j + (lane >> 2), c = lane & 3;
                const uint8_t *src = reinterpret_cast<const uint8_t *>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), 8 * j + (lane >> 2)));
                if (src) cp_async16(smem_u32(raw + code_chunk(key, c)), src + kCodeBytes4 * g + 16 * c);
            }
        } else if (row) {   // rows that are not multiples of 16 bytes
            const uint16_t *src = reinterpret_cast<const uint16_t *>(row + kCodeBytes4 * g);
            for (int h = 0; h < kCodeBytes4 / 2; ++h)
                *reinterpret_cast<uint16_t *>(raw + code_chunk(pt, h >> 3) + 2 * (h & 7)) = src[h];
        }
        nrm = row ? *reinterpret_cast<const uint16_t *>(row + norm_offset(TQ_TURBO4, g, cv.row_bytes / block_bytes(TQ_TURBO4))) : 0;
        walk.next(cv, p.seq);
        if (!IS_V) {
            const uint8_t *vrow = vwalk.row(p.vc, p.seq);
            vnrm = vrow ? *reinterpret_cast<const uint16_t *>(vrow + norm_offset(TQ_TURBO4, g, p.vc.row_bytes / block_bytes(TQ_TURBO4))) : 0;
            vwalk.next(p.vc, p.seq);
        }
        cp_async_commit();
    };
    if (n_tiles > 0) stage();
    for (int i = 0; i < n_tiles; ++i) {
        const int b = i & 1;
        cp_async_wait<0>();
        __syncwarp();
        if (i >= 2 && !*abort_v && !tc_wait(smem_u32(&sm.bar[wait_bar + b]), (uint32_t)(((i - 2) >> 1) & 1)))
            *abort_v = 1;
        uint8_t *tile = IS_V ? sm.v[b] : sm.k[b];
        __half2 u2 = __half2half2(__ushort_as_half(0));
        if (IS_V) {
            u2 = __half2half2(v_scale(nrm));
        } else {
            sm.kn[i & 3][pt] = __half2float(__ushort_as_half((uint16_t)nrm));
            const float u = __half2float(v_scale(vnrm));
            sm.vr[i & 3][pt] = u != 0.f ? __half2float(__ushort_as_half((uint16_t)vnrm)) / u : 0.f;
        }
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {   // a quarter at a time: unrolled in full, 476 us instead of 467: instruction caches
            const uint4 x = *reinterpret_cast<const uint4 *>(raw + code_chunk(pt, c));
            const uint32_t n[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t lo, hi, o[4];
                e4m3x8(n[w], lo, hi);
                o[0] = e4m3_to_half2(lo);
                o[1] = e4m3_to_half2_hi(lo);
                o[2] = e4m3_to_half2(hi);
                o[3] = e4m3_to_half2_hi(hi);
                if (IS_V)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&o[e]), u2);
                        o[e] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                const int at = 32 * c + 8 * w;
                *reinterpret_cast<uint4 *>(tile + (IS_V ? canon_mn(pt, at) : canon(pt, at))) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) tc_arrive(smem_u32(&sm.bar[full_bar + b]));
        if (i + 1 < n_tiles) stage();   // the warp has read its codes
    }
    cp_async_wait<0>();
}

// A chunk is 16 columns (keys) of the warp's 32 rows in the fragment form of the 16-row loads:
// element 8 h + 4 k + 2 s + e of a lane is row 16 h + 8 s + lane / 4, column 8 k + 2 (lane % 4) + e.
// A lane holds 4 columns of 4 rows, so it reads 4 norms from shared memory for 16 scores; with a
// whole row per lane it read one per score, 1,500 of a tile's 3,600 clocks of what shared memory
// returns (651 us, 578 us in this form).
constexpr int kP4Chunks = 8;
#define P4_16(c, u) c(u[0]), c(u[1]), c(u[2]), c(u[3]), c(u[4]), c(u[5]), c(u[6]), c(u[7]), \
                    c(u[8]), c(u[9]), c(u[10]), c(u[11]), c(u[12]), c(u[13]), c(u[14]), c(u[15])
#define P4_OUT(x) "=r"(x)
#define P4_IO(x) "+r"(x)
#define P4_IN(x) "r"(x)
__device__ __forceinline__ void p4_load(uint32_t taddr, uint32_t (&u)[16]) {   // to be followed by p4_loaded
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
                 "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];"
                 : P4_16(P4_OUT, u) : "r"(taddr), "r"(taddr + (16u << 16)));
}
__device__ __forceinline__ void p4_loaded(uint32_t (&u)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : P4_16(P4_IO, u));
}
__device__ __forceinline__ void p4_store(uint32_t taddr, const uint32_t (&u)[16]) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%2,%3,%4,%5,%6,%7,%8,%9};\n\t"
                 "tcgen05.st.sync.aligned.16x256b.x2.b32 [%1], {%10,%11,%12,%13,%14,%15,%16,%17};"
                 ::"r"(taddr), "r"(taddr + (16u << 16)), P4_16(P4_IN, u));
}
// 16 keys' weights as fp16 pairs, 8 columns: element 4 h + 2 k + s is row 16 h + 8 s + lane / 4,
// column 4 k + lane % 4
__device__ __forceinline__ void p4_store_pairs(uint32_t taddr, const uint32_t (&w)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%2,%3,%4,%5};\n\t"
                 "tcgen05.st.sync.aligned.16x128b.x2.b32 [%1], {%6,%7,%8,%9};"
                 ::"r"(taddr), "r"(taddr + (16u << 16)), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                   "r"(w[6]), "r"(w[7]));
}
#undef P4_16
#undef P4_OUT
#undef P4_IO
#undef P4_IN
__device__ __forceinline__ float2 f2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }
// First element of row r (16 (r >> 1) + 8 (r & 1) + lane / 4) in column group k of a chunk.
__device__ __forceinline__ constexpr int p4_at(int r, int k) { return 8 * (r >> 1) + 4 * k + 2 * (r & 1); }

template <bool MASK>
__device__ __forceinline__ float2 p4_mask(float2 x, int col, int lim, float v) {
    return MASK ? make_float2(col > lim ? v : x.x, col + 1 > lim ? v : x.y) : x;
}
// Raises mx[row] to the maxima of a chunk's scores, columns col ..; kn: their norms from this
// lane's first column on; columns past lim[row], counted from there, are masked.
template <bool MASK>
__device__ __forceinline__ void p4_max(const uint32_t (&u)[16], const float *kn, const int (&lim)[4], int col, float (&mx)[4]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float2 n = *reinterpret_cast<const float2 *>(kn + 8 * k);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float2 x = p4_mask<MASK>(mul2(f2(u[p4_at(r, k)], u[p4_at(r, k) + 1]), n), col + 8 * k, lim[r], -INFINITY);
            mx[r] = fmaxf(fmaxf(mx[r], x.x), x.y);
        }
    }
}
// The weights of a chunk: p into the rows' sums, p v / u into tensor memory.
template <bool MASK>
__device__ __forceinline__ void p4_weights(uint32_t taddr, const uint32_t (&u)[16], const float *kn, const float *vr,
                                           const int (&lim)[4], int col, const float (&neg_m)[4], float2 (&sum)[4]) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float2 n = *reinterpret_cast<const float2 *>(kn + 8 * k), v = *reinterpret_cast<const float2 *>(vr + 8 * k);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float2 x = p4_mask<MASK>(fma2(f2(u[p4_at(r, k)], u[p4_at(r, k) + 1]), n, make_float2(neg_m[r], neg_m[r])),
                                           col + 8 * k, lim[r], -INFINITY);
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            sum[r] = add2(sum[r], e);
            const float2 y = p4_mask<MASK>(mul2(e, v), col + 8 * k, lim[r], 0.f);   // a masked key's v / u may be anything
            w[4 * (r >> 1) + 2 * k + (r & 1)] = pack_half2(y.x, y.y);
        }
    }
    p4_store_pairs(taddr, w);
}

// One tile: scores (columns at s_addr), running maxima, weights; the rescaling of O (columns at
// o_addr, which hold every earlier product of this group: the scores were issued after them).
// The chunks go up for the maximum and down for the weights, whose columns 64 + 8 c .. then lie
// over scores that have been read.
template <bool MASK>
__device__ __forceinline__ void p4_tile(uint32_t s_addr, uint32_t o_addr, const float *kn, const float *vr,
                                        const int (&lim)[4], bool first, float (&m_run)[4], float2 (&l_run)[4]) {
    uint32_t ua[16], ub[16];
    float mx[4] = {m_run[0], m_run[1], m_run[2], m_run[3]};
    p4_load(s_addr, ua);
    p4_loaded(ua);
#pragma unroll 1
    for (int c = 0; c < kP4Chunks; c += 2) {
        p4_load(s_addr + 16u * (c + 1), ub);
        p4_max<MASK>(ua, kn + 16 * c, lim, 16 * c, mx);
        p4_loaded(ub);
        p4_load(s_addr + 16u * ((c + 2) & (kP4Chunks - 1)), ua);   // after the last one, unused
        p4_max<MASK>(ub, kn + 16 * c + 16, lim, 16 * c + 16, mx);
        p4_loaded(ua);
    }
    float alpha[4];
    bool moved = false;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        // the reference moves only when a score passes it by more than 2^kP4Lag, so p <= 2^8
        alpha[r] = 1.f;
        if (m_run[r] == -INFINITY || mx[r] > m_run[r] + kP4Lag) {
            alpha[r] = m_run[r] == -INFINITY ? 0.f : ex2(m_run[r] - mx[r]);
            m_run[r] = mx[r];
        }
        moved |= alpha[r] != 1.f;
        l_run[r] = make_float2(l_run[r].x * alpha[r], l_run[r].y * alpha[r]);   // this lane's share
        mx[r] = m_run[r] == -INFINITY ? 0.f : -m_run[r];   // all masked: every p is 0
    }
    if (!first && __any_sync(0xffffffffu, moved)) {
#pragma unroll 1
        for (int c = 0; c < kP4Chunks; ++c) {
            p4_load(o_addr + 16u * c, ua);
            p4_loaded(ua);
#pragma unroll
            for (int e = 0; e < 16; ++e)
                ua[e] = __float_as_uint(__uint_as_float(ua[e]) * alpha[2 * (e >> 3) + ((e >> 1) & 1)]);
            p4_store(o_addr + 16u * c, ua);
        }
    }
#pragma unroll 1
    for (int c = kP4Chunks - 2; c >= 0; c -= 2) {   // ub holds chunk c + 1
        p4_load(s_addr + 16u * c, ua);
        p4_weights<MASK>(s_addr + kP4P + 8u * (c + 1), ub, kn + 16 * c + 16, vr + 16 * c + 16, lim, 16 * c + 16, mx, l_run);
        p4_loaded(ua);
        p4_load(s_addr + 16u * max(c - 1, 0), ub);   // after the last one, unused
        p4_weights<MASK>(s_addr + kP4P + 8u * c, ua, kn + 16 * c, vr + 16 * c, lim, 16 * c, mx, l_run);
        p4_loaded(ub);
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kTcThreads, 1) prefill_t4_kernel(const TcParams p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    P4Smem &sm = *reinterpret_cast<P4Smem *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the query blocks with the most keys first; the CTAs of a cluster cut a block's key tiles
    const unsigned qcta = blockIdx.x / (unsigned)p.split;
    const int rank = (int)(blockIdx.x % (unsigned)p.split);
    const int g = (int)(qcta % (unsigned)p.n_kv_heads), G = p.group, Hq = p.n_q_heads;
    const int64_t j0 = (p.n_qblocks - 1 - (int64_t)(qcta / (unsigned)p.n_kv_heads)) * p.bq;
    const int64_t n_keys = p.pos0 + min64(p.n_q, j0 + p.bq);   // rows the CTA's last query sees
    const int64_t first_pos = p.pos0 + j0;                     // the CTA's first query position
    const int64_t n_all = (n_keys + kTcKeys - 1) / kTcKeys;
    const int tile0 = (int)(n_all * rank / p.split);
    const int n_tiles = (int)(n_all * (rank + 1) / p.split) - tile0;
    auto bar = [&](int i) { return smem_u32(&sm.bar[i]); };

    if (tid == 0) {
        abort_flag = 0;
        tc_bar_init(bar(kP4BarRaw), kTcSoftmax);
        tc_bar_init(bar(kP4BarRot), 1);
        tc_bar_init(bar(kP4BarQ), kTcSoftmax);
        for (int b = 0; b < 2; ++b) {
            tc_bar_init(bar(kP4BarKFull + b), kTcGroup / 32);
            tc_bar_init(bar(kP4BarVFull + b), kTcGroup / 32);
            tc_bar_init(bar(kP4BarSFull + b), 1);
            tc_bar_init(bar(kP4BarPFull + b), kTcGroup / 32);
            tc_bar_init(bar(kP4BarPvDone + b), 1);
        }
        tc_bar_init(bar(kP4BarDrain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kTcMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&sm.tmem)), "r"(kP4Tmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    volatile int *abort_v = &abort_flag;
    pdl_wait();
    pdl_launch_dependents();

    if (warp < kTcSoftmax / 32) {
        const int quad = warp & 3, grp = warp >> 2;
        const int r = 32 * quad + lane;   // this thread's row outside the tile loop
        const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
        // ---- the queries: 8 rows x 4 chunks of 8 coordinates per warp and step
        uint4 x[8];
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const int u = warp + 8 * it, row = 8 * (u >> 2) + (lane & 7), c = 4 * (u & 3) + (lane >> 3);
            const int rj = row / G, rh = row - rj * G;
            x[it] = make_uint4(0u, 0u, 0u, 0u);
            if (rj < p.bq && j0 + rj < p.n_q)
                x[it] = *reinterpret_cast<const uint4 *>(p.q + ((j0 + rj) * Hq + g * G + rh) * (int64_t)kBlock + 8 * c);
        }
        // ---- the rotation matrix: row n, coordinates 8c .. 8c + 7 as the sign bits of 8 ones,
        // parity(n & k) of the coordinate k and the rotation sign
#pragma unroll 2
        for (int it = 0; it < 8; ++it) {
            const int u = warp + 8 * it, n = 8 * (u >> 2) + (lane & 7), c = 4 * (u & 3) + (lane >> 3);
            const uint32_t sw = c < 4 ? p.kc.signs[0] : c < 8 ? p.kc.signs[1] : c < 12 ? p.kc.signs[2] : p.kc.signs[3];
            uint32_t bits = (uint32_t)(0x963C5AF066CCAA00ull >> (8 * (n & 7))) ^ (sw >> (8 * (c & 3)));
            if (__popc((unsigned)((n >> 3) & c)) & 1) bits = ~bits;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = 0x3c003c00u | ((bits >> (2 * e)) & 1u) << 15 | ((bits >> (2 * e + 1)) & 1u) << 31;
            *reinterpret_cast<uint4 *>(sm.q[0] + canon(n, 8 * c)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const int u = warp + 8 * it, row = 8 * (u >> 2) + (lane & 7), c = 4 * (u & 3) + (lane >> 3);
            *reinterpret_cast<uint4 *>(sm.q[1] + canon(row, 8 * c)) = x[it];
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_arrive(bar(kP4BarRaw));
        if (!*abort_v && !tc_wait(bar(kP4BarRot), 0)) *abort_v = 1;
        tc_fence_after();
        // Q~ = hi + lo, both fp16 (two MMAs per k-step): the query keeps about 22 bits
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
            const int c0 = 64 * grp + 32 * c;
            float x[32];
            tc_ld32(tmem + lane_base + kP4O + (uint32_t)c0, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t w[4], wl[4];
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    split_half2(x[8 * e + 2 * f] * p.score_scale, x[8 * e + 2 * f + 1] * p.score_scale, w[f], wl[f]);
                *reinterpret_cast<uint4 *>(sm.q[0] + canon(r, c0 + 8 * e)) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(sm.q[1] + canon(r, c0 + 8 * e)) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        tc_arrive(bar(kP4BarQ));

        // ---- every second tile.  After a timeout the remaining waits are skipped; the tensor
        // memory accesses stay in step.
        const int col = 2 * (lane & 3);   // the lane's first column and its rows, 8 apart
        int64_t qpos[4];                  // rows without a query see every key of the CTA
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int jl = (32 * quad + 8 * k + (lane >> 2)) / G;
            qpos[k] = jl < p.bq && j0 + jl < p.n_q ? p.pos0 + j0 + jl : INT64_MAX;
        }
        float m_run[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        float2 l_run[4] = {};
        const uint32_t s_addr = tmem + lane_base + 128u * grp, o_addr = tmem + lane_base + kP4O + 128u * grp;
#pragma unroll 1
        for (int i = grp; i < n_tiles; i += 2) {
            if (!*abort_v && !tc_wait(bar(kP4BarSFull + grp), (uint32_t)((i >> 1) & 1))) *abort_v = 1;
            __syncwarp();
            tc_fence_after();
            const int64_t t0 = (int64_t)(tile0 + i) * kTcKeys;
            const float *kn = sm.kn[i & 3] + col, *vr = sm.vr[i & 3] + col;
            int lim[4] = {0, 0, 0, 0};
            if (t0 + (kTcKeys - 1) <= first_pos) {   // every key is visible to every row
                p4_tile<false>(s_addr, o_addr, kn, vr, lim, i < 2, m_run, l_run);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)   // columns past lim, counted from col, are masked
                    lim[k] = (int)max64(-1, min64(qpos[k] - t0, kTcKeys)) - col;
                p4_tile<true>(s_addr, o_addr, kn, vr, lim, i < 2, m_run, l_run);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) tc_arrive(bar(kP4BarPFull + grp));
        }

        // ---- the two groups' sums join; thread (row, grp) takes coordinates 64 grp ..
        const bool done = __all_sync(0xffffffffu, tc_wait(bar(kP4BarDrain), 0) && !*abort_v);
        __syncwarp();
        tc_fence_after();
        const int pair_bar = 3 + quad;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float l = l_run[k].x + l_run[k].y;
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if ((lane & 3) == 0) {
                sm.ml[grp][0][32 * quad + 8 * k + (lane >> 2)] = m_run[k];
                sm.ml[grp][1][32 * quad + 8 * k + (lane >> 2)] = l;
            }
        }
        named_sync(pair_bar, 64);
        const float m0 = sm.ml[0][0][r], m1 = sm.ml[1][0][r], M = fmaxf(m0, m1);
        const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - M), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
        float o[64];
        if (n_tiles > 0) {
            tc_ld64(tmem + lane_base + kP4O + 64u * grp, o);
#pragma unroll
            for (int e = 0; e < 64; ++e) o[e] *= f0;
        } else {
#pragma unroll
            for (int e = 0; e < 64; ++e) o[e] = 0.f;
        }
        if (n_tiles > 1)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float t[16];
                tc_ld16(tmem + lane_base + kP4O + 128u + 64u * grp + 16u * c, t);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[16 * c + e] += f1 * t[e];
            }
        auto at = [&](int row, int c4) { return reinterpret_cast<float *>(sm.k[0]) + row * 128 + (((c4 ^ row) & 31) << 2); };
#pragma unroll
        for (int c = 0; c < 16; ++c)
            *reinterpret_cast<float4 *>(at(r, 16 * grp + c)) = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        if (grp == 0) {
            sm.row_ml[r][0] = M;
            sm.row_ml[r][1] = f0 * sm.ml[0][1][r] + f1 * sm.ml[1][1][r];
        }
        // ---- the CTAs of a cluster each finish a share of the rows from all of them, a warp a row:
        // sum, inverse rotation, V signs, store
        if (p.split > 1) cluster_sync_all();
        else named_sync(1, kTcSoftmax);
        const int rows = kTcRows / p.split;
        if (done)
#pragma unroll 2
            for (int row = rank * rows + warp; row < (rank + 1) * rows; row += kTcSoftmax / 32) {
                const int rj = row / G, rh = row - rj * G;
                if (rj >= p.bq || j0 + rj >= p.n_q) continue;
                // lane s < split reads CTA s's maximum and sum, then every lane its coordinates
                float m = -INFINITY, l = 0.f;
                if (lane < p.split) {
                    m = ld_cluster_f32(smem_u32(&sm.row_ml[row][0]), (uint32_t)lane);
                    l = ld_cluster_f32(smem_u32(&sm.row_ml[row][1]), (uint32_t)lane);
                }
                float4 u[kP4MaxSplit];
#pragma unroll
                for (int s = 0; s < kP4MaxSplit; ++s)
                    u[s] = s < p.split ? ld_cluster_f32x4(smem_u32(at(row, lane)), (uint32_t)s) : make_float4(0.f, 0.f, 0.f, 0.f);
                float Mx = m;
#pragma unroll
                for (int o = 1; o < kP4MaxSplit; o *= 2) Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, o));
                Mx = __shfl_sync(0xffffffffu, Mx, 0);
                const float f = m == -INFINITY ? 0.f : ex2(m - Mx);
                float L = f * l;
#pragma unroll
                for (int o = 1; o < kP4MaxSplit; o *= 2) L += __shfl_xor_sync(0xffffffffu, L, o);
                L = __shfl_sync(0xffffffffu, L, 0);
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int s = 0; s < kP4MaxSplit; ++s) {
                    const float fs = __shfl_sync(0xffffffffu, f, s);
                    y = make_float4(y.x + fs * u[s].x, y.y + fs * u[s].y, y.z + fs * u[s].z, y.w + fs * u[s].w);
                }
                const float inv = L > 0.f ? p.out_scale / L : 0.f;
                float v4[4] = {y.x * inv, y.y * inv, y.z * inv, y.w * inv};
                warp_fwht4(v4, lane);
                apply_signs4(v4, p.vc, 4 * lane);
                store_out4(p.out, ((j0 + rj) * Hq + g * G + rh) * (int64_t)kBlock + 4 * lane, v4[0], v4[1], v4[2], v4[3]);
            }
        if (p.split > 1) cluster_sync_all();   // the others have read this CTA's rows
    } else if (warp < kTcMmaWarp) {
        const int pt = (tid - kTcSoftmax) & (kTcGroup - 1);
        if (tid - kTcSoftmax < kTcGroup) p4_produce<false>(p, sm, g, n_keys, tile0, n_tiles, pt, abort_v);
        else p4_produce<true>(p, sm, g, n_keys, tile0, n_tiles, pt, abort_v);
    } else {
        // ================= MMA issue, the whole warp in step
        constexpr uint32_t idesc_s = idesc_f16(false), idesc_pv = idesc_f16(true);
        const uint64_t dq = sdesc(smem_u32(sm.q[0]), 128, 2048), dql = sdesc(smem_u32(sm.q[1]), 128, 2048);
        const uint64_t dk = sdesc(smem_u32(sm.k[0]), 128, 2048), dv = sdesc(smem_u32(sm.v[0]), 2048, 128);
        bool ok = __all_sync(0xffffffffu, tc_wait(bar(kP4BarRaw), 0));
        if (ok) {
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    tc_mma(tmem + kP4O, dql + (uint64_t)(16 * ks), dq + (uint64_t)(16 * ks), idesc_s, ks > 0);
                tc_commit(bar(kP4BarRot));
            }
            __syncwarp();
            ok = __all_sync(0xffffffffu, tc_wait(bar(kP4BarQ), 0));
        }
        // S(0), S(1), then P V(i) and S(i + 2) in turn, with blocking waits: a warp that polled for
        // whichever came first took issue slots from the softmax (513 us against 489 at the time)
        auto wait = [&](int first, int i) {
            if (ok && !__all_sync(0xffffffffu, tc_wait(bar(first + (i & 1)), (uint32_t)((i >> 1) & 1)) && !*abort_v)) ok = false;
        };
#pragma unroll 1
        for (int i = -2; i < n_tiles && ok; ++i) {
            if (i >= 0) {
                const int npv = i, bp = i & 1;
                wait(kP4BarPFull, i);
                wait(kP4BarVFull, i);
                tc_fence_after();
                if (ok && elect_one()) {   // 16 keys per MMA: 8 columns of weights, two 8-key groups of V
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        tc_mma_ts(tmem + kP4O + 128u * bp, tmem + 128u * bp + kP4P + 8u * kk,
                                  dv + (uint64_t)(2048 * bp + 256 * kk), idesc_pv, npv >= 2 || kk > 0);
                    tc_commit(bar(kP4BarPvDone + bp));
                }
                __syncwarp();
            }
            if (i + 2 < n_tiles) {
                const int bs = i & 1;
                wait(kP4BarKFull, i + 2);
                if (i >= 0) wait(kP4BarPvDone, i);
                tc_fence_after();
                if (ok && elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        tc_mma(tmem + 128u * bs, dq + (uint64_t)(16 * ks), dk + (uint64_t)(2048 * bs + 16 * ks), idesc_s, ks > 0);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)   // the low parts of the query
                        tc_mma(tmem + 128u * bs, dql + (uint64_t)(16 * ks), dk + (uint64_t)(2048 * bs + 16 * ks), idesc_s, 1u);
                    tc_commit(bar(kP4BarSFull + bs));
                }
                __syncwarp();
            }
        }
        if (!ok) *abort_v = 1;
        if (elect_one()) tc_commit(bar(kP4BarDrain));   // arrives once everything issued has completed
        __syncwarp();
        tc_wait(bar(kP4BarDrain), 0);
        __syncwarp();
    }
    if (p.split > 1 && warp >= kTcSoftmax / 32) {   // with the softmax warps' two
        cluster_sync_all();
        cluster_sync_all();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kTcMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kP4Tmem) : "memory");
}

}  // namespace

// params: a TcParams, complete but for split.
tq_status launch_prefill_t4(const void *params, int64_t n_ctas, cudaStream_t stream) {
    TcParams p = *static_cast<const TcParams *>(params);
    const size_t smem = sizeof(P4Smem) + 1024;   // room to align the tiles to 1024 bytes
    static_assert(sizeof(P4Smem) + 1024 <= 227 * 1024, "one CTA per SM");
    const tq_status st = kernel_setup(reinterpret_cast<const void *>(prefill_t4_kernel), (int)smem, kTcThreads, nullptr);
    if (st != TQ_OK) return st;
    // The key tiles of a query block over a cluster of 1, 2 or 4 CTAs, whichever ends first by the
    // count of waves times the tiles of a CTA and what a CTA spends around them (the queries'
    // rotation, the ends of the pipeline, the epilogue, the cluster's waits: about kAround
    // tiles).  1, 2, 4 CTAs take 38.7, 25.5, 18.1 us for 49 queries of 40 heads over 1,000 rows
    // and 467, 490, 530 us for 1,024 queries of 32 heads over 15,360; clusters of 8 took 32 and
    // 756 us, since 8 free SMs of one processing cluster are rare.
    const int64_t sms = device_sm_count();
    const int64_t tiles = (p.pos0 + p.n_q + kTcKeys - 1) / kTcKeys;
    if (tiles > INT32_MAX) return TQ_ERR_UNSUPPORTED;   // tile numbers are 32 bits wide
    constexpr int64_t kAround = 8;
    int64_t best = INT64_MAX;
    for (int s = 1; s <= kP4MaxSplit && s <= tiles; s *= 2) {
        const int64_t waves = (n_ctas * s + sms - 1) / sms, cost = waves * ((tiles + s - 1) / s + kAround);
        if (cost < best) best = cost, p.split = s;
    }
    PdlConfig lc(dim3((unsigned)(n_ctas * p.split)), dim3(kTcThreads), smem, stream);
    if (p.split > 1) {
        lc.attrs[1].id = cudaLaunchAttributeClusterDimension;
        lc.attrs[1].val.clusterDim.x = (unsigned)p.split;
        lc.attrs[1].val.clusterDim.y = 1;
        lc.attrs[1].val.clusterDim.z = 1;
        lc.cfg.numAttrs = 2;
    }
    return check_cuda(cudaLaunchKernelEx(&lc.cfg, prefill_t4_kernel, p));
}

}  // namespace tq
