// tq_decode.cu -- dequantise packed rows back to fp32 (tests, quality reports).
//
// "llama.cpp に TurboQuant を実装", "What TurboQuant does differently": the rotation is
// undone at read time and, being a Walsh-Hadamard transform, is its own inverse up to the
// 1/sqrt(128) scale.  x_hat = norm * (1/sqrt(128)) * W c(codes), in fp32.
//
// turbo4 runs on the tensor cores (decode4_kernel below); the other types:
// One warp per 128-value block, four values per lane: the codes are unpacked from the
// two bit planes, the two in-lane butterfly stages run in registers and the five
// cross-lane stages use warp shuffles; each lane writes one float4, so a warp writes its
// 512-byte output row segment fully coalesced.
#include "tq_internal.cuh"
#include "tq_codes.cuh"
#include "tq_simd.cuh"

namespace tq {
namespace {

struct DecodeParams {
    CacheView src;
    float *dst;
    int64_t pos0;
    int64_t n_blocks;   // n_tokens * bpr
    int32_t seq_id;
    int32_t bpr;
};

template <int TYPE>
__global__ void __launch_bounds__(256) decode_kernel(const DecodeParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t blk = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (blk >= p.n_blocks) return;
    const int64_t t = blk / p.bpr;
    const int fb = (int)(blk - t * p.bpr);
    const uint8_t *row = row_ptr(p.src, p.seq_id, p.pos0 + t);
    float4 *out = reinterpret_cast<float4 *>(p.dst + blk * kBlock) + lane;
    if (!row) {
        *out = make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    const uint8_t *b = row + codes_offset(TYPE, fb, p.bpr);
    const Codebook &cb = c_codebook[cb_index(TYPE)];
    // values 4*lane .. 4*lane+3
    const int i0 = 4 * lane;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = i0 + e;
        const int j = i & 15;
        const int lb = 32 * (i >> 4) + 4 * (j & 7) + 2 * (j >> 3);   // low-plane bit
        int code = (b[lb >> 3] >> (lb & 7)) & 3;
        if (TYPE == TQ_TURBO3) {
            const int jv = i & 31;
            const int hb = 32 * (i >> 5) + 4 * (jv & 7) + (jv >> 3);  // high-plane bit
            code |= ((b[32 + (hb >> 3)] >> (hb & 7)) & 1) << 2;
        }
        v[e] = cb.centroid[code];
    }
    // butterflies h = 1, 2 inside the lane
    float a0 = v[0] + v[1], a1 = v[0] - v[1], a2 = v[2] + v[3], a3 = v[2] - v[3];
    v[0] = a0 + a2;
    v[1] = a1 + a3;
    v[2] = a0 - a2;
    v[3] = a1 - a3;
    // h = 4 .. 64 across lanes (lane stride h/4)
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const bool upper = lane & m;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float o = __shfl_xor_sync(0xffffffffu, v[e], m);
            v[e] = upper ? o - v[e] : v[e] + o;
        }
    }
    const float sc = __half2float(*reinterpret_cast<const __half *>(row + norm_offset(TYPE, fb, p.bpr))) * kInvSqrt128;
    // rotation-sign variant: D W c, coordinate i negated when its sign bit is set
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = __uint_as_float(__float_as_uint(v[e] * sc) ^ sign_mask(p.src, i0 + e));
    *out = make_float4(o[0], o[1], o[2], o[3]);
}

// ------------------------------------------------------------------ turbo4
// W is a tensor product over the seven bits of the coordinate.  A warp takes 16 blocks; four of
// the bits (0, 1, 3, 4) are summed by m16n8k16 products with a 16 x 16 matrix of +-1, the other
// three (2, 5, 6) by butterflies between the eight k-steps' accumulators:
//   A[block][k]: lane (g, q) holds word q (bits 3, 4) of each 16-byte code chunk of blocks g and
//       g + 8; the chunk (bits 5, 6) and half word (bit 2) number the k-steps, the four values
//       (bits 0, 1) and q are the k of one step, as exact fp16 numbers;
//   B[k][n] = +-1 for output bits 0 (n & 1), 3, 4 (n >> 1) and 1 (which of two n-tiles).
// The sums are whole multiples of 1/16 below 2^11: exact in fp32, so the result has one rounding
// (times the norm).  Lane (g, q) ends with coordinates 32 e + 8 q + 0 .. 7 of its blocks, so the
// four lanes of a block store whole 128-byte lines (with 32 consecutive coordinates per lane each
// store touched 32 lines: 36.7 us where this took 32.2).
// The 32,768 x 8 blocks of a Llama-shape cache take 28.2 us, 5.4 TB/s of codes read and fp32
// written (floor 22.4); 127 us in the shuffle form above.  Four CTAs of four warps per SM: three
// take 29.6 us, five 29.5.
// (two 16-byte stores where the output starts on an odd 16-byte boundary)
__device__ __forceinline__ void store8(float *p, const float (&v)[8], bool wide) {
    if (!wide) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
}

constexpr int kDecodeWarps = 4;

// One lane's share of a tile: words q4 of the code chunks of blocks g8 and g8 + 8, their scales, and what
// becomes of them.
struct DecodeTile {
    uint32_t w[2][4];
    __half norm[2];
    bool present[2];
};
__device__ __forceinline__ void decode_load(const DecodeParams &p, int64_t tile, int g8, int q4, DecodeTile &d) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int64_t blk = tile * 16 + g8 + 8 * r;
        d.present[r] = false;
        d.norm[r] = __ushort_as_half(0);
#pragma unroll
        for (int e = 0; e < 4; ++e) d.w[r][e] = 0u;
        if (blk >= p.n_blocks) continue;
        const int64_t t = blk >> 32 ? blk / p.bpr : (int64_t)((uint32_t)blk / (uint32_t)p.bpr);
        const int fb = (int)(blk - t * p.bpr);
        const uint8_t *row = row_ptr(p.src, p.seq_id, p.pos0 + t);
        if (!row) continue;   // a row outside the cache reads as zeros
        d.present[r] = true;
        const uint8_t *c = row + fb * kCodeBytes4 + 4 * q4;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (p.src.row_bytes % 4 == 0)
                d.w[r][e] = *reinterpret_cast<const uint32_t *>(c + 16 * e);
            else
                d.w[r][e] = *reinterpret_cast<const uint16_t *>(c + 16 * e) | (uint32_t)*reinterpret_cast<const uint16_t *>(c + 16 * e + 2) << 16;
        d.norm[r] = *reinterpret_cast<const __half *>(row + norm_offset(TQ_TURBO4, fb, p.bpr));
    }
}

// A warp takes every n-th tile and has the next one's codes in flight while it works.
__global__ void __launch_bounds__(32 * kDecodeWarps, 4) decode4_kernel(const DecodeParams p) {
    const int lane = threadIdx.x & 31, g8 = lane >> 2, q4 = lane & 3;
    const int64_t step = (int64_t)gridDim.x * kDecodeWarps, n_tiles = (p.n_blocks + 15) / 16;
    const bool wide = reinterpret_cast<uintptr_t>(p.dst) % 32 == 0;
    pdl_wait();
    pdl_launch_dependents();
    // B fragments: column n = g8 is output (bit 0 = g8 & 1, bits 3-4 = g8 >> 1); row k is input
    // (bits 3-4 = q4, bits 0-1 = e), b0: e = 0, 1, b1: e = 2, 3; the second n-tile is output bit 1
    const uint32_t flip = (__popc(q4 & (g8 >> 1)) & 1) ? 0x80008000u : 0u;
    const uint32_t b0 = (0x3C003C00u | ((g8 & 1) ? 0x80000000u : 0u)) ^ flip, b1 = b0 ^ 0x80008000u;
    int64_t tile = (int64_t)blockIdx.x * kDecodeWarps + (threadIdx.x >> 5);
    DecodeTile next;
    decode_load(p, tile, g8, q4, next);
    for (; tile < n_tiles; tile += step) {
        const DecodeTile cur = next;
        if (tile + step < n_tiles) decode_load(p, tile + step, g8, q4, next);
        float d[8][2][4];   // [k-step: bit 2 + 2 (bits 5-6)][output bit 1][row g8: bit 0; row g8 + 8: bit 0]
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t xl, xh, yl, yh;
            e4m3x8(cur.w[0][e], xl, xh);
            e4m3x8(cur.w[1][e], yl, yh);
            const uint32_t a[2][4] = {{e4m3_to_half2(xl), e4m3_to_half2(yl), e4m3_to_half2_hi(xl), e4m3_to_half2_hi(yl)},
                                      {e4m3_to_half2(xh), e4m3_to_half2(yh), e4m3_to_half2_hi(xh), e4m3_to_half2_hi(yh)}};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mma16816_z(d[2 * e + h][0], a[h][0], a[h][1], a[h][2], a[h][3], b0, b0);
                mma16816_z(d[2 * e + h][1], a[h][0], a[h][1], a[h][2], a[h][3], b0, b1);
            }
        }
#pragma unroll
        for (int s = 1; s < 8; s <<= 1)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (!(k & s))
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float2 a = make_float2(d[k][t][e], d[k][t][e + 1]);
                            const float2 b = make_float2(d[k + s][t][e], d[k + s][t][e + 1]);
                            const float2 u = add2(a, b), v = sub2(a, b);
                            d[k][t][e] = u.x;
                            d[k][t][e + 1] = u.y;
                            d[k + s][t][e] = v.x;
                            d[k + s][t][e + 1] = v.y;
                        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (tile * 16 + g8 + 8 * r >= p.n_blocks) continue;
            const float scale = __half2float(cur.norm[r]) * (kInvSqrt128 * kE4m3Step4);
            float *out = p.dst + (tile * 16 + g8 + 8 * r) * kBlock + 8 * q4;
            // rotation-sign variant: the inverse is D W
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)   // (+ 0: a missing row, scale 0, reads as +0)
                    v[i] = fmaf(d[2 * e + (i >> 2)][(i >> 1) & 1][2 * r + (i & 1)], scale, 0.f);
                if (p.src.has_signs) {
                    const uint32_t sg = cur.present[r] ? p.src.signs[e] >> (8 * q4) : 0u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(__float_as_uint(v[i]) ^ ((sg >> i) << 31));
                }
                store8(out + 32 * e, v, wide);
            }
        }
    }
}

}  // namespace

tq_status launch_decode(const tq_cache &src, int32_t seq_id, int64_t pos0, int64_t n_tokens,
                        float *dst, cudaStream_t stream) {
    DecodeParams p;
    p.src = make_view(src);
    p.dst = dst;
    p.pos0 = pos0;
    p.seq_id = seq_id;
    p.bpr = src.n_kv_heads * (src.head_dim / kBlock);
    p.n_blocks = n_tokens * p.bpr;
    const int64_t grid = (p.n_blocks + 7) / 8;
    if (grid > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
    if (src.type == TQ_TURBO4) {
        // a wave of resident CTAs (four of four warps per SM)
        const int64_t ctas = min64((p.n_blocks + 16 * kDecodeWarps - 1) / (16 * kDecodeWarps), (int64_t)4 * device_sm_count());
        PdlConfig lc(dim3((unsigned)ctas), dim3(32 * kDecodeWarps), 0, stream);
        return check_cuda(cudaLaunchKernelEx(&lc.cfg, decode4_kernel, p));
    } else if (src.type == TQ_TURBO3)
        decode_kernel<TQ_TURBO3><<<(unsigned)grid, 256, 0, stream>>>(p);
    else
        decode_kernel<TQ_TURBO2><<<(unsigned)grid, 256, 0, stream>>>(p);
    return check_cuda(cudaGetLastError());
}

}  // namespace tq
