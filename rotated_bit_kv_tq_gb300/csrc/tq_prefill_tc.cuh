// tq_prefill_tc.cuh -- what the prompt-chunk kernels on tcgen05 share: the launch parameters, the
// operand layouts, the fp16 MMAs, the bounded wait and the cluster exchange.
#pragma once
#include "tq_internal.cuh"
#include "tq_simd.cuh"
#include "tq_codes.cuh"
#include "tq_tcgen05.cuh"

namespace tq {
namespace {

constexpr int kTcRows = 128;          // (query token, head) rows per CTA = TMEM lanes
constexpr int kTcKeys = 128;          // keys per tile
constexpr int kTcSoftmax = 256;       // warps 0-7: two threads per row (one per 64-key half)
constexpr int kTcGroup = 128;         // threads of one producer group (warps 8-11 K, 12-15 V)
constexpr int kTcProducer = 2 * kTcGroup;
constexpr int kTcMmaWarp = (kTcSoftmax + kTcProducer) / 32;
constexpr int kTcThreads = kTcSoftmax + kTcProducer + 32;
constexpr uint32_t kTcWaitLimit = 1u << 20;
constexpr uint32_t kTcPollLimit = 1u << 24;   // polls without progress of the MMA thread
constexpr float kTcLog2e = 1.4426950408889634f;

struct TcParams {
    CacheView kc, vc;
    const __half *q;        // [n_q][Hq][128] fp16
    OutPtr out;             // [n_q][Hq][head_dim]
    int64_t pos0, n_q;
    int32_t seq, n_q_heads, group, bq;
    int32_t n_kv_heads;
    int64_t n_qblocks;      // query blocks of bq tokens
    int32_t chunked_k, chunked_v;
    float score_scale;      // softmax scale * log2(e) / (sqrt(128) * h_scale of the K table)
    float out_scale;        // 1 / (sqrt(128) * h_scale of the V table)
    int32_t split;          // CTAs per query block: 1, or 2 (a cluster: key tiles cut in two halves)
};

// Byte offset of element (r, c) of a 128-column tile in the no-swizzle canonical layout with
// rows along M/N (8-row groups 2048 bytes apart) and columns along K (8-column groups 128
// bytes apart).
__device__ __forceinline__ uint32_t canon(int r, int c) {
    return (uint32_t)((r >> 3) * 2048 + (c >> 3) * 128 + (r & 7) * 16 + (c & 7) * 2);
}
// The MN-major V tile: keys are K (8-key groups 2048 bytes apart), coords are N (8-coord
// groups 128 bytes apart), coords contiguous inside a core matrix.
__device__ __forceinline__ uint32_t canon_mn(int key, int c) {
    return (uint32_t)((c >> 3) * 128 + (key >> 3) * 2048 + (key & 7) * 16 + (c & 7) * 2);
}

// Instruction descriptor, kind::f16: fp32 accumulate, fp16 A and B, M = 128, N = 128.
constexpr uint32_t idesc_f16(bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void tc_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
                 ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// The same with A read from tensor memory (row m = lane m, two fp16 K values per column).
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
                 ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// Bounded wait on a phase; false (and TQ_ERR_DEVICE_TIMEOUT recorded) on timeout.
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity) {
    for (uint32_t it = 0; it < kTcWaitLimit; ++it) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}\n"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        if (ok) return true;
    }
    record_error(TQ_ERR_DEVICE_TIMEOUT);
    return false;
}
// Cluster-wide barrier, each thread on its own (not warp-aligned): every thread of both CTAs
// of a split query block passes it exactly twice (before and after the partial exchange).
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t local, uint32_t rank) {
    uint32_t ra;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ra) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t local, uint32_t rank) {
    uint32_t ra;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(ra) : "memory");
    return v;
}

// The part u of a turbo4 V norm v that the V operand takes (u c is exact in fp16; the weights take
// v / u): the power of two at or below v, at most 2^12; a norm below fp16's normal range stays as
// it is.
__device__ __forceinline__ __half v_scale(uint32_t bits) {
    const uint32_t b = bits & 0xfc00u;
    return __ushort_as_half((uint16_t)((b & 0x7c00u) > 0x6c00u ? 0x6c00u : b & 0x7c00u ? b : bits));
}

// In-thread Walsh-Hadamard butterflies over 64 values, h = 1 .. 32.
__device__ __forceinline__ void fwht64(float (&x)[64]) {
#pragma unroll
    for (int h = 1; h < 64; h <<= 1)
#pragma unroll
        for (int i = 0; i < 64; ++i)
            if (!(i & h)) {
                const float a = x[i], b = x[i + h];
                x[i] = a + b;
                x[i + h] = a - b;
            }
}

}  // namespace
}  // namespace tq
