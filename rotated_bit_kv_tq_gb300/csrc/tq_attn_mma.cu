// tq_attn_mma.cu -- tensor-core decode attention: host side and the turbo2 / turbo3 kernels
// (tq_attn_mma_kernel.cuh holds the kernel).
#include <atomic>

#include "tq_attn_mma_kernel.cuh"

namespace tq {
namespace {

// Launches still to run with injected timeouts (tq_inject_wait_timeout).
std::atomic<int> g_inject_timeouts{0};

}  // namespace

bool take_injected_timeout() {
    for (int n = g_inject_timeouts.load(); n > 0;)
        if (g_inject_timeouts.compare_exchange_weak(n, n - 1)) return true;
    return false;
}

namespace {

template <int NB>
tq_status launch_nb(int tk, int tv, const MmaParams &p, int n_seqs, cudaStream_t stream) {
    if (tk == TQ_TURBO4 || tv == TQ_TURBO4) return launch_attn_mma_t4(tk, tv, NB, &p, n_seqs, stream);
    if (tk == TQ_TURBO3 && tv == TQ_TURBO3) return launch_t<3, 3, NB>(p, n_seqs, stream);
    if (tk == TQ_TURBO2 && tv == TQ_TURBO2) return launch_t<2, 2, NB>(p, n_seqs, stream);
    if (tk == TQ_TURBO3 && tv == TQ_TURBO2) return launch_t<3, 2, NB>(p, n_seqs, stream);
    return launch_t<2, 3, NB>(p, n_seqs, stream);
}

size_t stage_bytes_for(int tile_tokens, size_t rk, size_t rv) {
    return ((size_t)tile_tokens * (rk + rv) + 16 + 127) & ~size_t(127);
}

// Rows per tile: two 32-row slices per warp of a KV head, or one where two stages of those
// would not fit (pairs with a turbo4 cache at eight KV heads: 928-byte row pairs).
int tile_tokens_for(int wph, size_t qbytes, size_t rk, size_t rv) {
    const int full = kWarpTokens * wph;
    return qbytes + 128 + 2 * stage_bytes_for(full, rk, rv) <= kSmemBudget ? full : full / 2;
}

}  // namespace

bool grid_merge_fits(int n_seqs, int n_splits) {
    return n_seqs == 1 && n_splits <= std::min(device_sm_count(), kGridMergeMaxCtas);
}

bool attn_mma_supported(const tq_cache &k, const tq_cache &v, int n_q_heads) {
    const int hkv = k.n_kv_heads, nb = k.head_dim / kBlock, G = n_q_heads / hkv;
    if (nb < 1 || nb > 2 || G > 8) return false;
    if (hkv < 1 || hkv > consumers(nb) || consumers(nb) % hkv) return false;
    const size_t rk = tq_row_bytes(k.type, hkv, k.head_dim), rv = tq_row_bytes(v.type, hkv, v.head_dim);
    if (rk % 16 || rv % 16) return false;
    const int TT = tile_tokens_for(consumers(nb) / hkv, q_bytes(n_q_heads, nb), rk, rv);
    if (k.page_tokens && k.page_tokens % 16) return false;
    if (v.page_tokens && v.page_tokens % 16) return false;
    const size_t qbytes = q_bytes(n_q_heads, nb);
    return qbytes + 128 + 2 * stage_bytes_for(TT, rk, rv) <= kSmemBudget;
}

tq_status launch_attn_mma(const tq_cache &k, const tq_cache &v, const void *q, int n_seqs,
                          int n_q_heads, const int32_t *seq_lens, int64_t max_seq_len, float scale,
                          float *part, int n_splits, int tokens_per_split, int cluster,
                          const void *k_new, const void *v_new, OutPtr out, uint64_t *bar,
                          cudaStream_t stream) {
    MmaParams p;
    p.kc = make_view(k);
    p.vc = make_view(v);
    p.q = static_cast<const __half *>(q);
    p.k_new = static_cast<const __half *>(k_new);
    p.v_new = static_cast<const __half *>(v_new);
    p.seq_lens = seq_lens;
    p.part = part;
    p.score_scale = scale * kLog2e * kInvSqrt128 / centroid_h_scale(k.type);
    p.v_unscale = (v.type == TQ_TURBO4 ? kVUp<TQ_TURBO4> : 1.0f) / centroid_h_scale(v.type);
    p.max_len = max_seq_len;
    p.n_q_heads = n_q_heads;
    p.n_kv_heads = k.n_kv_heads;
    p.group = n_q_heads / k.n_kv_heads;
    p.head_dim = k.head_dim;
    p.n_splits = n_splits;
    p.tokens_per_split = tokens_per_split;
    const int nb = k.head_dim / kBlock;
    p.wph = consumers(nb) / k.n_kv_heads;
    p.tile_tokens = tile_tokens_for(p.wph, q_bytes(n_q_heads, nb), p.kc.row_bytes, p.vc.row_bytes);
    p.wait_limit = kWaitLimit;
    p.withhold_tiles = 0;
    p.out = out;
    p.bar = bar;
    p.grid_wait_limit = kGridWaitLimit;
    if (out.p && (cluster != 1 || !bar || !grid_merge_fits(n_seqs, n_splits))) return TQ_ERR_UNSUPPORTED;
    if (take_injected_timeout()) {
        p.wait_limit = kInjectedWaitLimit;
        p.withhold_tiles = 1;
    }
    p.mul2 = 2u;
    p.mul4 = 4u;
    p.hi16 = 1u << 16;
    p.hi30 = 1u << 30;
    p.hi31 = 1u << 31;
    const size_t stage = stage_bytes_for(p.tile_tokens, p.kc.row_bytes, p.vc.row_bytes);
    p.stage_bytes = (int)stage;
    const size_t qbytes = q_bytes(n_q_heads, nb);
    p.stages = (int)std::min<size_t>(4, (kSmemBudget - qbytes - 128) / stage);
    if (p.stages < 2) return TQ_ERR_UNSUPPORTED;
    if (cluster < 1 || cluster > kClusterSplits || n_splits % cluster) return TQ_ERR_UNSUPPORTED;
    p.cl = cluster;
    const size_t cpart = (size_t)n_q_heads * part_stride(k.head_dim) * sizeof(float);
    if (cpart > (size_t)p.stages * stage) return TQ_ERR_UNSUPPORTED;
    p.cpart_offset = (int)(((size_t)p.stages * stage - cpart) & ~size_t(15));
    return nb == 1 ? launch_nb<1>(k.type, v.type, p, n_seqs, stream)
                   : launch_nb<2>(k.type, v.type, p, n_seqs, stream);
}

tq_status inject_wait_timeout(int n_calls) {
    if (n_calls < 0) return TQ_ERR_INVALID_ARGUMENT;
    g_inject_timeouts.store(n_calls);
    return TQ_OK;
}

}  // namespace tq

extern "C" tq_status tq_inject_wait_timeout(int n_calls) { return tq::inject_wait_timeout(n_calls); }
