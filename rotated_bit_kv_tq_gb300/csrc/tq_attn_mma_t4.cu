// tq_attn_mma_t4.cu -- tensor-core decode attention over pairs with one turbo4 cache (mixed
// "-ctk" / "-ctv"); the kernel is tq_attn_mma_kernel.cuh's.  Two turbo4 caches run on
// tq_attn_t4.cu.
#include "tq_attn_mma_kernel.cuh"

namespace tq {
namespace {

template <int NB>
tq_status launch_nb(int tk, int tv, const MmaParams &p, int n_seqs, cudaStream_t stream) {
    if (tk == TQ_TURBO4)
        return tv == TQ_TURBO3 ? launch_t<TQ_TURBO4, TQ_TURBO3, NB>(p, n_seqs, stream)
                               : launch_t<TQ_TURBO4, TQ_TURBO2, NB>(p, n_seqs, stream);
    return tk == TQ_TURBO3 ? launch_t<TQ_TURBO3, TQ_TURBO4, NB>(p, n_seqs, stream)
                           : launch_t<TQ_TURBO2, TQ_TURBO4, NB>(p, n_seqs, stream);
}

}  // namespace

tq_status launch_attn_mma_t4(int tk, int tv, int nb, const void *params, int n_seqs, cudaStream_t stream) {
    const MmaParams &p = *static_cast<const MmaParams *>(params);
    return nb == 1 ? launch_nb<1>(tk, tv, p, n_seqs, stream) : launch_nb<2>(tk, tv, p, n_seqs, stream);
}

}  // namespace tq
