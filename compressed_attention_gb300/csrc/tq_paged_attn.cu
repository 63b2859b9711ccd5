// Attention over the paged cache: which kernels take a batch.
#include "tq_internal.h"

namespace tq {

// Batches of one row per sequence go to the split-K decode, which streams a key tile in about
// half the time of the chunk kernel's tile (its products fill 128 rows whatever the batch holds);
// the others to the chunk kernel.
bool paged_workspace(const tq_ctx *k, const PagedView &pv, int Hq, size_t *bytes) {
  return pv.max_q == 1 ? paged_decode_workspace(k, pv, Hq, bytes) : paged_prefill_workspace(k, pv, Hq, bytes);
}

cudaError_t launch_paged_attention(const tq_ctx *k, const tq_ctx *v, const PagedView &pv, const uint8_t *kp,
                                   const uint8_t *vp, const RowsView &q, int Hq, const RopeView &rope, float scale,
                                   const PagedOut &o, void *ws, cudaStream_t st) {
  return pv.max_q == 1 ? launch_paged_decode(k, v, pv, kp, vp, q, Hq, rope, scale, o, ws, st)
                       : launch_paged_prefill(k, v, pv, kp, vp, q, Hq, rope, scale, o, ws, st);
}

}  // namespace tq
