// Attention over the paged cache: which kernels take a batch.
#include "tq_internal.h"

namespace tq {

// Batches of one row per sequence go to the split-K decode, whose time grows with the groups of eight
// heads per KV head (it streams the keys once for each); the others to the chunk kernel, whose
// products fill 128 rows whatever the batch holds.  The same single rows through both, us (cold L2,
// 2 KV heads, bf16; the chunk kernel in two parts takes 1.2 times as long):
//   heads per KV head              4     8    12    16    24    32    64   chunk kernel, any
//   32 sequences of 32,000 keys   76   130   240   240   353   464   910   249
//   64 of 2,000                   27    36    54    54    74    91   163    69
//   8 of 8,000                    23    27    32    32    40    47    75    49
// So the decode is the slower one above 16 heads per KV head where the batch fills the GPU, above 32
// where it does not.  A batch with a chunk in it runs its single rows on the chunk kernel too: 512 rows of
// one sequence beside 32 single rows, 4,000 keys each, 32 heads on 8, take 200 us in one call and 71 + 53 in two.
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
