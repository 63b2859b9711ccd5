// Keeps a path of a drafted tree in the paged cache: records move towards the front of the
// tree's slots, in place.  A CTA per sequence: slot c + j takes slot c + path[j], path[j] >= j and ascending, so
// taking j in order, a chunk read before it is written, no slot is written before its own record has moved on (a
// later chunk's sources lie behind every slot that this one writes).  The same CTA reads the length and writes the
// new one, which may be the same word.  Latency bounds it (length, path, pages, then a chunk's words): 2.8 us for one sequence,
// 4.7 for 64 whose paths of some seven nodes move 0.5 MB (8 KV heads); more CTAs a sequence would have to wait for each
// other's reads.
#include "tq_paged.cuh"

namespace tq {

namespace {

constexpr int KEEP_T = 512;
constexpr int FLY = 8;                    // words of a thread in flight
constexpr int CHUNK = KEEP_T * FLY;       // words of a chunk
constexpr int ROW_W = PG_ROW / 4;

struct KeepParams {
  PagedView pv;
  uint32_t *pages[2];
  const int32_t *path;
  int64_t path_stride;
  const int32_t *n_path;
  int32_t *new_lens;
};

__global__ void __launch_bounds__(KEEP_T) k_paged_keep(const KeepParams p) {
  __shared__ int64_t from[TREE_MAX], to[TREE_MAX];  // first packed row of (page, row of the page), or -1
  __shared__ int bad;
  const int b = blockIdx.x, tid = threadIdx.x;
  const PagedView &v = p.pv;
  pdl_trigger();
  if (tid == 0) bad = 0;
  pdl_wait();
  const int len = paged_len(v, b, tid == 0);
  int T = 1, base = len - 1;
  if (v.cu_q) {
    const int a = v.cu_q[b], e = v.cu_q[b + 1];
    T = a < 0 || a >= v.n_tokens ? 0 : max(min(e, v.n_tokens) - a, 0);
    base = len - (e - a);  // (slots count rows past n_tokens too, as the append's)
  }
  const int n = T ? p.n_path[b] : 0;
  __syncthreads();
  if (T) {
    bool no = n < 0 || n > T || n > p.path_stride || n > v.max_q;  // (max_q: what a row of path holds)
    if (!no)
      for (int j = tid; j < n; j += KEEP_T) {
        const int at = p.path[b * p.path_stride + j];
        no |= at < (j ? p.path[b * p.path_stride + j - 1] + 1 : 0) || at >= T;
        from[j] = to[j] = -1;
        const int dst = base + j, src = base + at;
        if (no || at == j || dst < 0 || src >= len) continue;
        const int ps = paged_page(v, b, src, true), pd = paged_page(v, b, dst, true);
        if (ps < 0 || pd < 0) continue;
        const int m = (1 << v.page_shift) - 1;
        from[j] = (((int64_t)ps * v.Hkv) << v.page_shift) + (src & m);
        to[j] = (((int64_t)pd * v.Hkv) << v.page_shift) + (dst & m);
      }
    if (no) bad = 1;
  }
  __syncthreads();
  const bool take = T && !bad;
  if (tid == 0) {
    if (bad) atomicExch(v.status, (int32_t)DEVERR_TREE);
    p.new_lens[b] = T ? max(base + (take ? n : 0), 0) : len;
  }
  if (!take) return;
  // heads in blocks of which a slot fits a chunk; per block the slots in order, several to a chunk
  const int heads = min(2 * v.Hkv, CHUNK / ROW_W);  // of keys, then of values
  for (int h0 = 0; h0 < 2 * v.Hkv; h0 += heads) {
    const int nh = min(heads, 2 * v.Hkv - h0), per = CHUNK / (nh * ROW_W), slot_w = nh * ROW_W;
    for (int j0 = 0; j0 < n; j0 += per) {
      const int words = min(per, n - j0) * slot_w;
      uint32_t x[FLY];
      uint32_t *dst[FLY];
#pragma unroll
      for (int i = 0; i < FLY; ++i) {
        const int w = i * KEEP_T + tid;
        dst[i] = nullptr;
        if (w < words) {
          const int j = j0 + w / slot_w, hw = w % slot_w, sh = h0 + hw / ROW_W, k = hw % ROW_W;
          const int side = sh >= v.Hkv, h = sh - side * v.Hkv;
          if (from[j] >= 0) {
            const int64_t head = (int64_t)h << v.page_shift;
            x[i] = p.pages[side][(from[j] + head) * ROW_W + k];
            dst[i] = p.pages[side] + (to[j] + head) * ROW_W + k;
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < FLY; ++i)
        if (dst[i]) *dst[i] = x[i];
      __syncthreads();
    }
  }
}

}  // namespace

cudaError_t launch_paged_keep(const PagedView &pv, uint8_t *kp, uint8_t *vp, const int32_t *path, int64_t path_stride,
                              const int32_t *n_path, int32_t *new_lens, cudaStream_t st) {
  const KeepParams p{pv, {reinterpret_cast<uint32_t *>(kp), reinterpret_cast<uint32_t *>(vp)}, path, path_stride, n_path,
                     new_lens};
  return launch_pdl(k_paged_keep, dim3(pv.B), dim3(KEEP_T), 0, st, p);
}

}  // namespace tq
