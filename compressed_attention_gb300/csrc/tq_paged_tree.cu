// Attention of drafted trees over the paged cache.
//
// A CTA per (node, KV head): the node's heads one after the other over the keys that it sees, 128 at a
// time: a thread per key for the scores, a thread per dimension for the values.
#include <math.h>

#include "tq_decode_common.cuh"
#include "tq_paged.cuh"

namespace tq {

namespace {

struct SimpleParams {
  PagedView pv;
  const int32_t *parents;
  const uint8_t *kp, *vp;
  RowsView q;
  RopeView rope;
  PagedOut o;
  int Hq, gq;
  float scale;
  const float *kr, *vr;
  float kc[16], vc[16];
};

__global__ void __launch_bounds__(128) k_tree_simple(const SimpleParams p) {
  __shared__ float x[D], y[D], s[128], w[128];
  __shared__ uint32_t anc[TREE_MAX / 32];
  const int tok = blockIdx.x, kvh = blockIdx.y, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  if (tok >= paged_rows(p.pv)) return;
  const int b = paged_seq(p.pv, tok), n = paged_len(p.pv, b, true);
  const int lo = p.pv.cu_q ? p.pv.cu_q[b] : b, T = p.pv.cu_q ? p.pv.cu_q[b + 1] - lo : 1, i = tok - lo;
  const int base = n - T, slot = base + i;
  if (tid < TREE_MAX / 32) anc[tid] = 0;
  __syncthreads();
  const bool none = slot < 0 || i >= p.pv.max_q;
  if (i >= p.pv.max_q && tid == 0) atomicExch(p.pv.status, (int32_t)DEVERR_SEQLEN);
  if (tid == 0 && !none)
    for (int m = i; m >= 0; m = tree_parent(p.parents, lo, m, p.pv.status, true)) anc[m >> 5] |= 1u << (m & 31);
  __syncthreads();
  for (int h = kvh * p.gq; h < (kvh + 1) * p.gq; ++h) {
    float acc = 0.f, l = 0.f, M = -INFINITY;
    if (!none) {
      if (tid < 32) {
        float v[4];
        load_lane4(p.q.data + tok * p.q.token_bytes + h * p.q.head_bytes, p.q.dtype, tid, v);
        if (p.rope.rot_dim) rope_lane4(v, tid, p.rope, rope_pos(p.rope, tree_pos(p.pv, p.parents, b, tok, slot, false), p.pv.status, true));
        for (int e = 0; e < 4; ++e) x[4 * tid + e] = v[e];
      }
      __syncthreads();
      float a = 0.f;
      for (int k = 0; k < D; ++k) a = fmaf(p.kr[tid * D + k], x[k], a);
      y[tid] = a * p.scale * LOG2E;
      __syncthreads();
      for (int k0 = 0; k0 < n; k0 += 128) {
        const int t = k0 + tid, j = t - base;
        const bool see = t < n && (j < 0 || (j < TREE_MAX && ((anc[j >> 5] >> (j & 31)) & 1u)));
        float sc = -INFINITY;
        if (see) {
          const uint8_t *r = p.kp + paged_row(p.pv, max(paged_page(p.pv, b, t, true), 0), kvh, t & ((1 << p.pv.page_shift) - 1));
          float d = 0.f;
          for (int e = 0; e < 64; ++e) d += p.kc[r[4 + e] & 15] * y[2 * e] + p.kc[r[4 + e] >> 4] * y[2 * e + 1];
          sc = d * *reinterpret_cast<const float *>(r);
        }
        s[tid] = sc;
        __syncthreads();
        float bm = -INFINITY;
        for (int e = 0; e < 128; ++e) bm = fmaxf(bm, s[e]);
        const float mn = fmaxf(M, bm), mu = mn == -INFINITY ? 0.f : mn, f = exp2f(M - mu);
        w[tid] = see ? exp2f(sc - mu) : 0.f;
        __syncthreads();
        M = mn, l *= f, acc *= f;
        for (int e = 0; e < 128 && k0 + e < n; ++e) {
          if (w[e] == 0.f) continue;
          const int te = k0 + e;
          const uint8_t *r = p.vp + paged_row(p.pv, max(paged_page(p.pv, b, te, false), 0), kvh, te & ((1 << p.pv.page_shift) - 1));
          const int idx = (r[4 + tid / 2] >> (4 * (tid & 1))) & 15;
          l += w[e];
          acc += w[e] * *reinterpret_cast<const float *>(r) * p.vc[idx];
        }
        __syncthreads();
      }
    }
    x[tid] = l == 0.f ? 0.f : acc / l;
    __syncthreads();
    float o = 0.f;
    for (int k = 0; k < D; ++k) o = fmaf(p.vr[k * D + tid], x[k], o);
    y[tid] = o;
    __syncthreads();
    if (tid < 32) {
      const float v[4] = {y[4 * tid], y[4 * tid + 1], y[4 * tid + 2], y[4 * tid + 3]};
      if (i < p.pv.max_q) store_lane4(p.o.out, p.o.dtype, ((size_t)tok * p.Hq + h) * D, tid, v);
    }
    __syncthreads();
  }
}

}  // namespace

// One node per sequence sees all of its sequence's keys: a single row of the paged decode.
static bool is_decode(const PagedView &pv, int Hq) { return pv.max_q == 1 && Hq / pv.Hkv <= 16; }

bool paged_tree_workspace(const tq_ctx *k, const PagedView &pv, int Hq, size_t *bytes) {
  if (is_decode(pv, Hq)) return paged_decode_workspace(k, pv, Hq, bytes);
  *bytes = 256;
  return true;
}

cudaError_t launch_paged_tree(const tq_ctx *k, const tq_ctx *v, const PagedView &pv, const int32_t *parents,
                              const uint8_t *kp, const uint8_t *vp, const RowsView &q, int Hq, const RopeView &rope,
                              float scale, const PagedOut &o, void *ws, cudaStream_t st) {
  if (is_decode(pv, Hq)) return launch_paged_decode(k, v, pv, kp, vp, q, Hq, rope, scale, o, ws, st);
  SimpleParams p{};
  p.pv = pv, p.parents = parents, p.kp = kp, p.vp = vp, p.q = q, p.rope = rope, p.o = o;
  p.Hq = Hq, p.gq = Hq / pv.Hkv, p.scale = scale, p.kr = k->d_pi, p.vr = v->d_pi;
  for (int i = 0; i < 16; ++i) p.kc[i] = k->cb.c[i], p.vc[i] = v->cb.c[i];
  return launch_pdl(k_tree_simple, dim3(pv.n_tokens, pv.Hkv), dim3(128), 0, st, p);
}

}  // namespace tq
