// Causal attention over the paged cache, the plain kernel: a CTA takes one row and up to
// eight q-heads of a KV head, a warp one q-head.  q is rotated by its position and by R in
// shared memory; a lane scores one key at a time from its nibbles, the warp keeps the
// running maximum and sum, and the values are accumulated four elements per lane in the
// rotated basis; R^T o, the differential pair and the store end the row.
#include <math.h>

#include "tq_decode_common.cuh"
#include "tq_paged.cuh"

namespace tq {

namespace {

constexpr int AW = 8;

struct AttnParams {
  PagedView pv;
  const uint8_t *kp, *vp;
  RowsView q;
  RopeView rope;
  PagedOut o;
  int Hq, gq, n_hg;
  float scale;
  float kc[16], vc[16];
  const float *kr, *vr;  // R of the keys and of the values
};

__global__ void __launch_bounds__(AW * 32) k_paged_attention(const AttnParams p) {
  __shared__ float qs[AW][D];
  __shared__ float os[AW][D];
  __shared__ float kc[16], vc[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (threadIdx.x < 16) kc[threadIdx.x] = p.kc[threadIdx.x], vc[threadIdx.x] = p.vc[threadIdx.x];
  __syncthreads();
  pdl_wait();
  const int tok = blockIdx.x, kvh = blockIdx.y / p.n_hg, hg = blockIdx.y % p.n_hg;
  if (tok >= paged_rows(p.pv)) return;
  const int b = paged_seq(p.pv, tok), n = paged_len(p.pv, b, threadIdx.x == 0), pos = paged_pos(p.pv, b, tok, n);
  const int hh = hg * AW + warp, head = kvh * p.gq + hh;
  const bool live = hh < p.gq;
  const int psz = 1 << p.pv.page_shift;
  float M = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (live && pos >= 0) {
    float x[4];
    load_lane4(p.q.data + tok * p.q.token_bytes + head * p.q.head_bytes, p.q.dtype, lane, x);
    rope_lane4(x, lane, p.rope, p.rope.rot_dim ? rope_pos(p.rope, pos, p.pv.status, lane == 0) : 0);
    for (int e = 0; e < 4; ++e) os[warp][4 * lane + e] = x[e];
    __syncwarp();
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < D; ++k)
      for (int m = 0; m < 4; ++m) y[m] = fmaf(p.kr[(lane + 32 * m) * D + k], os[warp][k], y[m]);
    for (int m = 0; m < 4; ++m) qs[warp][lane + 32 * m] = y[m] * p.scale;
    __syncwarp();
    for (int t0 = 0; t0 <= pos; t0 += 32) {
      const int t = t0 + lane;
      float s = -INFINITY;
      size_t at = 0;
      if (t <= pos) {
        at = paged_row(p.pv, max(paged_page(p.pv, b, t, true), 0), kvh, t & (psz - 1));
        const uint32_t *rec = reinterpret_cast<const uint32_t *>(p.kp + at);
        float d = 0.f;
        for (int w = 0; w < 16; ++w) {
          const uint32_t x8 = rec[1 + w];
          for (int e = 0; e < 8; ++e) d = fmaf(kc[(x8 >> (4 * e)) & 15u], qs[warp][8 * w + e], d);
        }
        s = d * __uint_as_float(rec[0]);
      }
      float m = s;
      for (int h = 16; h >= 1; h >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, h));
      const float Mn = fmaxf(M, m), a = expf(M - Mn), w = t <= pos ? expf(s - Mn) : 0.f;
      M = Mn;
      l = l * a + w;
      for (int e = 0; e < 4; ++e) acc[e] *= a;
      for (int i = 0; i < 32 && t0 + i <= pos; ++i) {
        const float wi = __shfl_sync(FULL_MASK, w, i);
        const uint8_t *rec = p.vp + __shfl_sync(FULL_MASK, at, i);
        const float c = wi * *reinterpret_cast<const float *>(rec);
        const uint32_t x4 = *reinterpret_cast<const uint16_t *>(rec + 4 + 2 * lane);
        for (int e = 0; e < 4; ++e) acc[e] = fmaf(c, vc[(x4 >> (4 * e)) & 15u], acc[e]);
      }
    }
    for (int h = 16; h >= 1; h >>= 1) l += __shfl_xor_sync(FULL_MASK, l, h);
  }
  const float f = l > 0.f ? 1.f / l : 0.f;
  __syncwarp();
  for (int e = 0; e < 4; ++e) os[warp][4 * lane + e] = acc[e] * f;
  __syncwarp();
  float y[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < D; ++k) {
    const float4 r4 = *reinterpret_cast<const float4 *>(p.vr + k * D + 4 * lane);
    const float ok = os[warp][k];
    y[0] = fmaf(r4.x, ok, y[0]), y[1] = fmaf(r4.y, ok, y[1]), y[2] = fmaf(r4.z, ok, y[2]), y[3] = fmaf(r4.w, ok, y[3]);
  }
  if (!p.o.diff.lambda) {
    if (live) store_lane4(p.o.out, p.o.dtype, ((size_t)tok * p.Hq + head) * D, lane, y);
    return;
  }
  for (int e = 0; e < 4; ++e) qs[warp][4 * lane + e] = y[e];
  __syncthreads();
  if ((warp & 1) || !live) return;
  const int pair = head >> 1;
  const float lam = p.o.diff.lambda[(int64_t)tok * p.o.diff.lambda_stride + pair];
  float ss = 0.f;
  for (int e = 0; e < 4; ++e) {
    y[e] = fmaf(-lam, qs[warp + 1][4 * lane + e], y[e]);
    ss = fmaf(y[e], y[e], ss);
  }
  for (int h = 16; h >= 1; h >>= 1) ss += __shfl_xor_sync(FULL_MASK, ss, h);
  const float g = p.o.diff.gain ? rsqrtf(ss * (1.0f / D) + p.o.diff.eps) : 1.f;
  for (int e = 0; e < 4; ++e) y[e] *= g * p.o.diff.out_scale * (p.o.diff.gain ? p.o.diff.gain[4 * lane + e] : 1.f);
  store_lane4(p.o.out, p.o.dtype, ((size_t)tok * (p.Hq / 2) + pair) * D, lane, y);
}

}  // namespace

bool paged_workspace(const tq_ctx *k, const PagedView &pv, int Hq, size_t *bytes) {
  if (pv.max_q == 1) return paged_decode_workspace(k, pv, Hq, bytes);
  *bytes = 256;
  return true;
}

cudaError_t launch_paged_attention(const tq_ctx *k, const tq_ctx *v, const PagedView &pv, const uint8_t *kp,
                                   const uint8_t *vp, const RowsView &q, int Hq, const RopeView &rope, float scale,
                                   const PagedOut &o, void *ws, cudaStream_t st) {
  if (pv.max_q == 1) return launch_paged_decode(k, v, pv, kp, vp, q, Hq, rope, scale, o, ws, st);
  AttnParams p{};
  p.pv = pv, p.kp = kp, p.vp = vp, p.q = q, p.rope = rope, p.o = o;
  p.Hq = Hq, p.gq = Hq / pv.Hkv, p.n_hg = (p.gq + AW - 1) / AW;
  p.scale = scale;
  for (int i = 0; i < 16; ++i) p.kc[i] = k->cb.c[i], p.vc[i] = v->cb.c[i];
  p.kr = k->d_pi, p.vr = v->d_pi;
  return launch_pdl(k_paged_attention, dim3(pv.n_tokens, pv.Hkv * p.n_hg), dim3(AW * 32), 0, st, p);
}

}  // namespace tq
