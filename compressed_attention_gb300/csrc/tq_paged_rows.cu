// Append to the paged cache.
//
// k_paged_append_wht: SET_ROWS through the block table with the keys' position
// rotation applied on the way.  The row's encode is the write path's (tq_wht.cuh): four
// threads per row, eight rows per warp, the canonical order of norm, division and
// butterfly, so the stored bytes equal those of a plain fp32 sequence.  The rotation's
// pairs (j, j + 64) and (j, j + 32) and adjacent pairs lie inside one thread's chunks;
// pairs (j, j + 16) cross to the thread two over.  A CTA takes keys or values, so it keeps one
// codebook grid.
#include "tq_paged.cuh"
#include "tq_qprep.cuh"
#include "tq_wht.cuh"

namespace tq {

namespace {

struct AppendSide {
  RowsView src;
  uint8_t *pages;
  uint32_t wht_neg[4];
  float b[15];
  const BucketTable *bt;
  const float *pit;  // dense: R^T, fp32
};
struct AppendParams {
  PagedView pv;
  RopeView rope;
  AppendSide side[2];  // keys, values
  int only;            // 0 or 1: that side; 2: both
  int k_ctas;          // the first CTAs take the keys, the others the values
};

// Position rotation of a row in quarter layout (register element 8i + e = row element
// 32i + 8q + e); every thread of the warp calls.
__device__ __forceinline__ void rope_quarter(float (&x)[WT_E], int q, const RopeView &r, int pos) {
  const int half = r.rot_dim >> 1;
  const float *ct = r.cos_t + (size_t)pos * half, *st = r.sin_t + (size_t)pos * half;
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (32 * i < r.rot_dim) {
        const float4 c4 = *reinterpret_cast<const float4 *>(ct + 16 * i + 4 * q);
        const float4 s4 = *reinterpret_cast<const float4 *>(st + 16 * i + 4 * q);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float a = x[8 * i + 2 * m], b = x[8 * i + 2 * m + 1];
          x[8 * i + 2 * m] = rot_first(a, b, c[m], s[m]);
          x[8 * i + 2 * m + 1] = rot_second(a, b, c[m], s[m]);
        }
      }
    }
    return;
  }
  // eight angles from table entry `at` on, for register groups ga and gb
  auto turn8 = [&](int ga, int gb, int at) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 c4 = *reinterpret_cast<const float4 *>(ct + at + 4 * h);
      const float4 s4 = *reinterpret_cast<const float4 *>(st + at + 4 * h);
      const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int m = 0; m < 4; m += 2) {
        const int e = 4 * h + m;
        const F2 a = f2(x[8 * ga + e], x[8 * ga + e + 1]), b = f2(x[8 * gb + e], x[8 * gb + e + 1]);
        const F2 cc = f2(c[m], c[m + 1]), ss = f2(s[m], s[m + 1]);
        // packed products, scalar sums: a packed product feeding a packed sum may be contracted
        float ac0, ac1, bs0, bs1, as0, as1, bc0, bc1;
        f2_split(f2_mul(a, cc), ac0, ac1), f2_split(f2_mul(b, ss), bs0, bs1);
        f2_split(f2_mul(a, ss), as0, as1), f2_split(f2_mul(b, cc), bc0, bc1);
        x[8 * ga + e] = __fsub_rn(ac0, bs0), x[8 * ga + e + 1] = __fsub_rn(ac1, bs1);
        x[8 * gb + e] = __fadd_rn(as0, bc0), x[8 * gb + e + 1] = __fadd_rn(as1, bc1);
      }
    }
  };
  if (r.rot_dim == 128) {
    turn8(0, 2, 8 * q);
    turn8(1, 3, 32 + 8 * q);
  } else if (r.rot_dim == 64) {
    turn8(0, 1, 8 * q);
  } else {  // 32: elements 8q + e with those of thread q ^ 2
    const int at = 8 * (q & 1);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float o = __shfl_xor_sync(FULL_MASK, x[e], 2);
      const float c = ct[at + e], s = st[at + e];
      x[e] = (q & 2) ? rot_second(o, x[e], c, s) : rot_first(x[e], o, c, s);
    }
  }
}

// Where a batch row goes; row < 0: nowhere.
struct Place {
  int64_t at;  // byte of the packed row, or -1
  int pos;
};
__device__ __forceinline__ Place place_row(const PagedView &v, int tok, int h, bool flag) {
  const int b = paged_seq(v, tok);
  const int n = paged_len(v, b, flag);
  Place pl{-1, paged_pos(v, b, tok, n)};
  if (pl.pos >= 0 && pl.pos < n) {
    const int pg = paged_page(v, b, pl.pos, flag);
    if (pg >= 0) pl.at = (int64_t)paged_row(v, pg, h, pl.pos & ((1 << v.page_shift) - 1));
  }
  return pl;
}

template <int SRC>
__global__ void __launch_bounds__(WT_THREADS) k_paged_append_wht(const AppendParams p) {
  __shared__ WhtTables tb;
  const int side = (int)blockIdx.x < p.k_ctas ? 0 : 1;
  const AppendSide &sd = p.side[side];
  pdl_trigger();
  wht_tables_fill<TQ_FMT_TURBO4>(sd.b, sd.bt, tb);
  __syncthreads();
  pdl_wait();
  const float gs = tb.gs, go = tb.go;
  const int gn = tb.gn;
  const int q = threadIdx.x & 3, l16 = threadIdx.x & 15, sub = (threadIdx.x & 31) >> 2;
  uint32_t nq[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) nq[i] = sd.wht_neg[i] >> (8 * q);
  // Rows in groups of eight per warp: this thread's row moves on by 8 * step rows a turn, kept as
  // (token, head) with the sequence and its length beside it (tokens only grow, so the sequence
  // is found by stepping on from the last one).
  const int Hkv = p.pv.Hkv, n_rows = paged_rows(p.pv) * Hkv;
  const int cta = side ? blockIdx.x - p.k_ctas : blockIdx.x, n_cta = side ? gridDim.x - p.k_ctas : p.k_ctas;
  const int step = n_cta * (WT_THREADS / 32), n_iter = (n_rows + 7) / 8;
  const int d_tok = 8 * step / Hkv, d_head = 8 * step - d_tok * Hkv;
  int it = cta * (WT_THREADS / 32) + (threadIdx.x >> 5);
  int tok = (it * 8 + sub) / Hkv, head = it * 8 + sub - tok * Hkv;
  int b = -1, b_end = 0, len = 0;  // the row's sequence, the row after its last, its length
  const bool turn = side == 0 && p.rope.rot_dim != 0;
  Quarter<SRC> raw;
  Place pl{-1, 0};
  auto fetch = [&](int i) {
    pl.at = -1;
    if (i < n_iter && i * 8 + sub < n_rows) {
      load_quarter<SRC>(sd.src.data + tok * sd.src.token_bytes + head * sd.src.head_bytes, q, true, raw);
      if (b < 0 || tok >= b_end) {
        if (b < 0 || !p.pv.cu_q) b = paged_seq(p.pv, tok);
        else
          do ++b;
          while (b + 1 < p.pv.B && p.pv.cu_q[b + 1] <= tok);
        b_end = p.pv.cu_q ? p.pv.cu_q[b + 1] : tok + 1;
        len = paged_len(p.pv, b, q == 0);
      }
      pl.pos = len - (b_end - tok);
      if (pl.pos >= 0 && pl.pos < len) {
        const int pg = paged_page(p.pv, b, pl.pos, q == 0);
        if (pg >= 0) pl.at = (int64_t)paged_row(p.pv, pg, head, pl.pos & ((1 << p.pv.page_shift) - 1));
      }
      tok += d_tok, head += d_head;
      if (head >= Hkv) head -= Hkv, ++tok;
    }
  };
  fetch(it);
  for (; it < n_iter; it += step) {
    const Place at = pl;
    float v[WT_E];
    if (at.at >= 0) {
      unpack_quarter(raw, v);
    } else {
#pragma unroll
      for (int i = 0; i < WT_E; ++i) v[i] = 0.0f;
    }
    fetch(it + step);
    if (turn) rope_quarter(v, q, p.rope, rope_pos(p.rope, at.at >= 0 ? at.pos : 0, p.pv.status, q == 0));
    const float n = quarter_norm_normalize(v);  // shuffles: every lane of the warp takes part
    wht_quarter(v, nq, q);
    if (at.at >= 0) {
      uint8_t *dst = sd.pages + at.at;
      if (gn)
        pack_quarter<TQ_FMT_TURBO4, true>(v, n, tb.ce, l16, gs, go, gn, tb.sb, dst, q);
      else
        pack_quarter<TQ_FMT_TURBO4, false>(v, n, tb.ce, l16, gs, go, gn, tb.sb, dst, q);
    }
  }
}

// Dense rotation: a warp per row, R^T staged once per CTA.
constexpr int AD_WARPS = 8;
constexpr size_t AD_SMEM = (size_t)D * D * 4 + AD_WARPS * D * 4;
__global__ void __launch_bounds__(AD_WARPS * 32) k_paged_append_dense(const AppendParams p) {
  extern __shared__ __align__(16) float asm_f[];
  float *rt = asm_f, *uv = asm_f + D * D;
  const int side = (int)blockIdx.x < p.k_ctas ? 0 : 1;
  const int cta = side ? blockIdx.x - p.k_ctas : blockIdx.x, n_cta = side ? gridDim.x - p.k_ctas : p.k_ctas;
  const AppendSide &sd = p.side[side];
  __shared__ float sb[16];
  __shared__ __align__(16) uint8_t ib[AD_WARPS][D];
  pdl_trigger();
  stage_matrix(rt, sd.pit);
  if (threadIdx.x < 15) sb[threadIdx.x] = sd.b[threadIdx.x];
  __syncthreads();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *u = uv + warp * D;
  const int64_t n_rows = (int64_t)paged_rows(p.pv) * p.pv.Hkv;
  for (int64_t row = (int64_t)cta * AD_WARPS + warp; row < n_rows; row += (int64_t)n_cta * AD_WARPS) {
    const int tok = (int)(row / p.pv.Hkv), h = (int)(row - (int64_t)tok * p.pv.Hkv);
    const Place at = place_row(p.pv, tok, h, lane == 0);
    if (at.at < 0) continue;
    float x[4];
    load_lane4(sd.src.data + tok * sd.src.token_bytes + h * sd.src.head_bytes, sd.src.dtype, lane, x);
    if (side == 0) rope_lane4(x, lane, p.rope, p.rope.rot_dim ? rope_pos(p.rope, at.pos, p.pv.status, lane == 0) : 0);
    float s = __fadd_rn(__fadd_rn(__fmul_rn(x[0], x[0]), __fmul_rn(x[1], x[1])),
                        __fadd_rn(__fmul_rn(x[2], x[2]), __fmul_rn(x[3], x[3])));
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s = __fadd_rn(s, __shfl_xor_sync(FULL_MASK, s, m));
    const float n = __fsqrt_rn(s);
#pragma unroll
    for (int e = 0; e < 4; ++e) u[4 * lane + e] = n == 0.0f ? 0.0f : __fdiv_rn(x[e], n);
    __syncwarp();
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int k = 0; k < D; ++k) {
      const float uk = u[k];
#pragma unroll
      for (int m = 0; m < 4; ++m) y[m] = fmaf(rt[k * D + lane + 32 * m], uk, y[m]);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) ib[warp][lane + 32 * m] = (uint8_t)bucket<15>(y[m], sb);
    __syncwarp();
    uint32_t *dst = reinterpret_cast<uint32_t *>(sd.pages + at.at);
    if (lane < 16) {
      const uint2 w = *reinterpret_cast<const uint2 *>(&ib[warp][8 * lane]);
      uint32_t out = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) out |= ((w.x >> (8 * e)) & 15u) << (4 * e) | ((w.y >> (8 * e)) & 15u) << (16 + 4 * e);
      dst[1 + lane] = out;
    }
    if (lane == 0) dst[0] = __float_as_uint(n);
    __syncwarp();
  }
}

// A key row with its rotation takes about 5/4 of a value row's instructions: the CTAs are shared
// out in that proportion.
template <typename K>
cudaError_t launch_rows(K kern, AppendParams p, int threads, int rows_per_cta, size_t smem, int sms, cudaStream_t st) {
  cudaError_t e = smem ? kernel_smem_attr((const void *)kern, (int)smem) : cudaSuccess;
  int blocks = 1;
  if (e == cudaSuccess) e = kernel_occupancy((const void *)kern, threads, smem, &blocks);
  if (e != cudaSuccess) return e;
  const int sides = p.only == 2 ? 2 : 1;
  const int64_t want = ((int64_t)p.pv.n_tokens * p.pv.Hkv + rows_per_cta - 1) / rows_per_cta;
  const int64_t most = (int64_t)sms * blocks;
  const int grid = (int)(want * sides < most ? want * sides : most);
  p.k_ctas = p.only == 0 ? grid : (p.only == 1 ? 0 : grid / 2);
  if (p.only == 2 && grid == most && p.rope.rot_dim) p.k_ctas = grid * 5 / 9;
  return launch_pdl(kern, dim3(grid), dim3(threads), smem, st, p);
}

cudaError_t launch_append(const AppendParams &p, bool dense, int dtype, int sms, cudaStream_t st) {
  if (dense) return launch_rows(k_paged_append_dense, p, AD_WARPS * 32, AD_WARPS, AD_SMEM, sms, st);
  constexpr int per = 8 * (WT_THREADS / 32);
  if (dtype == TQ_DTYPE_F32) return launch_rows(k_paged_append_wht<TQ_DTYPE_F32>, p, WT_THREADS, per, 0, sms, st);
  if (dtype == TQ_DTYPE_BF16) return launch_rows(k_paged_append_wht<TQ_DTYPE_BF16>, p, WT_THREADS, per, 0, sms, st);
  return launch_rows(k_paged_append_wht<TQ_DTYPE_F16>, p, WT_THREADS, per, 0, sms, st);
}

}  // namespace

cudaError_t launch_paged_append(const tq_ctx *k, const tq_ctx *v, const PagedView &pv, uint8_t *kp, uint8_t *vp,
                                const RowsView &kr, const RowsView &vr, const RopeView &rope, cudaStream_t st) {
  AppendParams p{};
  p.pv = pv;
  p.rope = rope;
  const tq_ctx *ctx[2] = {k, v};
  const RowsView *rows[2] = {&kr, &vr};
  for (int i = 0; i < 2; ++i) {
    AppendSide &s = p.side[i];
    s.src = *rows[i];
    s.pages = i ? vp : kp;
    for (int j = 0; j < 4; ++j) s.wht_neg[j] = ctx[i]->wht_neg[j];
    for (int j = 0; j < 15; ++j) s.b[j] = ctx[i]->cb.b[j];
    s.bt = ctx[i]->d_bt;
    s.pit = ctx[i]->d_pit;
  }
  const bool dk = k->p.rotation == TQ_ROT_DENSE, dv = v->p.rotation == TQ_ROT_DENSE;
  if (dk == dv) {
    p.only = 2;
    return launch_append(p, dk, kr.dtype, k->num_sms, st);
  }
  for (p.only = 0; p.only < 2; ++p.only) {  // one rotation kind each: one launch per side
    const cudaError_t e = launch_append(p, p.only ? dv : dk, kr.dtype, k->num_sms, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace tq
