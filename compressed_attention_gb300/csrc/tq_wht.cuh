// The randomized-WHT encode of a row by four threads (norm, division, butterfly, nearest
// centroid, packing): the write path's kernels and the paged append share it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

// Two fp32 values in a register pair: one instruction does both, each rounded exactly as the
// scalar operation, so that the canonical order keeps its bits at half the issue slots.
struct F2 {
  uint64_t v;
};
static __device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
static __device__ __forceinline__ void f2_split(F2 x, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
static __device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
static __device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
static __device__ __forceinline__ F2 f2_sub(F2 a, F2 b) {
  F2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
static __device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// x / n rounded to nearest, given r = RN(1/n): q = RN(x r) is within one ulp of x / n,
// the residual x - q n is exact under a fused multiply-add, and one correction
// q + (x - q n) r rounded to nearest is RN(x / n) (Markstein's theorem for binary
// floating point with a correctly rounded reciprocal).  The theorem needs the
// residual and the quotient away from the subnormal range and 1/n normal; other
// operands (zeros included) take the IEEE division.
static __device__ __forceinline__ float div_rn(float x, float n, float r) {
  const float q = __fmul_rn(x, r);
  if (fabsf(x) >= 0x1p-100f && fabsf(q) >= 0x1p-124f && n <= 0x1p125f)
    return __fmaf_rn(__fmaf_rn(-q, n, x), r, q);
  return __fdiv_rn(x, n);
}

// Number of boundaries strictly below y (binary search over NB sorted boundaries).
template <int NB>
static __device__ __forceinline__ uint32_t bucket(float y, const float *sb) {
  uint32_t pos = 0;
#pragma unroll
  for (int step = (NB + 1) / 2; step >= 1; step >>= 1)
    if (y > sb[pos + step - 1]) pos += step;
  return pos;
}

// Four threads per row (a warp takes eight rows).  Thread q holds the four 8-element
// chunks 32i + 8q .. 32i + 8q + 7 (i = 0..3) in registers, so one load instruction reads
// 64 contiguous bytes of each row, the butterfly stages 1, 2, 4, 32, 64 and the norm
// tree's strides 16, 8, 1 run inside the thread, and only butterfly stages 8, 16 and tree
// strides 4, 2 cross threads (shuffles within the row's four lanes).  The operation order
// is the canonical one -- four-element partial sums of squares combined over strides
// 16, 8, 4, 2, 1; butterfly stages of distance 1, 2, ..., 64 with the lower element taking
// a + b and the upper a - b -- so every value is bit-identical to a sequential fp32
// implementation of the same order.  Register element 8i + e is row element 32i + 8q + e.
constexpr int WT_THREADS = 256;
constexpr int WT_E = 32;     // elements per thread
constexpr int WT_REP = 16;   // copies of the grid table (one per half-warp lane)

// A thread's four chunks as loaded (16-bit words or fp32), kept while the previous row is
// encoded.
template <int SRC>
struct Quarter {
  uint2 w[8];  // chunk i: w[2i], w[2i + 1] (eight 16-bit elements)
};
template <>
struct Quarter<TQ_DTYPE_F32> {
  float4 w[8];  // chunk i: w[2i], w[2i + 1]
};

// row: the row's first element; v16: 16-bit rows are 16-byte aligned (one 16-byte load per
// chunk); fp32 rows always are.
template <int SRC>
static __device__ __forceinline__ void load_quarter(const void *row, int q, bool v16, Quarter<SRC> &raw) {
  if constexpr (SRC == TQ_DTYPE_F32) {
    const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + 8 * q);
#pragma unroll
    for (int i = 0; i < 4; ++i) raw.w[2 * i] = s[8 * i], raw.w[2 * i + 1] = s[8 * i + 1];
  } else if (v16) {
    const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + 8 * q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 c = s[4 * i];
      raw.w[2 * i] = make_uint2(c.x, c.y), raw.w[2 * i + 1] = make_uint2(c.z, c.w);
    }
  } else {
    const uint2 *s = reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(row) + 8 * q);
#pragma unroll
    for (int i = 0; i < 4; ++i) raw.w[2 * i] = s[8 * i], raw.w[2 * i + 1] = s[8 * i + 1];
  }
}

static __device__ __forceinline__ void unpack_quarter(const Quarter<TQ_DTYPE_F32> &raw, float (&x)[WT_E]) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    x[4 * k] = raw.w[k].x, x[4 * k + 1] = raw.w[k].y, x[4 * k + 2] = raw.w[k].z, x[4 * k + 3] = raw.w[k].w;
}
static __device__ __forceinline__ void unpack_quarter(const Quarter<TQ_DTYPE_F16> &raw, float (&x)[WT_E]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&raw.w[k].x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&raw.w[k].y));
    x[4 * k] = a.x, x[4 * k + 1] = a.y, x[4 * k + 2] = b.x, x[4 * k + 3] = b.y;
  }
}
static __device__ __forceinline__ void unpack_quarter(const Quarter<TQ_DTYPE_BF16> &raw, float (&x)[WT_E]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[4 * k] = bf16_bits_to_f32(raw.w[k].x & 0xFFFFu), x[4 * k + 1] = bf16_bits_to_f32(raw.w[k].x >> 16);
    x[4 * k + 2] = bf16_bits_to_f32(raw.w[k].y & 0xFFFFu), x[4 * k + 3] = bf16_bits_to_f32(raw.w[k].y >> 16);
  }
}

// Canonical fp32 norm of the row (the four threads end with the same value), then u = x / n
// in place (u = 0 when n == 0).  Group g = 8i + 2q + h of the row is register group 2i + h.
static __device__ __forceinline__ float quarter_norm_normalize(float (&x)[WT_E]) {
  float p[8];  // four-element partial sums of register groups 2i + h
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const F2 a = f2(x[4 * k], x[4 * k + 1]), b = f2(x[4 * k + 2], x[4 * k + 3]);
    float a0, a1, b0, b1;
    f2_split(f2_mul(a, a), a0, a1);
    f2_split(f2_mul(b, b), b0, b1);
    p[k] = __fadd_rn(__fadd_rn(a0, a1), __fadd_rn(b0, b1));
  }
  float s[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // stride 16 (chunk i + 2) and stride 8 (chunk i + 1), in this thread
    const float s16a = __fadd_rn(p[h], p[4 + h]), s16b = __fadd_rn(p[2 + h], p[6 + h]);
    s[h] = __fadd_rn(s16a, s16b);
  }
  // stride 4: threads q and q ^ 2; stride 2: q and q ^ 1; stride 1: h = 0 and 1 here
#pragma unroll
  for (int h = 0; h < 2; ++h) s[h] = __fadd_rn(s[h], __shfl_xor_sync(FULL_MASK, s[h], 2));
#pragma unroll
  for (int h = 0; h < 2; ++h) s[h] = __fadd_rn(s[h], __shfl_xor_sync(FULL_MASK, s[h], 1));
  const float n = __fsqrt_rn(__fadd_rn(s[0], s[1]));
  const float r = __frcp_rn(n);
  // Markstein's correction is exact when every nonzero |x| >= 2^-100 and n <= 2^24 (then
  // |q| >= 2^-124 and 1/n is normal); zeros come out as zeros.  Otherwise (a row with a zero
  // among its elements asks again, element by element) the guarded per-element division.
  float mn = fabsf(x[0]);
#pragma unroll
  for (int j = 1; j < WT_E; ++j) mn = fminf(mn, fabsf(x[j]));
  bool fast = n <= 0x1p24f && mn >= 0x1p-100f;
  if (n <= 0x1p24f && !fast) {
    uint32_t mb = 0xFFFFFFFFu;  // min over elements of |x| bits - 1 (zero -> 0xFFFFFFFF)
#pragma unroll
    for (int j = 0; j < WT_E; ++j) mb = min(mb, (__float_as_uint(x[j]) & 0x7FFFFFFFu) - 1u);
    fast = mb >= 0x0D800000u - 1u;  // 0x0D800000: 2^-100
  }
  if (n == 0.0f) {
#pragma unroll
    for (int j = 0; j < WT_E; ++j) x[j] = 0.0f;
  } else if (fast) {
#pragma unroll
    for (int j = 0; j < WT_E; j += 2) {  // q + (x - q n) r; fma(q, -n, x) is fma(-q, n, x)
      const F2 xx = f2(x[j], x[j + 1]), rr = f2(r, r), qq = f2_mul(xx, rr);
      f2_split(f2_fma(f2_fma(qq, f2(-n, -n), xx), rr, qq), x[j], x[j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < WT_E; ++j) x[j] = div_rn(x[j], n, r);
  }
  return n;
}

// Randomized Hadamard of the row: sign flips (bit j % 32 of word j / 32 for row element j;
// nq[i] = sign word i shifted down by 8q), the butterfly, times RN(1/sqrt(128)).
static __device__ __forceinline__ void wht_quarter(float (&v)[WT_E], const uint32_t (&nq)[4], int q) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[8 * i + e] = __uint_as_float(__float_as_uint(v[8 * i + e]) ^ ((nq[i] << (31 - e)) & 0x80000000u));
  auto stage = [&](int h, int hr) {  // row distance h = register distance hr, in this thread
#pragma unroll
    for (int k = 0; k < WT_E; ++k)
      if (!(k & hr) && hr == 1) {
        const float a = v[k], b = v[k + hr];
        v[k] = __fadd_rn(a, b);
        v[k + hr] = __fsub_rn(a, b);
      } else if (!(k & hr) && !(k & 1)) {
        const F2 a = f2(v[k], v[k + 1]), b = f2(v[k + hr], v[k + hr + 1]);
        f2_split(f2_add(a, b), v[k], v[k + 1]);
        f2_split(f2_sub(a, b), v[k + hr], v[k + hr + 1]);
      }
    (void)h;
  };
  stage(1, 1);
  stage(2, 2);
  stage(4, 4);
  // distances 8 and 16: partner thread q ^ 1, then q ^ 2; the lower one keeps v + o, the
  // upper one o - v, both as one fused o + (+-1) v (the product by +-1 is exact)
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    const float sgn = (q & m) ? -1.0f : 1.0f;
#pragma unroll
    for (int k = 0; k < WT_E; k += 2) {
      const float o0 = __shfl_xor_sync(FULL_MASK, v[k], m), o1 = __shfl_xor_sync(FULL_MASK, v[k + 1], m);
      f2_split(f2_fma(f2(sgn, sgn), f2(v[k], v[k + 1]), f2(o0, o1)), v[k], v[k + 1]);
    }
  }
  stage(32, 8);
  stage(64, 16);
  const float inv_sqrt_d = __int_as_float(0x3DB504F3);  // fp32 nearest 1/sqrt(128)
#pragma unroll
  for (int k = 0; k < WT_E; k += 2)
    f2_split(f2_mul(f2(v[k], v[k + 1]), f2(inv_sqrt_d, inv_sqrt_d)), v[k], v[k + 1]);
}

// #{k : y > b_k}: the grid (copy l16 of cell t: boundary .x, count .y as integer bits) or,
// without GRID, binary search over the NB boundaries.
template <bool GRID, int NB>
static __device__ __forceinline__ uint32_t cell_index(float y, const float2 *ce, int l16, float gs, float go, int gn,
                                               const float *sb) {
  if (GRID) {
    // unsigned round-down conversion: negative, -inf and NaN give 0, +inf saturates
    const uint32_t t = min(__float2uint_rd(fmaf(y, gs, go)), (uint32_t)(gn - 1));
    const float2 c = ce[t * WT_REP + l16];
    return __float_as_uint(c.y) + (y > c.x ? 1u : 0u);
  }
  return bucket<NB>(y, sb);
}

// Nearest-centroid indices of this thread's elements, packed into its part of the row
// record at row (4-byte aligned).  turbo4 (fp32 norm + 64 nibble bytes): chunk i fills
// word 1 + 4i + q; thread 0 writes the norm.  turbo3 (four 14-byte blocks {fp16 norm,
// qs[8] with the low two index bits of block element j at bits 2 (j % 4) of qs[j / 4],
// signs[4] with the high bit at bit j % 8 of signs[j / 8]}): chunk i is elements
// 8q .. 8q+7 of block i, i.e. qs[2q], qs[2q + 1] and signs[q].
template <int FMT, bool GRID>
static __device__ __forceinline__ void pack_quarter(const float (&y)[WT_E], float n, const float2 *ce, int l16,
                                             float gs, float go, int gn, const float *sb, uint8_t *row,
                                             int q) {
  constexpr int NB = (FMT == TQ_FMT_TURBO4) ? 15 : 7;
  if (FMT == TQ_FMT_TURBO4) {
    uint32_t *w = reinterpret_cast<uint32_t *>(row);
    if (q == 0) w[0] = __float_as_uint(n);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t word = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) word |= cell_index<GRID, NB>(y[8 * i + e], ce, l16, gs, go, gn, sb) << (4 * e);
      w[1 + 4 * i + q] = word;
    }
  } else {
    const __half hn = __float2half_rn(n);
    const uint16_t nb = *reinterpret_cast<const uint16_t *>(&hn);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t idx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) idx[e] = cell_index<GRID, NB>(y[8 * i + e], ce, l16, gs, go, gn, sb);
      uint32_t lo = 0, sg = 0;  // qs[2q] | qs[2q + 1] << 8, signs[q]
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo |= (idx[e] & 3u) << (2 * e);
        sg |= (idx[e] >> 2) << e;
      }
      uint8_t *blk = row + 14 * i;  // 2-byte aligned
      if (q == 0) *reinterpret_cast<uint16_t *>(blk) = nb;
      *reinterpret_cast<uint16_t *>(blk + 2 + 2 * q) = (uint16_t)lo;
      blk[10 + q] = (uint8_t)sg;
    }
  }
}

// The WHT write's shared tables: the boundaries, the grid table (cell t, copy c at
// t * WT_REP + c: boundary .x, count .y as integer bits) and its scale, offset and size.
struct WhtTables {
  float sb[16];
  float2 ce[GRID_CELLS * WT_REP];
  float2 cell0[GRID_CELLS];  // one copy, read from memory
  float gs, go;
  int gn;
};

// Filled by every thread of the CTA (the caller synchronises again before use).
template <int FMT>
static __device__ __forceinline__ void wht_tables_fill(const float *b, const BucketTable *bt, WhtTables &tb) {
  constexpr int NB = (FMT == TQ_FMT_TURBO4) ? 15 : 7;
  if (threadIdx.x < NB) tb.sb[threadIdx.x] = b[threadIdx.x];
  // each cell read from memory once (one latency for the whole table), then copied with
  // consecutive threads on consecutive entries
  for (int t = threadIdx.x; t < GRID_CELLS; t += blockDim.x)
    tb.cell0[t] = make_float2(bt->e[t], __uint_as_float((uint32_t)bt->cnt[t]));
  if (threadIdx.x == 0) tb.gs = bt->scale, tb.go = bt->offset, tb.gn = bt->n;
  __syncthreads();
  for (int k = threadIdx.x; k < GRID_CELLS * WT_REP; k += blockDim.x) tb.ce[k] = tb.cell0[k / WT_REP];
}

}  // namespace tq
