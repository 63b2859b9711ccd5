// Device side of the paged cache's calls: where a batch row sits (sequence, position, page),
// the position rotation of a row held by a warp, and row conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

constexpr int PG_ROW = 68;  // bytes of a packed row

// The attention's weights are 2^W_SHIFT exp2(score - m), m the running maximum of score + log2(value
// norm) (norms below 2^-64 count as 2^-64), up to RESCALE_SLACK past it: from 2^-127 at the largest finite norm
// to 2^72 at none ahead of the shift, which leaves 23 octaves of smaller weights above exp2's flush
// at 2^-126, and 2^31 keys below 2^127.
constexpr int W_SHIFT = 24;
constexpr float W_MOST = 0x1p96f;         // 2^(64 + RESCALE_SLACK + W_SHIFT)
constexpr float NORM_FACTOR = 0x1p-17f;   // of a value norm, for a probability operand at 2^P_SHIFT: 2^(P_SHIFT - W_SHIFT)

// x 2^d, d <= 0, of a sum of weights when its maximum is raised: in two halves, since 2^d alone may be
// flushed (weights beside values of no norm, merged with values of norm 2^60) where the product is not.
static __device__ __forceinline__ float lower(float x, float half_factor) { return x * half_factor * half_factor; }
static __device__ __forceinline__ float lower_by(float x, float d) { return lower(x, exp2f(0.5f * d)); }

// Rows that belong to a sequence.
static __device__ __forceinline__ int paged_rows(const PagedView &v) {
  if (!v.cu_q) return v.B;
  const int n = v.cu_q[v.B];
  return n < 0 ? 0 : min(n, v.n_tokens);
}

// Length of sequence b, clamped to [0, max_len] (flagged by the thread with `flag`).
static __device__ __forceinline__ int paged_len(const PagedView &v, int b, bool flag) {
  const int n = v.seq_lens[b];
  if (n >= 0 && n <= v.max_len) return n;
  if (flag) atomicExch(v.status, (int32_t)DEVERR_SEQLEN);
  return n < 0 ? 0 : v.max_len;
}

// The sequence of row i: the largest b with cu_q[b] <= i (in [0, B) whatever cu_q holds).
static __device__ __forceinline__ int paged_seq(const PagedView &v, int i) {
  if (!v.cu_q) return i;
  int lo = 0, hi = v.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v.cu_q[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Position of row i of sequence b of n tokens; negative: the row has no place.
static __device__ __forceinline__ int paged_pos(const PagedView &v, int b, int i, int n) {
  return v.cu_q ? n - (v.cu_q[b + 1] - i) : n - 1;
}

// Page of position pos (< max_len) of sequence b, or -1 (flagged) for an id out of range.
static __device__ __forceinline__ int paged_page(const PagedView &v, int b, int pos, bool flag) {
  const int pg = v.table[(int64_t)b * v.table_stride + (pos >> v.page_shift)];
  if ((unsigned)pg < (unsigned)v.n_pages) return pg;
  if (flag) atomicExch(v.status, (int32_t)DEVERR_PAGE);
  return -1;
}

// Packed row of (page, KV head, row of the page).
static __device__ __forceinline__ size_t paged_row(const PagedView &v, int page, int h, int i) {
  return ((((size_t)page * v.Hkv + h) << v.page_shift) + i) * PG_ROW;
}

static __device__ __forceinline__ int rope_pos(const RopeView &r, int pos, int32_t *status, bool flag) {
  if (pos < r.n_pos) return max(pos, 0);
  if (flag) atomicExch(status, (int32_t)DEVERR_ROPE);
  return r.n_pos - 1;
}

// (a, b) -> (a c - b s, a s + b c), every operation rounded once.
static __device__ __forceinline__ float rot_first(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
static __device__ __forceinline__ float rot_second(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
}

// Elements 4l .. 4l + 3 of a row: as loaded, and as fp32.
static __device__ __forceinline__ uint4 load_lane4_raw(const uint8_t *row, int dtype, int lane) {
  if (dtype == TQ_DTYPE_F32) return reinterpret_cast<const uint4 *>(row)[lane];
  const uint2 v = reinterpret_cast<const uint2 *>(row)[lane];
  return make_uint4(v.x, v.y, 0u, 0u);
}
static __device__ __forceinline__ void lane4_floats(const uint4 &v, int dtype, float (&x)[4]) {
  if (dtype == TQ_DTYPE_F32) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  } else {
    if (dtype == TQ_DTYPE_BF16) {
      x[0] = bf16_bits_to_f32(v.x & 0xFFFFu), x[1] = bf16_bits_to_f32(v.x >> 16);
      x[2] = bf16_bits_to_f32(v.y & 0xFFFFu), x[3] = bf16_bits_to_f32(v.y >> 16);
    } else {
      const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x));
      const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
      x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    }
  }
}
static __device__ __forceinline__ void load_lane4(const uint8_t *row, int dtype, int lane, float (&x)[4]) {
  lane4_floats(load_lane4_raw(row, dtype, lane), dtype, x);
}

// Angles of a row's elements 4l .. 4l + 3 (lane l), loaded ahead of the row they turn.
struct LaneAngles {
  float4 c, s;  // interleaved: two pairs, in .x and .y
};
static __device__ __forceinline__ LaneAngles rope_angles(int lane, const RopeView &r, int pos) {
  LaneAngles a;
  a.c = make_float4(1.f, 1.f, 1.f, 1.f), a.s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (4 * lane >= r.rot_dim) return a;
  const int half = r.rot_dim >> 1;
  const float *ct = r.cos_t + (size_t)pos * half, *st = r.sin_t + (size_t)pos * half;
  if (r.interleaved) {
    const float2 c = reinterpret_cast<const float2 *>(ct)[lane], z = reinterpret_cast<const float2 *>(st)[lane];
    a.c.x = c.x, a.c.y = c.y, a.s.x = z.x, a.s.y = z.y;
  } else {
    const int at = lane & ((r.rot_dim >> 3) - 1);
    a.c = reinterpret_cast<const float4 *>(ct)[at], a.s = reinterpret_cast<const float4 *>(st)[at];
  }
  return a;
}

// Position rotation of a row held as elements 4l .. 4l + 3 of lane l (the whole warp calls).
static __device__ __forceinline__ void rope_turn(float (&x)[4], int lane, const RopeView &r, const LaneAngles &an) {
  const bool act = 4 * lane < r.rot_dim;
  if (r.interleaved) {
    if (act) {
      const float a = x[0], b = x[1], e = x[2], f = x[3];
      x[0] = rot_first(a, b, an.c.x, an.s.x), x[1] = rot_second(a, b, an.c.x, an.s.x);
      x[2] = rot_first(e, f, an.c.y, an.s.y), x[3] = rot_second(e, f, an.c.y, an.s.y);
    }
    return;
  }
  const int m = r.rot_dim >> 3;  // lanes of a half
  float o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = __shfl_xor_sync(FULL_MASK, x[e], m);
  if (act) {
    const float cc[4] = {an.c.x, an.c.y, an.c.z, an.c.w}, ss[4] = {an.s.x, an.s.y, an.s.z, an.s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = (lane & m) ? rot_second(o[e], x[e], cc[e], ss[e]) : rot_first(x[e], o[e], cc[e], ss[e]);
  }
}
static __device__ __forceinline__ void rope_lane4(float (&x)[4], int lane, const RopeView &r, int pos) {
  if (r.rot_dim) rope_turn(x, lane, r, rope_angles(lane, r, pos));
}

// The exponent whose power of two brings amax down (or up) to [2^13, 2^14), fp16's upper end with a
// bit to spare; 0 for a row of zeros, infinity or NaN.  In [-126, 114]: a row below 2^-113 is
// brought up by 2^126 only, so that the power and its inverse are normal numbers.
static __device__ __forceinline__ int scale_exp(float amax) {
  const int eb = __float_as_int(amax) >> 23;
  return amax > 0.f && eb < 255 ? max(eb - 127, -113) - 13 : 0;
}
static __device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }  // |e| <= 126

static __device__ __forceinline__ uint32_t pack_bf162(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Elements 4l .. 4l + 3 of a dense output row of `dtype` starting at element `at`.
static __device__ __forceinline__ void store_lane4(void *out, int dtype, size_t at, int lane, const float (&x)[4]) {
  if (dtype == TQ_DTYPE_F32)
    reinterpret_cast<float4 *>(static_cast<float *>(out) + at)[lane] = make_float4(x[0], x[1], x[2], x[3]);
  else if (dtype == TQ_DTYPE_BF16)
    reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at)[lane] =
        make_uint2(pack_bf162(x[0], x[1]), pack_bf162(x[2], x[3]));
  else
    reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at)[lane] =
        make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
}

// out_scale * rsqrt(mean(d^2) + eps) of a pair's ss = sum d^2.  All zero (a row without keys) stays zero
// whatever eps is, NaN stays, and a mean below fp32's normal numbers counts as the least of them: the
// factor, and with it the row, stays finite.
static __device__ __forceinline__ float diff_factor(float ss, const DiffView &d) {
  const float m = fmaf(ss, 1.0f / D, d.eps);
  return ss == 0.f ? 0.f : d.out_scale * rsqrtf(m < 0x1p-126f ? 0x1p-126f : m);
}

// The end of a differential pair: a = out_scale * d [* rsqrt(mean(d^2) + eps) * gain],
// d = a - lambda b, elements 4l .. 4l + 3 of lane l (the whole warp calls).
static __device__ __forceinline__ void diff_finish(float (&a)[4], const float (&b)[4], const DiffView &d, int row,
                                                   int pair, int lane) {
  const float lam = d.lambda[(int64_t)row * d.lambda_stride + pair];
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    a[e] = fmaf(-lam, b[e], a[e]);
    ss = fmaf(a[e], a[e], ss);
  }
  float f = d.out_scale;
  float4 g = make_float4(1.f, 1.f, 1.f, 1.f);
  if (d.gain) {
#pragma unroll
    for (int h = 16; h >= 1; h >>= 1) ss += __shfl_xor_sync(FULL_MASK, ss, h);
    f = diff_factor(ss, d);
    g = reinterpret_cast<const float4 *>(d.gain)[lane];
  }
  a[0] *= f * g.x, a[1] *= f * g.y, a[2] *= f * g.z, a[3] *= f * g.w;
}

// floor(x m / d), in 32 bits where the product fits.
static __device__ __forceinline__ int mul_div(uint32_t x, uint32_t m, uint32_t d) {
  const uint64_t p = (uint64_t)x * m;
  return (p >> 32) ? (int)(p / d) : (int)((uint32_t)p / d);
}
// Equal shares of V virtual tiles over G CTAs: CTA c takes [floor(c V / G), floor((c + 1) V / G)).
static __device__ __forceinline__ int share_start(int c, int V, int G) { return mul_div(c, V, G); }
// The CTA whose share holds virtual tile v: the largest c with floor(c V / G) <= v.
static __device__ __forceinline__ int share_of(int v, int V, int G) {
  const uint64_t p = (uint64_t)(uint32_t)(v + 1) * (uint32_t)G - 1;
  return (p >> 32) ? (int)(p / (uint32_t)V) : (int)((uint32_t)p / (uint32_t)V);
}

}  // namespace tq
