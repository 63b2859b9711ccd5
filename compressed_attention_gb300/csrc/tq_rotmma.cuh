// The rotation of up to eight vectors by one CTA on the tensor cores: Y = M X for
// M = R or R^T (128 x 128) and X of eight columns, as m16n8k16 products of bf16 parts,
// M_hi X_hi + M_hi X_lo + M_lo X_hi (fp32 sums).  The dropped parts are below 2^-16 of
// |M||x| per product, under the fp16 rounding of the operands the results become.
// M comes from the context in fragment order (tq_ctx::d_rfrag), so a lane's share of one
// 16-row tile is eight consecutive-lane 16-byte loads per part, all in flight at once: one
// L2 latency for the 64 KB, where rows staged in shared memory would need them twice.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

constexpr int ROT_PITCH = D + 8;  // bf16 elements between columns of X (bank spread)

struct RotColumns {
  alignas(16) uint16_t hi[8][ROT_PITCH];
  alignas(16) uint16_t lo[8][ROT_PITCH];
};

// Elements 4l .. 4l + 3 of column h from lane l.
static __device__ __forceinline__ void rot_put(RotColumns &x, int h, int lane, const float (&v)[4]) {
  uint32_t hi[2], lo[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    const float2 af = __bfloat1622float2(a);
    // an infinite element keeps a zero low part (inf - inf would turn it into NaN)
    const __nv_bfloat162 b = __floats2bfloat162_rn(isinf(af.x) ? 0.f : v[2 * i] - af.x,
                                                   isinf(af.y) ? 0.f : v[2 * i + 1] - af.y);
    hi[i] = *reinterpret_cast<const uint32_t *>(&a);
    lo[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  *reinterpret_cast<uint2 *>(&x.hi[h][4 * lane]) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2 *>(&x.lo[h][4 * lane]) = make_uint2(lo[0], lo[1]);
}

// One part (0 hi, 1 lo) of the 16-row tile mt of matrix m (0: R, 1: R^T).
static __device__ __forceinline__ void rot_load(uint4 (&a)[8], const uint4 *frag, int m, int part, int mt, int lane) {
  const uint4 *src = frag + ((size_t)((2 * m + part) * 8 + mt) * 8) * 32 + lane;
#pragma unroll
  for (int s = 0; s < 8; ++s) a[s] = __ldg(src + 32 * s);
}

static __device__ __forceinline__ void mma_bf16(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// The A operand of 16 rows by 16 elements; lane l gives the address of row l % 16, half l / 16.
static __device__ __forceinline__ uint4 ldmatrix_x4(const void *row) {
  uint4 r;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"((uint32_t)__cvta_generic_to_shared(row))
               : "memory");
  return r;
}

// acc += A (X_hi [+ X_lo]): rows g, g + 8 of the tile, columns 2t, 2t + 1 (lane 4g + t).
template <bool LO>
static __device__ __forceinline__ void rot_mul(float (&acc)[4], const uint4 (&a)[8], const RotColumns &x, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const uint32_t *h = reinterpret_cast<const uint32_t *>(&x.hi[g][16 * s + 2 * t]);
    mma_bf16(acc, a[s], h[0], h[4]);
    if (LO) {
      const uint32_t *l = reinterpret_cast<const uint32_t *>(&x.lo[g][16 * s + 2 * t]);
      mma_bf16(acc, a[s], l[0], l[4]);
    }
  }
}

// Row-tile mt of Y = M X, from its loaded parts, into y[column][16 mt ..] (rows of `pitch` floats).
static __device__ __forceinline__ void rot_tile(const uint4 (&hi)[8], const uint4 (&lo)[8], int mt, int lane,
                                                const RotColumns &x, float *y, int pitch) {
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
  rot_mul<true>(acc, hi, x, lane);
  rot_mul<false>(acc2, lo, x, lane);
  const int g = lane >> 2, t = lane & 3;
  float *d = y + 2 * t * pitch + 16 * mt + g;
  d[0] = acc[0] + acc2[0], d[pitch] = acc[1] + acc2[1];
  d[8] = acc[2] + acc2[2], d[pitch + 8] = acc[3] + acc2[3];
}

}  // namespace tq
