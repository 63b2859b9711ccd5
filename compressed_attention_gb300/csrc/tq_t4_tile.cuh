// Operand decoding of the turbo4 split-K decode kernels: 4-bit indices to fp16x2 centroid
// pairs through a conflict-free shared-memory table, the probability operand, and the order
// of a 16-key block's rows.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "tq_device.cuh"

namespace tq {

// Table lookup of byte I of w.  FIXED: the table is at window address LUT_WINDOW and
// the load carries it as an immediate; otherwise the table's address is added.
template <bool FIXED, int I>
static __device__ __forceinline__ uint32_t lut_byte(uint32_t lut_addr, uint32_t laneword, uint32_t w) {
  const uint32_t off = prmt(laneword, w, 0x1100u | ((4u + I) << 4));
  uint32_t v;
  if (FIXED)
    asm("ld.shared.u32 %0, [%1+65536];" : "=r"(v) : "r"(off));
  else
    asm("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(off + lut_addr));
  return v;
}

// Four bytes of w -> four fp16x2 words, from the table or by byte permutes.
template <bool PRMT, bool FIXED>
static __device__ __forceinline__ void decode4(uint32_t lut_addr, uint32_t laneword, uint32_t w,
                                        const uint32_t (&lo)[2], const uint32_t (&hi)[2],
                                        uint32_t (&r)[4]) {
  if (PRMT) {
    decode8<0x5140u, 0x7362u>(w, lo, hi, r);
  } else {
    r[0] = lut_byte<FIXED, 0>(lut_addr, laneword, w);
    r[1] = lut_byte<FIXED, 1>(lut_addr, laneword, w);
    r[2] = lut_byte<FIXED, 2>(lut_addr, laneword, w);
    r[3] = lut_byte<FIXED, 3>(lut_addr, laneword, w);
  }
}

static __device__ __forceinline__ uint32_t ld_u32(const uint8_t *p) {
  return *reinterpret_cast<const uint32_t *>(p);
}

// The PV B operand of one column group from the probabilities of this lane's two score
// rows: column g takes head g/2, its fp16 hi (g even) or lo (g odd) part, for the keys
// a_t, a_t+2 (k 2t, 2t+1) and a_t+4, a_t+6 (k 2t+8, 2t+9), gathered from the lanes that
// own those keys' scores.
static __device__ __forceinline__ void p_operand(float pp0, float pp1, int src0, int src1, float lo_sel,
                                          uint32_t (&pb)[2]) {
  const float va = __shfl_sync(FULL_MASK, pp0, src0), vb = __shfl_sync(FULL_MASK, pp0, src1);
  const float vc = __shfl_sync(FULL_MASK, pp1, src0), vd = __shfl_sync(FULL_MASK, pp1, src1);
  const __half2 hab = __floats2half2_rn(va, vb), hcd = __floats2half2_rn(vc, vd);
  const float2 fab = __half22float2(hab), fcd = __half22float2(hcd);
  const __half2 rab = __floats2half2_rn(fmaf(-lo_sel, fab.x, va), fmaf(-lo_sel, fab.y, vb));
  const __half2 rcd = __floats2half2_rn(fmaf(-lo_sel, fcd.x, vc), fmaf(-lo_sel, fcd.y, vd));
  pb[0] = *reinterpret_cast<const uint32_t *>(&rab);
  pb[1] = *reinterpret_cast<const uint32_t *>(&rcd);
}

// Physical key (within a 16-key block) of score row r.  Rows g and g+8 belong to
// lane group g.  With this order the packed-word loads of a warp hit every bank at
// most twice, and the PV operand of lane (g, t) -- keys a_t, a_t+2, a_t+4, a_t+6
// with a_t = {0, 1, 8, 9}[t] -- comes from score rows t, 4+t, 8+t, 12+t, i.e. from
// the same register of lanes 4t+h and 4(4+t)+h.
static __device__ __forceinline__ int key_of_row(int r) {
  // rows 0..7: 0 1 8 9 2 3 10 11; rows 8..15: 4 5 12 13 6 7 14 15
  return ((r & 1) | ((r & 2) << 2) | ((r & 4) >> 1) | ((r & 8) >> 1));
}

}  // namespace tq
