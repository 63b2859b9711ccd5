// Read rows back from the paged cache as dense rows: x = norm * R^T c[idx].
//
// k_paged_gather_tc  Tiles of 128 output rows (token-major, so a tile's output is one
//     contiguous range), a warpgroup per tile, two to four of them sharing R in shared
//     memory.  A tile's packed rows come in as 4-byte asynchronous copies spread over the
//     warp (17 lanes a row), a thread decodes its row into a swizzled fp16 operand tile,
//     C R runs on the 5th-generation tensor cores with R as the MN-major B operand (one
//     512-cycle product where a butterfly or a matvec would take 1,000 to 32,000
//     operations a row), and the accumulator lanes are scaled by norm / alpha, rounded and
//     stored through a swizzled staging tile, whole lines at a time.  Both rotation kinds
//     take the same path.  Parts: bf16 outputs take fp16 centroids and one fp16 part of R
//     (errors of 2^-11 at most against a half step of 2^-8), fp16 outputs R in hi + lo, fp32
//     outputs both in hi + lo (three products, 2^-22).  122 MB of bf16 rows from 33 MB of
//     records: 43 us (49 with a search for each row's sequence, 44.9 with its page found a tile
//     earlier), bound by the latency of the row copies and of the staging.
//     13.8K tokens of 8 KV heads, keys and values: 26 us in bf16, 27 in fp16, 45 in fp32.
// k_paged_gather     the rotated basis (no product): a warp per row; the same rows 35 us.
#include "tq_paged.cuh"
#include "tq_qprep.cuh"
#include "tq_tc.cuh"

namespace tq {

namespace {

struct GatherSide {
  const uint8_t *pages;
  void *out;
  float c[16];              // centroids
  uint32_t lo[2], hi[2];    // byte planes of the fp16 magnitudes alpha * |c|
  float inv_alpha;
  const uint8_t *rtile;     // R as fp16 hi, lo tile images
};
struct GatherParams {
  PagedView pv;
  GatherSide side[2];
  int dtype;
  int only;  // 0 or 1: one side; 2: both, alternating CTAs
};

// The sequence of a thread's last row, [lo, hi) its rows: the next row is mostly of the same one, and
// then costs one load (its page), not the search's chain of them.
struct SeqOf {
  int b = 0, lo = 0, hi = 0, n = 0;
};
// The packed row of output row `row` (token-major), -1 without one.
__device__ __forceinline__ int64_t source_row(const PagedView &v, SeqOf &s, int64_t row, bool flag) {
  const int tok = (int)((uint32_t)row / (uint32_t)v.Hkv), h = (int)(row - (int64_t)tok * v.Hkv);
  if (tok < s.lo || tok >= s.hi) {
    s.b = paged_seq(v, tok);
    s.lo = v.cu_q ? v.cu_q[s.b] : tok, s.hi = v.cu_q ? v.cu_q[s.b + 1] : tok + 1;
    s.n = paged_len(v, s.b, flag);
  }
  const int pos = s.n - (s.hi - tok);
  if (pos < 0 || pos >= s.n) return -1;
  return (int64_t)paged_row(v, max(paged_page(v, s.b, pos, flag), 0), h, pos & ((1 << v.page_shift) - 1));
}

constexpr int RAW = 128 * PG_ROW;

// PARTS: 1 (C R_hi), 2 (C R_hi + C R_lo), 3 (and C_lo R_hi).
template <int PARTS>
struct GatherCfg {
  static constexpr int GROUPS = PARTS == 1 ? 4 : (PARTS == 2 ? 3 : 2);
  static constexpr uint32_t R_BYTES = (PARTS == 1 ? 1 : 2) * SW_TILE_BYTES;
  static constexpr uint32_t A_BYTES = (PARTS == 3 ? 2 : 1) * SW_TILE_BYTES;
  static constexpr uint32_t OFF_A = R_BYTES, OFF_RAW = OFF_A + GROUPS * A_BYTES;
  static constexpr uint32_t OFF_MISC = OFF_RAW + GROUPS * RAW;
  static constexpr uint32_t SMEM = OFF_MISC + 256 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

template <int PARTS>
__global__ void __launch_bounds__(GatherCfg<PARTS>::GROUPS * 128) k_paged_gather_tc(const GatherParams p) {
  using C = GatherCfg<PARTS>;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t *smem = smem_dyn + ((1024u - (smem_addr(smem_dyn) & 1023u)) & 1023u);
  uint64_t *r_full = reinterpret_cast<uint64_t *>(smem + C::OFF_MISC), *done = r_full + 1;
  uint32_t *tmem_at = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC + 64);
  uint32_t *lut = tmem_at + 16;  // PARTS 3: fp16 hi | lo << 16 of alpha * c
  const int side = p.only == 2 ? (blockIdx.x & 1) : p.only, n_side = p.only == 2 ? 2 : 1;
  const GatherSide &sd = p.side[side];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = warp >> 2, r = tid & 127;
  pdl_trigger();
  if (warp == 0) tmem_alloc(smem_addr(tmem_at), 512);
  if (tid == 0) {
    mbar_init(r_full, 1);
    for (int i = 0; i < C::GROUPS; ++i) mbar_init(&done[i], 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(r_full, C::R_BYTES);  // R belongs to the context: before the wait
    bulk_g2s(smem, sd.rtile, C::R_BYTES, r_full);
  }
  if (PARTS == 3 && tid < 16) {
    const float a = 1.0f / sd.inv_alpha, x = sd.c[tid] * a;
    const __half h = __float2half_rn(x), l = __float2half_rn(x - __half2float(h));
    lut[tid] = (uint32_t)__half_as_ushort(h) | ((uint32_t)__half_as_ushort(l) << 16);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tm = *tmem_at + 128 * grp, lane_off = (uint32_t)((warp & 3) * 32) << 16;
  uint8_t *at = smem + C::OFF_A + grp * C::A_BYTES;
  uint32_t *raw = reinterpret_cast<uint32_t *>(smem + C::OFF_RAW + grp * RAW);
  const uint32_t clo[2] = {sd.lo[0], sd.lo[1]}, chi[2] = {sd.hi[0], sd.hi[1]};
  auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory"); };
  const int64_t n_rows = (int64_t)paged_rows(p.pv) * p.pv.Hkv, n_tiles = (n_rows + 127) / 128;
  const int n_cta = gridDim.x / n_side;
  // this warp's 32 packed rows of tile t: lane l copies words l, l + 32, ... of the 32 x 17
  int64_t src = -1;
  SeqOf seq;
  auto fetch = [&](int64_t t) {
    const int64_t row = t * 128 + r;
    src = t < n_tiles && row < n_rows ? source_row(p.pv, seq, row, true) : -1;
    uint32_t *dst = raw + (warp & 3) * 32 * 17;
#pragma unroll
    for (int k = 0; k < 17; ++k) {
      const int idx = 32 * k + lane, rr = idx / 17;
      const int64_t o = __shfl_sync(FULL_MASK, src, rr);
      if (o >= 0)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst + idx)),
                     "l"(sd.pages + o + 4 * (idx - 17 * rr))
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int64_t t = (int64_t)grp * n_cta + blockIdx.x / n_side;
  const int64_t step = (int64_t)n_cta * C::GROUPS;
  uint32_t phase = 0;
  bool r_ok = false, ok = true;
  fetch(t);
  for (; t < n_tiles; t += step) {
    const bool have = src >= 0;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();  // a warp decodes the rows that it copied
    const uint32_t *w = raw + r * 17;
    const float norm = have ? __uint_as_float(w[0]) * sd.inv_alpha : 0.f;
#pragma unroll
    for (int ch = 0; ch < 16; ++ch) {
      const uint32_t x = w[1 + ch];  // stale words of a row without a source: finite centroids times 0
      if (PARTS < 3) {
        uint32_t d[4];
        decode8<0x5140u, 0x7362u>(x, clo, chi, d);
        *reinterpret_cast<uint4 *>(at + sw128_offset(r, 8 * ch)) = make_uint4(d[0], d[1], d[2], d[3]);
      } else {
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a = lut[(x >> (8 * e)) & 15u], b = lut[(x >> (8 * e + 4)) & 15u];
          h[e] = prmt(a, b, 0x5410u), l[e] = prmt(a, b, 0x7632u);
        }
        *reinterpret_cast<uint4 *>(at + sw128_offset(r, 8 * ch)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(at + SW_TILE_BYTES + sw128_offset(r, 8 * ch)) = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
    __syncwarp();
    fetch(t + step);  // under the product and the stores
    fence_async_smem();
    tc_fence_before();
    group_sync();
    if ((warp & 3) == 0) {
      tc_fence_after();
      if (!r_ok) ok = mbar_wait_bounded(r_full, 0, 2000000000ull), r_ok = true;
      ok = __all_sync(FULL_MASK, ok);
      const uint64_t da = sw128_desc(smem_addr(at)), dr = sw128_mn_desc(smem_addr(smem));
      if (ok && elect_lane()) {
#pragma unroll
        for (int part = 0; part < PARTS; ++part)  // C R_hi, C R_lo, C_lo R_hi
#pragma unroll
          for (int s = 0; s < 8; ++s)
            umma<IDESC_F16_BMN>(tm, desc_step(da, (part == 2 ? SW_TILE_BYTES : 0) + sw128_kstep(s)),
                                desc_step(dr, (part == 1 ? SW_TILE_BYTES : 0) + 2048 * s), (part || s) ? 1u : 0u);
        umma_commit(&done[grp]);
      }
      __syncwarp();
    }
    bool up = mbar_wait_bounded(&done[grp], phase & 1, 4000000000ull);
    ++phase;
    up = __all_sync(FULL_MASK, up);
    if (!up) {  // only after R's copy never landed: no product is in flight
      if (lane == 0) atomicExch(p.pv.status, (int32_t)DEVERR_TIMEOUT);
      break;
    }
    tc_fence_after();
    // columns in halves of 256 bytes a row, staged over the operand tile (its products are done)
    constexpr int ESZ = PARTS == 3 ? 4 : 2, COLS = 256 / ESZ;
    const int64_t row0 = t * 128;
    const int rows = (int)min((int64_t)128, n_rows - row0);
#pragma unroll 1
    for (int half = 0; half < D / COLS; ++half) {
#pragma unroll 1
      for (int c0 = 0; c0 < COLS; c0 += 32) {
        float v[32];
        tmem_ld32(tm + lane_off + half * COLS + c0, v);
        if constexpr (PARTS == 3) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int ch = c0 / 4 + c;
            *reinterpret_cast<float4 *>(at + r * 256 + ((ch ^ (r & 7)) << 4)) =
                make_float4(v[4 * c] * norm, v[4 * c + 1] * norm, v[4 * c + 2] * norm, v[4 * c + 3] * norm);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int ch = c0 / 8 + c;
            uint32_t x[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float a = v[8 * c + 2 * m] * norm, b = v[8 * c + 2 * m + 1] * norm;
              x[m] = PARTS == 1 ? pack_bf162(a, b) : pack_half2(a, b);
            }
            *reinterpret_cast<uint4 *>(at + r * 256 + ((ch ^ (r & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      }
      __syncwarp();  // a warp stores the rows that it staged
      uint8_t *out = static_cast<uint8_t *>(sd.out) + (row0 + (warp & 3) * 32) * (D * ESZ) + half * 256;
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int rr = 2 * i + (lane >> 4), ch = lane & 15, gr = (warp & 3) * 32 + rr;
        if (gr < rows)
          *reinterpret_cast<uint4 *>(out + (size_t)rr * (D * ESZ) + 16 * ch) =
              *reinterpret_cast<const uint4 *>(at + gr * 256 + ((ch ^ (gr & 7)) << 4));
      }
      __syncwarp();
    }
    tc_fence_before();
    group_sync();  // the group's accumulator and operand tile are free again
    tc_fence_after();
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (tid == 0 && !r_ok) (void)mbar_wait_bounded(r_full, 0, 2000000000ull);  // R's copy must land before the CTA ends
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(*tmem_at, 512);
}

// Rotated basis: a warp per row, lane l elements 4l .. 4l + 3.
constexpr int GA_WARPS = 8;
__global__ void __launch_bounds__(GA_WARPS * 32) k_paged_gather(const GatherParams p) {
  __shared__ float ct[16];
  const int side = p.only == 2 ? (blockIdx.x & 1) : p.only, step = p.only == 2 ? 2 : 1;
  const GatherSide &sd = p.side[side];
  pdl_trigger();
  if (threadIdx.x < 16) ct[threadIdx.x] = sd.c[threadIdx.x];
  __syncthreads();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n_rows = (int64_t)paged_rows(p.pv) * p.pv.Hkv;
  const int n_cta = gridDim.x / step;
  SeqOf seq;
  for (int64_t row = (int64_t)(blockIdx.x / step) * GA_WARPS + warp; row < n_rows; row += (int64_t)n_cta * GA_WARPS) {
    const int64_t at = source_row(p.pv, seq, row, lane == 0);
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (at >= 0) {
      const float norm = *reinterpret_cast<const float *>(sd.pages + at);
      const uint32_t w = *reinterpret_cast<const uint16_t *>(sd.pages + at + 4 + 2 * lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = norm * ct[(w >> (4 * e)) & 15u];
    }
    store_lane4(sd.out, p.dtype, (size_t)row * D, lane, x);
  }
}

template <int PARTS>
cudaError_t launch_tc(const GatherParams &p, int sms, cudaStream_t st) {
  using C = GatherCfg<PARTS>;
  cudaError_t e = kernel_smem_attr((const void *)k_paged_gather_tc<PARTS>, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  const int sides = p.only == 2 ? 2 : 1;
  const int64_t tiles = ((int64_t)p.pv.n_tokens * p.pv.Hkv + 127) / 128, most = sms / sides > 0 ? sms / sides : 1;
  return launch_pdl(k_paged_gather_tc<PARTS>, dim3(sides * (unsigned)(tiles < most ? tiles : most)),
                    dim3(C::GROUPS * 128), C::SMEM, st, p);
}

}  // namespace

cudaError_t launch_paged_gather(const tq_ctx *k, const tq_ctx *v, const PagedView &pv, const uint8_t *kp,
                                const uint8_t *vp, int unrotate, void *k_out, void *v_out, int out_dtype,
                                cudaStream_t st) {
  GatherParams p{};
  p.pv = pv;
  p.dtype = out_dtype;
  p.only = k_out && v_out ? 2 : (k_out ? 0 : 1);
  const tq_ctx *ctx[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    GatherSide &s = p.side[i];
    s.pages = i ? vp : kp;
    s.out = i ? v_out : k_out;
    for (int j = 0; j < 16; ++j) s.c[j] = ctx[i]->cb.c[j];
    for (int j = 0; j < 2; ++j) s.lo[j] = ctx[i]->f16.lo[j], s.hi[j] = ctx[i]->f16.hi[j];
    s.inv_alpha = 1.0f / ctx[i]->f16.alpha;
    s.rtile = reinterpret_cast<const uint8_t *>(ctx[i]->d_rtile);
  }
  if (unrotate) {
    if (out_dtype == TQ_DTYPE_BF16) return launch_tc<1>(p, k->num_sms, st);
    return out_dtype == TQ_DTYPE_F16 ? launch_tc<2>(p, k->num_sms, st) : launch_tc<3>(p, k->num_sms, st);
  }
  int blocks = 1;
  const cudaError_t e = kernel_occupancy((const void *)k_paged_gather, GA_WARPS * 32, 0, &blocks);
  if (e != cudaSuccess) return e;
  const int sides = p.only == 2 ? 2 : 1;
  const int64_t want = ((int64_t)pv.n_tokens * pv.Hkv + GA_WARPS - 1) / GA_WARPS;
  const int64_t most = (int64_t)k->num_sms * blocks / sides;
  return launch_pdl(k_paged_gather, dim3(sides * (unsigned)(want < most ? want : most)), dim3(GA_WARPS * 32), 0, st, p);
}

}  // namespace tq
