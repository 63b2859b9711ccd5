// Append to the paged cache.
//
// k_paged_append_wht: SET_ROWS through the block table with the keys' position
// rotation applied on the way.  The row's encode is the write path's (tq_wht.cuh): four
// threads per row, eight rows per warp, the canonical order of norm, division and
// butterfly, so the stored bytes equal those of a plain fp32 sequence.  The rotation's
// pairs (j, j + 64) and (j, j + 32) and adjacent pairs lie inside one thread's chunks;
// pairs (j, j + 16) cross to the thread two over.  A CTA takes keys or values, so it keeps one
// codebook grid.  The next row's elements and page id are in flight under a row's encode.  13.8K
// tokens of 8 KV heads (bf16, keys turned): 40 us for 79 MB, 129 warp instructions a row; issue and
// latency at 16 warps an SM bind it (128 registers; 24 warps at 80 spilled and were slower).
#include "tq_decode_common.cuh"
#include "tq_paged.cuh"
#include "tq_qprep.cuh"
#include "tq_rotmma.cuh"
#include "tq_wht.cuh"

namespace tq {

namespace {

struct AppendSide {
  RowsView src;
  uint8_t *pages;
  uint32_t wht_neg[4];
  float b[15];
  const BucketTable *bt;
  const uint4 *rfrag;  // dense: R as bf16 hi + lo fragments
  const float *pit;    // dense: R^T, fp32
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
  // the next row: its page as in the table (loaded, and looked at when its turn comes), head and position
  int nx_page = -1, nx_head = 0, nx_pos = -1;
  auto fetch = [&](int i) {
    nx_pos = -1;
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
      const int pos = len - (b_end - tok);
      if (pos >= 0 && pos < len) {
        nx_page = p.pv.table[(int64_t)b * p.pv.table_stride + (pos >> p.pv.page_shift)];
        nx_pos = pos, nx_head = head;
      }
      tok += d_tok, head += d_head;
      if (head >= Hkv) head -= Hkv, ++tok;
    }
  };
  fetch(it);
  for (; it < n_iter; it += step) {
    Place at{-1, nx_pos};
    if (nx_pos >= 0) {
      if ((unsigned)nx_page < (unsigned)p.pv.n_pages)
        at.at = (int64_t)paged_row(p.pv, nx_page, nx_head, nx_pos & ((1 << p.pv.page_shift) - 1));
      else if (q == 0) atomicExch(p.pv.status, (int32_t)DEVERR_PAGE);
    }
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

// Dense rotation on the tensor cores: each warp takes tiles of 16 rows by itself.  Rows are loaded
// and turned by position as in q's preparation, normalised, split into bf16 parts in the warp's
// shared memory and multiplied by R (fragments of its parts, 64 KB per CTA from one bulk copy).
// y = R u, |u| = 1, in four products of parts: what the parts drop of u and of R is at most 2^-18
// of |u| |row of R| each, 7.6e-6 together with the sums' rounding below the 1e-5 within which an
// index may differ; three products (without lo lo) could reach 1.2e-5.  Lane (g, t) holds columns
// 8 j + 2 t and the next of rows g and g + 8, one byte of nibbles of word j: the four lanes of a row
// transpose their bytes and store words.  13.8K tokens of 8 KV heads, keys and values: 112 us; a
// warp per row on the CUDA cores took 560 us.
constexpr int AD_WARPS = 16;
struct DenseSmem {
  uint4 r[2][8][8][32];            // R, bf16 hi and lo
  uint16_t xs[AD_WARPS][2][16][D]; // a warp's rows, bf16 hi and lo; 16-byte chunk c of row r at c ^ (r % 8)
  WhtTables tb;
  uint64_t full;
};

static_assert(sizeof(DenseSmem) <= 227 * 1024, "shared memory budget");

// Four lanes' words of bytes transposed: byte u of lane t's result is byte t of lane u's word.
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t v, int t) {
  const uint32_t o = __shfl_xor_sync(FULL_MASK, v, 2);
  v = prmt(v, o, (t & 2) ? 0x3276u : 0x5410u);
  const uint32_t w = __shfl_xor_sync(FULL_MASK, v, 1);
  return prmt(v, w, (t & 1) ? 0x3715u : 0x6240u);
}

template <int DT>
__global__ void __launch_bounds__(AD_WARPS * 32) k_paged_append_dense(const AppendParams p) {
  extern __shared__ __align__(128) uint8_t smem_dense[];
  DenseSmem &sm = *reinterpret_cast<DenseSmem *>(smem_dense);
  const int side = (int)blockIdx.x < p.k_ctas ? 0 : 1;
  const int cta = side ? blockIdx.x - p.k_ctas : blockIdx.x, n_cta = side ? gridDim.x - p.k_ctas : p.k_ctas;
  const AppendSide &sd = p.side[side];
  pdl_trigger();
  if (threadIdx.x == 0) {
    mbar_init(&sm.full, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&sm.full, sizeof(sm.r));
    bulk_g2s(&sm.r[0][0][0][0], sd.rfrag, sizeof(sm.r), &sm.full);
  }
  WhtTables &tb = sm.tb;
  wht_tables_fill<TQ_FMT_TURBO4>(sd.b, sd.bt, tb);
  __syncthreads();
  const bool ok = mbar_wait_bounded(&sm.full, 0, WAIT_LIMIT_NS);
  pdl_wait();
  if (!ok) {
    if (threadIdx.x == 0) atomicExch(p.pv.status, (int32_t)DEVERR_TIMEOUT);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, l16 = lane & 15;
  const float gs = tb.gs, go = tb.go;
  const int gn = tb.gn, Hkv = p.pv.Hkv;
  const bool turn = side == 0 && p.rope.rot_dim;
  auto &xs = sm.xs[warp];
  const int64_t n_rows = (int64_t)paged_rows(p.pv) * Hkv;
  // lane i < 16: the place and source of row i of a tile
  struct Spot {
    int64_t at;
    uint64_t src;
    int pos;
  };
  auto find = [&](int64_t tile) -> Spot {
    Spot sp{-1, 0, 0};
    const int64_t r = tile * 16 + lane;
    if (lane < 16 && r < n_rows) {
      const int tok = (int)((uint32_t)r / (uint32_t)Hkv), h = (int)(r - (int64_t)tok * Hkv);
      const Place pl = place_row(p.pv, tok, h, true);
      sp.at = pl.at, sp.pos = pl.pos;
      if (pl.at >= 0) sp.src = (uint64_t)(uintptr_t)(sd.src.data + tok * sd.src.token_bytes + h * sd.src.head_bytes);
    }
    return sp;
  };
  // tiles over the CTAs first: a few rows use as many SMs as they can
  const int64_t step = (int64_t)AD_WARPS * n_cta;
  int64_t tile = (int64_t)warp * n_cta + cta;
  Spot spot = find(tile);
  for (; tile * 16 < n_rows; tile += step) {
    const Spot at = spot;
    const int ang = turn ? rope_pos(p.rope, at.at >= 0 ? at.pos : 0, p.pv.status, true) : 0;
    __syncwarp();  // the last tile's fragments are read
    constexpr int NR = 8;
#pragma unroll 1
    for (int rb = 0; rb < 16; rb += NR) {  // eight rows' loads in flight
      float x[NR][4];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const uint8_t *src = reinterpret_cast<const uint8_t *>((uintptr_t)__shfl_sync(FULL_MASK, at.src, rb + i));
        if (src) load_lane4(src, DT, lane, x[i]);
        else x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
      }
      if (turn) {
        const int a0 = __shfl_sync(FULL_MASK, ang, rb);
        if (__all_sync(FULL_MASK, ang == a0 || (lane & 8) != rb || lane >= 16)) {  // one token's heads
          const LaneAngles an = rope_angles(lane, p.rope, a0);
#pragma unroll
          for (int i = 0; i < NR; ++i) rope_turn(x[i], lane, p.rope, an);
        } else {
#pragma unroll
          for (int i = 0; i < NR; ++i)
            rope_turn(x[i], lane, p.rope, rope_angles(lane, p.rope, __shfl_sync(FULL_MASK, ang, rb + i)));
        }
      }
      // norms in the canonical order of the plain fp32 sequence, a row per four lanes in the end
      float s[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i)
        s[i] = __fadd_rn(__fadd_rn(__fmul_rn(x[i][0], x[i][0]), __fmul_rn(x[i][1], x[i][1])),
                         __fadd_rn(__fmul_rn(x[i][2], x[i][2]), __fmul_rn(x[i][3], x[i][3])));
#pragma unroll
      for (int m = 16, k = 4; m >= 4; m >>= 1, k >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < k; ++i) {
          const float keep = up ? s[i + k] : s[i], give = up ? s[i] : s[i + k];
          s[i] = __fadd_rn(keep, __shfl_xor_sync(FULL_MASK, give, m));
        }
      }
      s[0] = __fadd_rn(s[0], __shfl_xor_sync(FULL_MASK, s[0], 2));
      s[0] = __fadd_rn(s[0], __shfl_xor_sync(FULL_MASK, s[0], 1));
      const float n = __fsqrt_rn(s[0]);  // of row rb + lane / 4
      // a norm that is not zero is at least 2^-74.5, the root of the smallest fp32: 1 / n is finite
      const float inv = n > 0.f ? __fdiv_rn(1.0f, n) : 0.0f;
      const int64_t to = __shfl_sync(FULL_MASK, at.at, rb + (lane >> 2));
      if (t == 0 && to >= 0) *reinterpret_cast<float *>(sd.pages + to) = n;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float r = __shfl_sync(FULL_MASK, inv, 4 * i);
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float u0 = x[i][2 * m] * r, u1 = x[i][2 * m + 1] * r;
          hi[m] = pack_bf162(u0, u1);
          lo[m] = pack_bf162(u0 - __uint_as_float(hi[m] << 16), u1 - __uint_as_float(hi[m] & 0xFFFF0000u));
        }
        const int c = 8 * ((lane >> 1) ^ i) + 4 * (lane & 1);  // i is the row modulo 8
        *reinterpret_cast<uint2 *>(&xs[0][rb + i][c]) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2 *>(&xs[1][rb + i][c]) = make_uint2(lo[0], lo[1]);
      }
    }
    __syncwarp();
    spot = find(tile + step);  // its loads run under the products
    float acc[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll 2
    for (int k = 0; k < 8; ++k) {
      uint4 a[2];
#pragma unroll
      for (int part = 0; part < 2; ++part) a[part] = ldmatrix_x4(&xs[part][lane & 15][8 * ((2 * k + (lane >> 4)) ^ (lane & 7))]);
      // R's A fragments hold the B fragments of two column tiles each: registers (0, 2) and (1, 3)
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        const uint4 rh = sm.r[0][m][k][lane], rl = sm.r[1][m][k][lane];
        mma_bf16(acc[2 * m], a[1], rl.x, rl.z), mma_bf16(acc[2 * m + 1], a[1], rl.y, rl.w);
        mma_bf16(acc[2 * m], a[1], rh.x, rh.z), mma_bf16(acc[2 * m + 1], a[1], rh.y, rh.w);
        mma_bf16(acc[2 * m], a[0], rl.x, rl.z), mma_bf16(acc[2 * m + 1], a[0], rl.y, rl.w);
        mma_bf16(acc[2 * m], a[0], rh.x, rh.z), mma_bf16(acc[2 * m + 1], a[0], rh.y, rh.w);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t dst = __shfl_sync(FULL_MASK, at.at, g + 8 * i);
#pragma unroll
      for (int j4 = 0; j4 < 4; ++j4) {
        uint32_t v = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float y0 = acc[4 * j4 + j][2 * i], y1 = acc[4 * j4 + j][2 * i + 1];
          const uint32_t c0 = gn ? cell_index<true, 15>(y0, tb.ce, l16, gs, go, gn, tb.sb) : bucket<15>(y0, tb.sb);
          const uint32_t c1 = gn ? cell_index<true, 15>(y1, tb.ce, l16, gs, go, gn, tb.sb) : bucket<15>(y1, tb.sb);
          v |= (c0 | (c1 << 4)) << (8 * j);
        }
        v = transpose_bytes(v, t);
        if (dst >= 0) reinterpret_cast<uint32_t *>(sd.pages + dst)[1 + 4 * j4 + t] = v;
      }
    }
  }
}

// Dense rotation, few rows: a warp per row on the CUDA cores, R^T staged once per CTA.
constexpr int AF_WARPS = 8;
constexpr size_t AF_SMEM = (size_t)D * D * 4 + AF_WARPS * D * 4;
__global__ void __launch_bounds__(AF_WARPS * 32) k_paged_append_dense_few(const AppendParams p) {
  extern __shared__ __align__(16) float asm_f[];
  float *rt = asm_f, *uv = asm_f + D * D;
  const int side = (int)blockIdx.x < p.k_ctas ? 0 : 1;
  const int cta = side ? blockIdx.x - p.k_ctas : blockIdx.x, n_cta = side ? gridDim.x - p.k_ctas : p.k_ctas;
  const AppendSide &sd = p.side[side];
  __shared__ float sb[16];
  __shared__ __align__(16) uint8_t ib[AF_WARPS][D];
  pdl_trigger();
  stage_matrix(rt, sd.pit);
  if (threadIdx.x < 15) sb[threadIdx.x] = sd.b[threadIdx.x];
  __syncthreads();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *u = uv + warp * D;
  const int64_t n_rows = (int64_t)paged_rows(p.pv) * p.pv.Hkv;
  for (int64_t row = (int64_t)cta * AF_WARPS + warp; row < n_rows; row += (int64_t)n_cta * AF_WARPS) {
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
  if (dense) {
    // Up to a 16-row tile per SM a warp takes a row.  Back to back, 64 rows of each side take 5.1 us so and
    // 8.1 us in tiles, whose latency so few rows do not hide; 512 rows 8.8 and 8.4, 1,200 rows 10.4 and 9.2,
    // 2,400 rows 13.3 and 9.5.
    if ((int64_t)p.pv.n_tokens * p.pv.Hkv <= 16 * sms)
      return launch_rows(k_paged_append_dense_few, p, AF_WARPS * 32, AF_WARPS, AF_SMEM, sms, st);
    if (dtype == TQ_DTYPE_F32)
      return launch_rows(k_paged_append_dense<TQ_DTYPE_F32>, p, AD_WARPS * 32, 16, sizeof(DenseSmem), sms, st);
    if (dtype == TQ_DTYPE_BF16)
      return launch_rows(k_paged_append_dense<TQ_DTYPE_BF16>, p, AD_WARPS * 32, 16, sizeof(DenseSmem), sms, st);
    return launch_rows(k_paged_append_dense<TQ_DTYPE_F16>, p, AD_WARPS * 32, 16, sizeof(DenseSmem), sms, st);
  }
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
    s.rfrag = ctx[i]->d_rfrag;
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
