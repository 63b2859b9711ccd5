// Chunked attention over the paged cache on the 5th-generation tensor cores: ragged batches
// of several rows per sequence, causal, in three launches.
//
//   k_paged_prep      CTA 0 plans: the key tiles (128 keys) of all units (sequence, tile of
//                     queries, KV head) laid end to end, each after a few empty tiles for its
//                     start, cut into one equal share per CTA.  In the other CTAs each warp
//                     turns 16 rows of q by position (fp32), by R (bf16 parts, m16n8k16) and
//                     rounds them to fp16 parts, stored as images of the operand tiles; rows
//                     without a key get their zeros.
//   k_paged_prefill   persistent, one CTA per SM, specialised warps:
//                       loaders    packed tiles, one bulk copy per page, on a ring of three;
//                                  q's tiles, one copy per part and half of the dims
//                       decoders   4 warps each for K and V: nibbles -> fp16 centroids (byte
//                                  permutes) in 128-byte swizzled operand tiles, two stages
//                                  each.  Both are written row by row as 16-byte chunks: K
//                                  is the K-major B operand of S = Q K^T, V the MN-major B
//                                  operand of O += P V, so V needs no transposition.  In one part
//                                  the rows' norms go into the operands: the softmax then reads
//                                  no norms (two 16-byte reads of shared memory per four scores
//                                  of every row, a quarter of its traffic).
//                       2 issuers  one thread each for S, PV and the un-rotation of one
//                                  softmax group
//                       softmax    2 groups of 4 warps, a thread per accumulator row, 64 keys at a
//                                  time while the other 64 columns' products run.  The
//                                  exponentials are taken against the running maximum of
//                                  earlier tiles, and only when the probabilities' sum passed
//                                  2^15 is the maximum raised, O rescaled and the pass repeated;
//                                  then P takes over S's columns.
//                     Groups take two 128-row tiles of one unit (sharing the decoded K and
//                     V), or, where a unit has at most 128 rows or q and P are carried in
//                     two parts, alternate key tiles of one 128-row tile.
//                     At the end of an item O / l goes through the tensor cores once more,
//                     times R (loaded as if it were a value tile), and a unit that lies in
//                     one CTA is finished there: differential pairs, norm, rounding.
//   k_paged_join      units shared by CTAs: the log-sum-exp merge of their partials.
//
// Parts: for bf16 outputs q, K, V, P, O / l and R enter as one fp16 each (off by 2^-11 at most, random over
// 128 dims or the keys).  Together 6e-4 of the output's norm in rms at 300 keys and 8e-4 at 16,000
// (1 to 4% of the rows beyond 1e-3, one in a thousand beyond 2e-3) next to bf16's own 1.7e-3; the largest
// share is that of the scores, where a key's 16 values round alike.  For fp16 and fp32 outputs q, P
// and O / l enter as hi + lo and K, V as centroids with fp32 norms outside the products, which leaves
// the fp16 centroid table's 6e-5.
//
// Measured (GB300): 4 chunks of 200 .. 512 tokens on 4K .. 16K keys, 32 q-heads on 8, bf16: 240 us
// for 199 GFLOP (prep 20, join 13, the rest the attention), 43% of the cuBLAS bf16 rate; prompts of
// 129 .. 2047 tokens, 8 heads on 8, fp16 in two parts: 73 us.  A step of 64 keys takes 1.2 us
// for 2 x 128 rows: 0.9 us from S to P (64 exponentials a thread, beside the decoders' issue slots) and
// 0.3 us of barriers between the roles.  Shared memory carries 41% operands and 23% loads and
// stores of its bandwidth, the issue slots are 60% used, the tensor pipe 44%: no one unit is
// full, the chain S -> P -> PV -> S of a group is.  Tried and slower: two threads a row
// (28 warps, 375 us when this form took 312), scores in registers ahead of the next product
// (spills at the registers 640 threads leave: 298 us to 240), 152 and 56 registers.
#include <math.h>
#include <stddef.h>

#include <type_traits>

#include "tq_decode_common.cuh"
#include "tq_paged.cuh"
#include "tq_rotmma.cuh"
#include "tq_tc.cuh"

namespace tq {

namespace {

constexpr int KT = 128;                // keys per tile
// Cost of an item ahead of its tiles, in tiles, as measured (differential chunks, prompts: 45.5 and 81 us
// with 1, 43.1 and 72.9 with 2, 41.2 and 72.6 with 3, 42.5 and 75.5 with 5).
constexpr int UNIT_TILES = 3;
constexpr int RAW = KT * PG_ROW;       // a packed tile
constexpr int NRAW = 3;
constexpr int W_DEC = 8, W_MMA = 16, W_LOAD = 18, W_Q = 19, N_WARPS = 20;
constexpr int THREADS = N_WARPS * 32;
// Registers: 640 threads x 96 at launch; the softmax groups take 128 (64 scores, 32 packed
// probabilities), the other three groups give theirs up to 72 (the decoders' 17 words of a row
// and norm parts): 256 * 128 + 384 * 72 <= 640 * 96.  144 and 64 spilled in the issuers.
constexpr int REGS_LAUNCH = 96, REGS_SOFTMAX = 128, REGS_OTHER = 72;
static_assert(256 * REGS_SOFTMAX + (THREADS - 256) * REGS_OTHER <= THREADS * REGS_LAUNCH, "the launch's registers");
constexpr uint32_t IDESC_S = (1u << 4) | ((64u >> 3) << 17) | ((128u >> 4) << 24);  // fp16, M = 128, N = 64
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;  // S / P of the groups, O of the groups

constexpr uint32_t OFF_Q = 0, OFF_K = 2 * SW_TILE_BYTES, OFF_V = 4 * SW_TILE_BYTES;
constexpr uint32_t OFF_RAW = 6 * SW_TILE_BYTES, OFF_MISC = OFF_RAW + NRAW * RAW;
struct Misc {
  uint64_t raw_full[NRAW], raw_empty[NRAW];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_full[2], q_empty[2];  // q's tiles (ALT: the first, for both groups and parts)
  uint64_t s_free[2], drain[2];    // [group] the un-rotation has read the columns of S (ALT: the first)
  // [group][half of the key tile]: a thread that waits for a phase of one of these is at most one
  // phase behind, so that the parity tells; the items' final P and un-rotation use half 0 and 1
  uint64_t s_done[2][2], p_ready[2][2], pv_done[2][2];
  // Key norms of the last four K tiles (0 past the end): a K stage is free once its product
  // is done, while the softmax still needs the norms; the decoders reach tile j + 4 only after
  // every group has finished tile j.  The value norms of the two V stages times NORM_FACTOR.
  alignas(16) float kn[4][KT];
  alignas(16) float nv[2][KT], nu[2][KT];  // and log2 of the norms
  // One part: the norms are in the operands, and these hold for 32 rows of a K tile its power of two, and
  // for 32 of a V tile log2 of its power (+ P_SHIFT), 2^- of that (negative: some norms are not finite), and the rows of those.
  alignas(8) float ks[4][KT / 32];
  alignas(8) float ve[2][KT / 32], vi[2][KT / 32];
  uint32_t vbad[2][KT / 32];
  float xm[2][128], xl[2][128], xa[2][128];  // alternating groups: max, sum, largest |O| of a row
  uint32_t tmem;
  int abort_flag;
};
constexpr uint32_t SMEM = OFF_MISC + sizeof(Misc) + 1024;  // + slack to align to 1024
static_assert(SMEM <= 227 * 1024, "shared memory budget");
static_assert(OFF_MISC % 16 == 0 && RAW % 16 == 0, "alignment");

struct Start {
  int b, qt, h, off, left, v, V, G;
};
struct JoinInfo {
  int row, T, base, h, first, n;  // first batch row of the unit, its rows, position of row 0, KV head
};

// Prepared q as images of the operand tiles: for each KV head, part and half of the dims the rows
// (64 dims, 128 bytes, 16-byte chunk c of row r at c ^ (r % 8)) of all 128-row tiles one after the
// other, so that a tile is loaded by a bulk copy per part and half.  A sequence's tiles start at a
// multiple of eight rows and take tr = 8 ceil(qpt gq / 8) each.  With phi(x) = tr floor(x / qpt) + gq (x mod qpt),
// which is superadditive, 8 ceil(phi(a) / 8) + 8 b is past the rows of all sequences before
// sequence b of first row a, whatever their lengths: no sums over sequences.
struct QImage {
  int gq, qpt, tr, rows;  // rows: of a plane
  __host__ __device__ static int phi(int x, int gq, int qpt, int tr) { return x / qpt * tr + x % qpt * gq; }
  __device__ __forceinline__ int first(int a, int b) const { return ((phi(a, gq, qpt, tr) + 7) & ~7) + 8 * b; }
  // element offset of image row r in the plane of (KV head, part, half)
  __device__ __forceinline__ size_t at(int h, int parts, int part, int half, int r) const {
    return (((size_t)(h * parts + part) * 2 + half) * rows + r) * 64;
  }
};

struct PrefillParams {
  PagedView pv;
  const uint8_t *kp, *vp;
  PagedOut o;
  int Hq, gq, qpt, qpu;        // q-heads; per KV head; queries per 128-row tile; per unit
  const uint16_t *qh;          // prepared q: see QImage
  const float *qsc;            // [KV head][image row] power-of-two scales
  QImage qi;
  const Start *start;          // per CTA
  JoinInfo *join;              // per CTA: the unit its first item continues
  float *split;                // [CTA][2][128-row tiles of a unit][PART] partials
  uint32_t klo[2], khi[2], vlo[2], vhi[2];
  float inv_vscale;            // 1 / (2^P_SHIFT * alpha_V) times 2^-NORM_EXP (one part) or 2^W_SHIFT (two)
  const uint8_t *vr;           // R of the values as fp16 hi, lo tile images
};
// Norms in the operands: up to 2^13 times a scaled centroid (below 4) stays below 2^15.
constexpr int NORM_EXP = 12;
// The least power of two of 32 value norms.  A weight beside values of no norm is 2^(7 + V_EXP_LEAST - e) when the
// row's maximum has norms of 2^e: at 2^64, the largest that the encode writes, 21 octaves above exp2's flush.
// Smaller norms use the operand's own range: 2^-67 keeps its precision.
constexpr int V_EXP_LEAST = -48;
// Floats of a 128-row partial: float4 e of row r at e * 128 + r, so that the threads of a warp, a row
// each, write 512 bytes in a row (a row at a time they took 5 us an item); then maxima, sums.
constexpr int PART = 128 * D + 256;

// ------------------------------------------------------------------------------ schedule
struct Seq {
  int row, T, base, n_qt;  // first row, rows taken, position of the first row, query tiles
};
__device__ __forceinline__ Seq seq_of(const PagedView &v, int b, int qpu, bool flag) {
  Seq s{0, 0, 0, 0};
  if (b >= v.B) return s;
  const int n = paged_len(v, b, flag);
  int a = b, e = b + 1;
  if (v.cu_q) a = v.cu_q[b], e = v.cu_q[b + 1];
  if (a < 0 || a >= v.n_tokens || e <= a) return s;
  s.row = a;
  s.base = n - (e - a);
  s.T = min(min(e, v.n_tokens) - a, v.max_q);
  if (flag && e - a > s.T) atomicExch(v.status, (int32_t)DEVERR_SEQLEN);
  s.n_qt = (s.T + qpu - 1) / qpu;
  return s;
}
// Keys the unit's rows see, and their tiles.
__device__ __forceinline__ int unit_keys(const Seq &s, int qt, int qpu) {
  return max(s.base + min(s.T, (qt + 1) * qpu), 0);
}
__device__ __forceinline__ int unit_tiles(const Seq &s, int qt, int qpu) {
  return (unit_keys(s, qt, qpu) + KT - 1) / KT;
}

struct Item {
  int b, qt, h, t0, t1, tiles, keys, vstart;
  Seq s;
};
struct Walk {
  int b, qt, h, off, left, v, tiles;
  Seq s;
};
__device__ __forceinline__ void walk_begin(const PrefillParams &p, Walk &w) {
  const Start st = p.start[blockIdx.x];
  w.b = st.b, w.qt = st.qt, w.h = st.h, w.off = st.off, w.left = st.left, w.v = st.v;
  if (w.left > 0) {
    w.s = seq_of(p.pv, w.b, p.qpu, false);
    w.tiles = unit_tiles(w.s, w.qt, p.qpu);
  }
}
__device__ __forceinline__ Seq seq_from_lane(const Seq &s, int src) {
  return Seq{__shfl_sync(FULL_MASK, s.row, src), __shfl_sync(FULL_MASK, s.T, src), __shfl_sync(FULL_MASK, s.base, src),
             __shfl_sync(FULL_MASK, s.n_qt, src)};
}
// The next sequence with rows, looked for 32 at a time by the whole warp (idle slots may be many).
__device__ __forceinline__ bool next_seq(const PrefillParams &p, Walk &w) {
  for (int b0 = w.b + 1; b0 < p.pv.B; b0 += 32) {
    const Seq s = seq_of(p.pv, b0 + (int)(threadIdx.x & 31), p.qpu, false);
    const uint32_t m = __ballot_sync(FULL_MASK, s.n_qt > 0);
    if (m) {
      w.b = b0 + __ffs(m) - 1;
      w.s = seq_from_lane(s, __ffs(m) - 1);
      return true;
    }
  }
  return false;
}
// (the whole warp calls)
__device__ __forceinline__ bool next_item(const PrefillParams &p, Walk &w, Item &it) {
  while (w.left > 0) {
    if (w.h >= p.pv.Hkv || w.tiles == 0) {  // next query tile, or sequence
      w.h = 0, w.off = 0;
      if (++w.qt >= w.s.n_qt) {
        w.qt = 0;
        if (!next_seq(p, w)) return false;
      }
      w.tiles = unit_tiles(w.s, w.qt, p.qpu);
      continue;
    }
    const int vt = w.tiles + UNIT_TILES, n = min(vt - w.off, w.left);
    it.b = w.b, it.qt = w.qt, it.h = w.h, it.s = w.s, it.tiles = w.tiles;
    it.keys = unit_keys(w.s, w.qt, p.qpu);
    it.t0 = max(w.off - UNIT_TILES, 0), it.t1 = w.off + n - UNIT_TILES;
    it.vstart = w.v - w.off + UNIT_TILES;
    w.v += n, w.left -= n, w.off += n;
    if (w.off == vt) ++w.h, w.off = 0;
    if (it.t1 > it.t0) return true;
  }
  return false;
}

// ------------------------------------------------------------------------------ preparation
constexpr int PREP_WARPS = 20;
struct PrepParams {
  PagedView pv;
  RowsView q;
  RopeView rope;
  PagedOut o;
  int Hq, qpu, grid;      // grid: CTAs of the attention
  float qmul;             // log2(e) * scale / alpha_K
  const uint4 *kfrag;
  uint16_t *qh;
  float *qsc;
  QImage qi;
  int32_t *prefix;        // [B + 1] virtual tiles ahead of each sequence
  Start *start;
  JoinInfo *join;
  int lo;                 // also write the lo parts
};


// Virtual tiles of query tile qt of s (0 past its end), one head.
__device__ __forceinline__ int unit_vtiles(const Seq &s, int qt, int qpu) {
  const int t = qt < s.n_qt ? unit_tiles(s, qt, qpu) : 0;
  return t ? t + UNIT_TILES : 0;
}
__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const int o = __shfl_up_sync(FULL_MASK, x, h);
    if (lane >= h) x += o;
  }
  return x;
}

// One CTA of PREP_WARPS warps: prefix sums over the sequences (in shared memory up to n_sm of them), then
// every share's start.  A thread per sequence, then per share; query tiles are walked 32 at a time
// by the whole warp, one sequence or share after the other (a thread walking 64 tiles by itself,
// twice, took 30 us: longer than all of q's preparation beside it).
__device__ void plan(const PrepParams &p, int *sm_prefix, int n_sm) {
  int *prefix = p.pv.B <= n_sm ? sm_prefix : p.prefix;
  __shared__ int wsum[PREP_WARPS];
  __shared__ int carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, Hkv = p.pv.Hkv;
  if (tid == 0) carry = 0;
  __syncthreads();
  for (int b0 = 0; b0 < p.pv.B; b0 += PREP_WARPS * 32) {
    const int b = b0 + tid;
    const Seq s = seq_of(p.pv, b, p.qpu, true);
    int t = unit_vtiles(s, 0, p.qpu);
    for (uint32_t m = __ballot_sync(FULL_MASK, s.n_qt > 1); m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const Seq w = seq_from_lane(s, src);
      int sum = 0;
      for (int qt = lane; qt < w.n_qt; qt += 32) sum += unit_vtiles(w, qt, p.qpu);
      sum = __reduce_add_sync(FULL_MASK, sum);
      if (lane == src) t = sum;
    }
    t *= Hkv;
    const int inc = warp_scan(t, lane);
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (b < p.pv.B) prefix[b] = before + inc - t;
    __syncthreads();
    if (tid == PREP_WARPS * 32 - 1) carry = before + inc;
    __syncthreads();
  }
  const int V = carry, G = min(p.grid, V);
  for (int c0 = 0; c0 < p.grid; c0 += PREP_WARPS * 32) {
    const int c = c0 + lane * PREP_WARPS + warp;  // neighbours in different warps: all of them have work
    Start st{0, 0, 0, 0, 0, 0, V, G};
    Seq s{0, 0, 0, 0};
    int o = 0;
    if (c < G) {
      st.v = share_start(c, V, G);
      st.left = share_start(c + 1, V, G) - st.v;
      int lo = 0, hi = p.pv.B - 1;  // the last sequence whose prefix is <= v (empty ones are passed over)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= st.v) lo = mid;
        else hi = mid - 1;
      }
      st.b = lo;
      o = st.v - prefix[lo];
      s = seq_of(p.pv, lo, p.qpu, false);
    }
    // the query tile that holds o: the first whose inclusive sum passes it
    for (uint32_t m = __ballot_sync(FULL_MASK, s.n_qt > 0); m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const Seq w = seq_from_lane(s, src);
      int wo = __shfl_sync(FULL_MASK, o, src);
      for (int q0 = 0; q0 < w.n_qt; q0 += 32) {
        const int vt = unit_vtiles(w, q0 + lane, p.qpu), inc = warp_scan(vt * Hkv, lane);
        const uint32_t past = __ballot_sync(FULL_MASK, inc > wo);
        if (past) {
          const int f = __ffs(past) - 1, fvt = __shfl_sync(FULL_MASK, vt, f);
          const int ahead = __shfl_sync(FULL_MASK, inc, f) - fvt * Hkv;
          if (lane == src) {
            st.qt = q0 + f;
            st.h = (wo - ahead) / fvt;
            st.off = wo - ahead - st.h * fvt;
          }
          break;
        }
        wo -= __shfl_sync(FULL_MASK, inc, 31);
      }
    }
    if (c < p.grid) {
      p.join[c].n = 0;
      p.start[c] = st;
    }
  }
}

// Elements 4l .. 4l + 3 of N rows at once (all loads in flight); a null row gives zeros.
template <int N>
__device__ __forceinline__ void load_rows(const uint8_t *const (&row)[N], int dtype, int lane, float (&x)[N][4]) {
  if (dtype == TQ_DTYPE_F32) {
    float4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = row[i] ? reinterpret_cast<const float4 *>(row[i])[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i][0] = v[i].x, x[i][1] = v[i].y, x[i][2] = v[i].z, x[i][3] = v[i].w;
    return;
  }
  uint2 v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = row[i] ? reinterpret_cast<const uint2 *>(row[i])[lane] : make_uint2(0u, 0u);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (dtype == TQ_DTYPE_BF16) {
      x[i][0] = bf16_bits_to_f32(v[i].x & 0xFFFFu), x[i][1] = bf16_bits_to_f32(v[i].x >> 16);
      x[i][2] = bf16_bits_to_f32(v[i].y & 0xFFFFu), x[i][3] = bf16_bits_to_f32(v[i].y >> 16);
    } else {
      const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v[i].x));
      const float2 c = __half22float2(*reinterpret_cast<const __half2 *>(&v[i].y));
      x[i][0] = a.x, x[i][1] = a.y, x[i][2] = c.x, x[i][3] = c.y;
    }
  }
}

// CTA 0 plans; in the others each warp takes tiles of 16 q rows by itself: loaded in rows, turned
// by position, split into bf16 parts in the warp's own shared memory, multiplied by R (three
// products of parts) and stored from the product's fragments.  R's fragments (64 KB) lie in shared
// memory once per SM, from one bulk copy ahead of the wait.  20 warps of their own pace hide each
// other's latencies; blocks of 64 rows that eight warps shared, with barriers between the steps,
// took 36 us for 47488 rows.
struct PrepSmem {
  uint4 r[2][8][8][32];  // R, bf16 hi and lo
  uint16_t xs[PREP_WARPS][2][16][D];  // a warp's rows, bf16 hi and lo; 16-byte chunk c of row r at c ^ (r % 8)
  uint64_t full;
};

__global__ void __launch_bounds__(PREP_WARPS * 32) k_paged_prep(const PrepParams p) {
  extern __shared__ __align__(128) uint8_t smem_prep[];
  PrepSmem &sm = *reinterpret_cast<PrepSmem *>(smem_prep);
  pdl_trigger();
  if (blockIdx.x == 0) {
    pdl_wait();
    plan(p, reinterpret_cast<int *>(&sm.xs[0][0][0][0]), (int)(sizeof(sm.xs) / 4));
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(&sm.full, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&sm.full, sizeof(sm.r));
    bulk_g2s(&sm.r[0][0][0][0], p.kfrag, sizeof(sm.r), &sm.full);
  }
  __syncthreads();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  auto &xs = sm.xs[warp];
  const int64_t n = (int64_t)paged_rows(p.pv) * p.Hq;
  const int ctas = gridDim.x - 1;
  bool have_r = false;
  // tiles over the CTAs first: a few rows use as many SMs as they can
  for (int64_t tile = (int64_t)warp * ctas + blockIdx.x - 1; tile * 16 < n; tile += (int64_t)PREP_WARPS * ctas) {
    const int64_t r0 = tile * 16;
    int my_tok = -1, my_pos = -1;  // of row r0 + lane, its address (0: no key), and its place in q's image
    uint64_t my_src = 0;
    int my_row = -1, my_kvh = 0;
    if (lane < 16 && r0 + lane < n) {
      my_tok = (int)((uint32_t)(r0 + lane) / (uint32_t)p.Hq);
      const int b = paged_seq(p.pv, my_tok);
      my_pos = paged_pos(p.pv, b, my_tok, paged_len(p.pv, b, false));
      const int h = (int)(r0 + lane - (int64_t)my_tok * p.Hq), a = p.pv.cu_q ? p.pv.cu_q[b] : b, li = my_tok - a;
      my_kvh = h / p.qi.gq;
      if (a >= 0 && li >= 0)
        my_row = p.qi.first(a, b) + QImage::phi(li, p.qi.gq, p.qi.qpt, p.qi.tr) + h - my_kvh * p.qi.gq;
      if (my_pos >= 0) my_src = (uint64_t)(uintptr_t)(p.q.data + my_tok * p.q.token_bytes + h * p.q.head_bytes);
    }
    for (uint32_t m = __ballot_sync(FULL_MASK, my_tok >= 0 && my_pos < 0); m; m &= m - 1) {  // no key: the row's output is zero
      const int64_t r = r0 + __ffs(m) - 1;
      const float z[4] = {0.f, 0.f, 0.f, 0.f};
      if (!p.o.diff.lambda) store_lane4(p.o.out, p.o.dtype, (size_t)r * D, lane, z);
      else if (!(r & 1)) store_lane4(p.o.out, p.o.dtype, (size_t)(r >> 1) * D, lane, z);  // Hq is even
    }
    int my_turn = 0;
    if (p.rope.rot_dim) my_turn = rope_pos(p.rope, my_pos, p.pv.status, true);
    __syncwarp();  // the last tile's fragments are read
    constexpr int NR = 8;
#pragma unroll 1
    for (int rb = 0; rb < 16; rb += NR) {  // eight rows' loads in flight
      const uint8_t *src[NR];
      float x[NR][4];
#pragma unroll
      for (int i = 0; i < NR; ++i)
        src[i] = reinterpret_cast<const uint8_t *>((uintptr_t)__shfl_sync(FULL_MASK, my_src, rb + i));
      if (p.rope.rot_dim) {
        const int turn = __shfl_sync(FULL_MASK, my_turn, rb);
        // the heads of a token share its angles
        if (__all_sync(FULL_MASK, my_turn == turn || (lane & 8) != rb || lane >= 16)) {
          const LaneAngles an = rope_angles(lane, p.rope, turn);
          load_rows(src, p.q.dtype, lane, x);
#pragma unroll
          for (int i = 0; i < NR; ++i) rope_turn(x[i], lane, p.rope, an);
        } else {
          load_rows(src, p.q.dtype, lane, x);
#pragma unroll
          for (int i = 0; i < NR; ++i)
            rope_turn(x[i], lane, p.rope, rope_angles(lane, p.rope, __shfl_sync(FULL_MASK, my_turn, rb + i)));
        }
      } else {
        load_rows(src, p.q.dtype, lane, x);
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        uint32_t hi[2], lo[2];
        float f[4];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          hi[m] = pack_bf162(x[i][2 * m], x[i][2 * m + 1]);
          f[2 * m] = __uint_as_float(hi[m] << 16), f[2 * m + 1] = __uint_as_float(hi[m] & 0xFFFF0000u);
        }
        const float big = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
        if (big == INFINITY) {  // an infinite part has no rest
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][e] = isinf(f[e]) ? f[e] = 0.f : x[i][e];
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) lo[m] = pack_bf162(x[i][2 * m] - f[2 * m], x[i][2 * m + 1] - f[2 * m + 1]);
        const int at = 8 * ((lane >> 1) ^ i) + 4 * (lane & 1);  // NR rows: i is the row modulo 8
        *reinterpret_cast<uint2 *>(&xs[0][rb + i][at]) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2 *>(&xs[1][rb + i][at]) = make_uint2(lo[0], lo[1]);
      }
    }
    __syncwarp();
    if (!have_r) {
      if (!mbar_wait_bounded(&sm.full, 0, WAIT_LIMIT_NS)) {
        if (lane == 0) atomicExch(p.pv.status, (int32_t)DEVERR_TIMEOUT);
        return;
      }
      have_r = true;
    }
    // Y = X R^T; R's A fragments hold the B fragments of two column tiles each: registers (0, 2)
    // and (1, 3)
    float acc[16][4];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll 2
    for (int s = 0; s < 8; ++s) {
      uint4 a[2];
#pragma unroll
      for (int part = 0; part < 2; ++part) a[part] = ldmatrix_x4(&xs[part][lane & 15][8 * ((2 * s + (lane >> 4)) ^ (lane & 7))]);
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        const uint4 rh = sm.r[0][m][s][lane], rl = sm.r[1][m][s][lane];
        mma_bf16(acc[2 * m], a[0], rh.x, rh.z), mma_bf16(acc[2 * m + 1], a[0], rh.y, rh.w);
        mma_bf16(acc[2 * m], a[1], rh.x, rh.z), mma_bf16(acc[2 * m + 1], a[1], rh.y, rh.w);
        mma_bf16(acc[2 * m], a[0], rl.x, rl.z), mma_bf16(acc[2 * m + 1], a[0], rl.y, rl.w);
      }
    }
    // rows g and g + 8, columns 8 j + 2 t and the next
    float amax[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[j][e] *= p.qmul;
        amax[e >> 1] = fmaxf(amax[e >> 1], fabsf(acc[j][e]));
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = __shfl_sync(FULL_MASK, my_row, g + 8 * i), kvh = __shfl_sync(FULL_MASK, my_kvh, g + 8 * i);
      float m = amax[i];
      m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, 1));
      m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, 2));
      if (row < 0) continue;
      // The power of two that brings the largest element to [2^13, 2^14).  One part leaves rows alone
      // whose largest element already lies in [2^-10, 2^14) (what fp16 drops there is below 2^-14 of
      // it).
      const bool as_is = !p.lo && m >= 0x1p-10f && m < 0x1p14f;
      const int e = as_is ? 0 : scale_exp(m);
      const float down = pow2i(-e);
      const int parts = p.lo ? 2 : 1;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint16_t *hi_p = p.qh + p.qi.at(kvh, parts, 0, half, row) + 2 * t;
        uint16_t *lo_p = p.qh + p.qi.at(kvh, parts, parts - 1, half, row) + 2 * t;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int j = 8 * half + c, to = 8 * (c ^ (row & 7));
          if (p.lo) {
            uint32_t hi, lo;
            split_half2(acc[j][2 * i] * down, acc[j][2 * i + 1] * down, hi, lo);
            *reinterpret_cast<uint32_t *>(hi_p + to) = hi;
            *reinterpret_cast<uint32_t *>(lo_p + to) = lo;
          } else {
            *reinterpret_cast<uint32_t *>(hi_p + to) = pack_half2(acc[j][2 * i] * down, acc[j][2 * i + 1] * down);
          }
        }
      }
      if (t == 0) p.qsc[(size_t)kvh * p.qi.rows + row] = pow2i(e);
    }
  }
  // (a CTA without rows: R's copy must land before it ends)
  if (!have_r && threadIdx.x == 0) (void)mbar_wait_bounded(&sm.full, 0, WAIT_LIMIT_NS);
}

// ------------------------------------------------------------------------------ attention
__device__ __forceinline__ uint64_t pk2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void upk2(uint64_t r, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Barrier over the 256 softmax threads that ORs a failure flag across them.
__device__ __forceinline__ bool softmax_sync_or(bool fail) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " bar.red.or.pred q, 1, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)fail)
      : "memory");
  return r != 0;
}

// ALT: the groups take alternate key tiles of one 128-row tile.  LO (with ALT): q, P and O / l in
// two fp16 parts.
template <bool ALT, bool LO>
__global__ void __launch_bounds__(THREADS, 1) k_paged_prefill(const PrefillParams p) {
  static_assert(ALT || !LO, "two parts take both q tiles");
  extern __shared__ uint8_t smem_dyn[];
  uint8_t *smem = smem_dyn + ((1024u - (smem_addr(smem_dyn) & 1023u)) & 1023u);
  Misc &ms = *reinterpret_cast<Misc *>(smem + OFF_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int R_TILES = LO ? 2 : 1;  // R as hi [+ lo] value tiles at an item's end
  pdl_trigger();
  if (warp == 0) tmem_alloc(smem_addr(&ms.tmem), TM_COLS);
  if (tid == 0) {
    for (int i = 0; i < NRAW; ++i) mbar_init(&ms.raw_full[i], 1), mbar_init(&ms.raw_empty[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.k_full[i], 4), mbar_init(&ms.v_full[i], 4);
      mbar_init(&ms.k_empty[i], ALT ? 1 : 2), mbar_init(&ms.v_empty[i], ALT ? 1 : 2);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&ms.s_done[i][h], 1), mbar_init(&ms.p_ready[i][h], 4);
        mbar_init(&ms.pv_done[i][h], 1);
      }
      mbar_init(&ms.drain[i], 1), mbar_init(&ms.s_free[i], 1);
      mbar_init(&ms.q_full[i], 1), mbar_init(&ms.q_empty[i], ALT ? 2 : 1);
    }
    ms.abort_flag = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = ms.tmem;
  // Bounded wait; fails at once when another thread has given up already.
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    if (*reinterpret_cast<volatile int *>(&ms.abort_flag)) return false;
    const bool done = mbar_wait_bounded(bar, parity, WAIT_LIMIT_NS);
    if (!done) {
      atomicExch(&ms.abort_flag, 1);
      atomicExch(p.pv.status, (int32_t)DEVERR_TIMEOUT);
    }
    return done;
  };
  Walk w;
  Item it;
  walk_begin(p, w);
  bool ok = true;

  if (warp >= W_DEC) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
  if (warp == W_LOAD) {
    // ================ loader: K and V tiles in turn on the ring
    const int psh = p.pv.page_shift, P = 1 << psh;
    uint32_t n = 0;  // tiles loaded
    while (ok && next_item(p, w, it)) {
      auto page_of = [&](int j) -> int {
        const int pi = ((j * KT) >> psh) + lane;
        if (j >= it.t1 || lane >= 8 || (pi << psh) >= min((j + 1) * KT, it.keys)) return -1;
        return max(paged_page(p.pv, it.b, pi << psh, true), 0);
      };
      int pg = page_of(it.t0);
      for (int j = it.t0; ok && j < it.t1; ++j) {
        const int kf = j * KT, nk4 = (min(KT, it.keys - kf) + 3) & ~3;
        const int pg_next = page_of(j + 1);
        const int k0 = max((((kf >> psh) + lane) << psh), kf), k1 = min(((k0 >> psh) + 1) << psh, kf + nk4);
        for (int side = 0; side < 2; ++side, ++n) {
          const int s = n % NRAW;
          if (n >= NRAW) ok = __all_sync(FULL_MASK, wait(&ms.raw_empty[s], ((n / NRAW) - 1) & 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&ms.raw_full[s], nk4 * PG_ROW);
          __syncwarp();
          if (pg >= 0)
            bulk_g2s(smem + OFF_RAW + s * RAW + (k0 - kf) * PG_ROW,
                     (side ? p.vp : p.kp) + paged_row(p.pv, pg, it.h, k0 & (P - 1)), (uint32_t)(k1 - k0) * PG_ROW,
                     &ms.raw_full[s]);
        }
        pg = pg_next;
      }
    }
    // after a failed wait: let the copies in flight land before the CTA ends
    if (*reinterpret_cast<volatile int *>(&ms.abort_flag))
      for (uint32_t c = n > NRAW ? n - NRAW : 0; c < n; ++c)
        (void)mbar_wait_bounded(&ms.raw_full[c % NRAW], (c / NRAW) & 1, WAIT_LIMIT_NS);
  } else if (warp == W_Q) {
    // ================ q's tiles, each as soon as the last item's scores are done
    uint32_t nl[2] = {0, 0};
    while (ok && next_item(p, w, it)) {
#pragma unroll
      for (int gr = 0; gr < (ALT ? 1 : 2); ++gr) {
        const int q0 = it.qt * p.qpu + gr * p.qpt;
        if (!ok || q0 >= it.s.T) continue;
        if (nl[gr]) ok = __all_sync(FULL_MASK, wait(&ms.q_empty[gr], (nl[gr] - 1) & 1));
        if (!ok) continue;
        const int row = p.qi.first(it.s.row, it.b) + q0 / p.qpt * p.qi.tr;
        const uint32_t bytes = min(p.qi.tr, ((it.s.T - q0) * p.gq + 7) & ~7) * 128;
        if (lane == 0) {
          mbar_arrive_expect_tx(&ms.q_full[gr], bytes * (LO ? 4 : 2));
#pragma unroll
          for (int x = 0; x < (LO ? 4 : 2); ++x)  // part, half
            bulk_g2s(smem + OFF_Q + (gr + (x >> 1)) * SW_TILE_BYTES + (x & 1) * SW_HALF_BYTES,
                     p.qh + p.qi.at(it.h, LO ? 2 : 1, x >> 1, x & 1, row), bytes, &ms.q_full[gr]);
        }
        __syncwarp();
        ++nl[gr];
      }
    }
    // after a failed wait: let the copies in flight land before the CTA ends
    if (*reinterpret_cast<volatile int *>(&ms.abort_flag))
      for (int gr = 0; gr < 2; ++gr)
        if (nl[gr]) (void)mbar_wait_bounded(&ms.q_full[gr], (nl[gr] - 1) & 1, WAIT_LIMIT_NS);
  } else if (warp < W_MMA) {
    // ================ decoders: a group for the keys, one for the values, thread = row of the tile
    const int row = tid & 127;
    const bool side = warp >= W_DEC + 4;
    uint32_t lo2[2], hi2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) lo2[i] = side ? p.vlo[i] : p.klo[i], hi2[i] = side ? p.vhi[i] : p.khi[i];
    uint64_t *full = side ? ms.v_full : ms.k_full, *empty = side ? ms.v_empty : ms.k_empty;
    uint8_t *stages = smem + (side ? OFF_V : OFF_K);
    uint32_t nr = side ? 1 : 0, c = 0;  // raw tiles of both sides passed; stages filled
    uint32_t last_r = 0;                // stages filled with R by a copy of thread 0: see the drain below
    while (ok && next_item(p, w, it)) {
      for (int j = it.t0; ok && j < it.t1; ++j, nr += 2, ++c) {
        const bool live = j * KT + row < it.keys;
        const int st = c & 1, rs = nr % NRAW;
        if (c >= 2) ok = wait(&empty[st], ((c >> 1) - 1) & 1);
        if (ok) ok = wait(&ms.raw_full[rs], (nr / NRAW) & 1);
        ok = __all_sync(FULL_MASK, ok);
        if (!ok) break;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(smem + OFF_RAW + rs * RAW + row * PG_ROW);
        uint8_t *dst = stages + st * SW_TILE_BYTES;
        const float norm = live ? __uint_as_float(src[0]) : 0.f;
        if constexpr (LO) {
#pragma unroll
          for (int ch = 0; ch < 16; ++ch) {
            uint32_t d[4];
            decode8<0x5140u, 0x7362u>(src[1 + ch], lo2, hi2, d);
            *reinterpret_cast<uint4 *>(dst + sw128_offset(row, 8 * ch)) = make_uint4(d[0], d[1], d[2], d[3]);
          }
          if (side) ms.nv[st][row] = norm * NORM_FACTOR, ms.nu[st][row] = fmaxf(log2_approx(norm), -64.f);
          else ms.kn[c & 3][row] = norm;
        } else {
          // The norm goes into the operand: x (nh + nl), the norm as two fp16 parts after the power of
          // two that brings the largest of the warp's 32 rows to [2^NORM_EXP, 2^(NORM_EXP + 1)).  One
          // rounding an element, like q's and P's; a norm 2^20 times smaller than the largest keeps
          // its precision.
          const float an = fabsf(norm);
          const bool bad = !(an < (side ? 0x1p120f : INFINITY));  // (past 2^120 a sum of weights would underflow)
          const uint32_t most = __reduce_max_sync(FULL_MASK, bad ? 0u : __float_as_uint(an));
          const int em = max((int)(most >> 23) - 127, side ? V_EXP_LEAST : -114);
          const float sn = side && bad ? 0.f : norm * pow2i(NORM_EXP - em);
          const __half nh = __float2half_rn(sn), nl = __float2half_rn(sn - __half2float(nh));
          const __half2 nh2 = __half2half2(nh), nl2 = __half2half2(nl);
#pragma unroll
          for (int ch = 0; ch < 16; ++ch) {
            uint32_t d[4];
            decode8<0x5140u, 0x7362u>(src[1 + ch], lo2, hi2, d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 x = *reinterpret_cast<const __half2 *>(&d[e]), y = __hfma2(x, nh2, __hmul2(x, nl2));
              d[e] = *reinterpret_cast<const uint32_t *>(&y);
            }
            *reinterpret_cast<uint4 *>(dst + sw128_offset(row, 8 * ch)) = make_uint4(d[0], d[1], d[2], d[3]);
          }
          const uint32_t bads = __ballot_sync(FULL_MASK, bad);
          const int blk = warp & 3;
          if (lane == 0) {
            // a value of no finite norm: zeros here, so that rows that do not see it stay clean; the
            // softmax makes the others NaN
            if (side) ms.ve[st][blk] = (float)em + P_SHIFT, ms.vi[st][blk] = (bads ? -1.f : 1.f) * pow2i(-em) * exp2f(-P_SHIFT), ms.vbad[st][blk] = bads;
            else ms.ks[c & 3][blk] = pow2i(em - NORM_EXP);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]), mbar_arrive(&ms.raw_empty[rs]);
      }
      if (!side) continue;
      // R of the values as the item's last value tiles
      for (int r = 0; ok && r < R_TILES; ++r, ++c) {
        const int st = c & 1;
        if (c >= 2) ok = __all_sync(FULL_MASK, wait(&ms.v_empty[st], ((c >> 1) - 1) & 1));
        if (!ok) break;
        if (row == 0) {
          mbar_arrive_expect_tx(&ms.v_full[st], SW_TILE_BYTES);
          bulk_g2s(smem + OFF_V + st * SW_TILE_BYTES, p.vr + r * SW_TILE_BYTES, SW_TILE_BYTES, &ms.v_full[st]);
          last_r = c + 1;
        } else if (lane == 0) {
          mbar_arrive(&ms.v_full[st]);
        }
      }
    }
    // after a failed wait: the copy of R must land before the CTA ends (every thread of the
    // warp group arrives for a stage it has passed, so the phase completes with the copy)
    if (side && row == 0 && last_r && *reinterpret_cast<volatile int *>(&ms.abort_flag))
      (void)mbar_wait_bounded(&ms.v_full[(last_r - 1) & 1], ((last_r - 1) >> 1) & 1, WAIT_LIMIT_NS);
  } else if (warp == W_MMA || warp == W_MMA + 1) {
    // ================ issuers: a warp per softmax group, its elected lane issues
    const int gr = __shfl_sync(FULL_MASK, warp - W_MMA, 0);
    const bool lead = elect_lane();
    const uint32_t tS = __shfl_sync(FULL_MASK, tmem, 0) + TM_S + 128 * gr, tO = tS + TM_O - TM_S;
    const uint64_t dq = sw128_desc(smem_addr(smem + OFF_Q) + (ALT ? 0 : gr) * SW_TILE_BYTES);
    const uint64_t dk = sw128_desc(smem_addr(smem + OFF_K)), dv = sw128_mn_desc(smem_addr(smem + OFF_V));
    uint32_t kc = 0, vc = 0, nt = 0;  // K, V stages passed; tiles
    uint32_t nf = 0, nt1 = 0;         // items finished; ALT, group 0: group 1's tiles
    bool issued = false;
    // where P's K-step s (of a half, or of a whole row for the un-rotation) lies
    auto p_col = [](int part, int s) { return LO ? 32 * (s >> 1) + 16 * part + 8 * (s & 1) : 8 * s; };
    while (ok && next_item(p, w, it)) {
      const int n = it.t1 - it.t0;
      const int q0 = it.qt * p.qpu + (ALT ? 0 : gr * p.qpt);
      const bool act = q0 < it.s.T;  // (not ALT) the second row tile may be empty
      const int step = ALT ? 2 : 1, i0 = ALT ? gr : 0, tiles = n > i0 ? (n - i0 + step - 1) / step : 0;
      if (!act) {  // pass the stages on
        for (int i = 0; ok && i < n; ++i) {
          ok = wait(&ms.k_full[(kc + i) & 1], ((kc + i) >> 1) & 1);
          if (ok && lead) mbar_arrive(&ms.k_empty[(kc + i) & 1]);
          if (ok) ok = wait(&ms.v_full[(vc + i) & 1], ((vc + i) >> 1) & 1);
          if (ok && lead) mbar_arrive(&ms.v_empty[(vc + i) & 1]);
          ok = __all_sync(FULL_MASK, ok);
        }
      } else {
        // q, and the columns of S: the last item's un-rotation has read them
        ok = wait(&ms.q_full[ALT ? 0 : gr], nf & 1);
        if (ok && nf) ok = wait(&ms.s_free[ALT ? 0 : gr], (nf - 1) & 1);
        if (!(ok = __all_sync(FULL_MASK, ok))) break;
        tc_fence_after();
        // S of half m & 1 (64 keys) of the group's tile m / 2
        auto issue_s = [&](int m) -> bool {
          const uint32_t c = kc + i0 + step * (m >> 1), h = m & 1;
          if (!h && !__all_sync(FULL_MASK, wait(&ms.k_full[c & 1], (c >> 1) & 1))) return false;
          tc_fence_after();
          const uint64_t kb = desc_step(dk, (c & 1) * SW_TILE_BYTES + h * 64 * 128);
          if (lead) {
#pragma unroll
            for (int part = 0; part < (LO ? 2 : 1); ++part)
#pragma unroll
              for (int s = 0; s < 8; ++s)
                umma<IDESC_S>(tS + 64 * h, desc_step(dq, part * SW_TILE_BYTES + sw128_kstep(s)),
                              desc_step(kb, sw128_kstep(s)), (part || s) ? 1u : 0u);
            umma_commit(&ms.s_done[gr][h]);
            if (h) umma_commit(&ms.k_empty[c & 1]);
            if (m == 2 * tiles - 1) umma_commit(&ms.q_empty[ALT ? 0 : gr]);
          }
          __syncwarp();
          issued = true;
          return true;
        };
        if (ALT && tiles == 0 && lead) mbar_arrive(&ms.q_empty[0]);
        for (int m = 0; ok && m < 2 && m < 2 * tiles; ++m) ok = issue_s(m);
        for (int m = 0; ok && m < 2 * tiles; ++m) {
          const uint32_t c = vc + i0 + step * (m >> 1), h = m & 1;
          ok = wait(&ms.p_ready[gr][h], (h ? nt + (m >> 1) : nt + nf + (m >> 1)) & 1);
          if (ok && !h) ok = wait(&ms.v_full[c & 1], (c >> 1) & 1);
          if (!(ok = __all_sync(FULL_MASK, ok))) break;
          tc_fence_after();
          const uint64_t vb = desc_step(dv, (c & 1) * SW_TILE_BYTES + 2048 * 4 * h);
          if (lead) {
#pragma unroll
            for (int part = 0; part < (LO ? 2 : 1); ++part)
#pragma unroll
              for (int s = 0; s < 4; ++s)
                umma_ts<IDESC_F16_BMN>(tO, tS + 64 * h + p_col(part, s), desc_step(vb, 2048 * s), (m || part || s) ? 1u : 0u);
            umma_commit(&ms.pv_done[gr][h]);
            if (h) umma_commit(&ms.v_empty[c & 1]);
          }
          __syncwarp();
          // the half's next S takes over P's columns: PV must have finished (products on
          // different accumulators may run out of issue order); the softmax is on the other half
          // (ALT: group 1 has no un-rotation of its own)
          ok = __all_sync(FULL_MASK, wait(&ms.pv_done[gr][h], (nt + (h && !(ALT && gr) ? nf : 0) + (m >> 1)) & 1));
          if (ok && m + 2 < 2 * tiles) ok = issue_s(m + 2);
        }
        nt += tiles;
      }
      kc += n, vc += n;
      // un-rotation: O = (O / l) R with O / l where P was
      if (ok && (!ALT || gr == 0)) {
        for (int r = 0; ok && r < R_TILES; ++r) {
          const uint32_t c = vc + r;
          if (act && r == 0) {
            ok = wait(&ms.p_ready[gr][0], (nt + nf) & 1);
            // group 1's last one too (its earlier ones are complete: both groups met before)
            if (ALT && ok) nt1 += n / 2, ok = wait(&ms.p_ready[1][0], (nt1 + nf) & 1);
          }
          if (ok) ok = wait(&ms.v_full[c & 1], (c >> 1) & 1);
          if (!(ok = __all_sync(FULL_MASK, ok))) break;
          tc_fence_after();
          if (lead) {
            if (act) {
              const uint64_t vb = desc_step(dv, (c & 1) * SW_TILE_BYTES);
#pragma unroll
              for (int src = 0; src < (ALT ? 2 : 1); ++src)
#pragma unroll
                for (int part = 0; part < (LO ? 2 : 1); ++part)
                  if (part == 0 || r == 0) {
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                      umma_ts<IDESC_F16_BMN>(tO, tS + 128 * src + p_col(part, s), desc_step(vb, 2048 * s),
                                             (r || src || part || s) ? 1u : 0u);
                  }
              umma_commit(&ms.v_empty[c & 1]);
            } else {
              mbar_arrive(&ms.v_empty[c & 1]);
            }
          }
          __syncwarp();
        }
        if (ok && act && lead) umma_commit(&ms.pv_done[gr][1]), umma_commit(&ms.s_free[gr]);
      }
      if (act) ++nf;  // (ALT: group 1's last P is waited for by group 0's issuer)
      vc += R_TILES;
    }
    if (issued && lead && *reinterpret_cast<volatile int *>(&ms.abort_flag)) {
      umma_commit(&ms.drain[gr]);
      (void)mbar_wait_bounded(&ms.drain[gr], 0, WAIT_LIMIT_NS);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    // ================ softmax: group gr, thread = accumulator row r
    const int gr = warp >> 2, r = tid & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + TM_S + 128 * gr, tO = tmem + lane_off + TM_O + 128 * gr;
    const int rq = r / p.gq, rh = r - rq * p.gq;
    uint32_t kc = 0, vc = 0, ns = 0, nf = 0;  // K, V stages passed; S tiles; items finished
    // After a failed wait a warp goes on to the next barrier of all softmax warps (ALT), where they
    // leave together; without one (not ALT) it leaves by itself.
    bool alive = true;
    while (alive && next_item(p, w, it)) {
      const int n = it.t1 - it.t0;
      const int q0 = it.qt * p.qpu + (ALT ? 0 : gr * p.qpt);
      if (q0 >= it.s.T) {  // (not ALT) no second row tile
        kc += n, vc += n + R_TILES;
        continue;
      }
      const int qi = q0 + rq;
      const bool live = rq < p.qpt && qi < it.s.T;
      const int64_t brow = (int64_t)it.s.row + qi;                       // batch row
      const int head = it.h * p.gq + rh;
      const int64_t qrow = brow * p.Hq + head;
      const int pos = live ? it.s.base + qi : -1;
      const float rsc = live ? p.qsc[(size_t)it.h * p.qi.rows + p.qi.first(it.s.row, it.b) + q0 / p.qpt * p.qi.tr + r] : 0.f;
      [[maybe_unused]] const uint64_t rsc2 = pk2(rsc, rsc);
      float M = -INFINITY, l = 0.f;
      int done = 0;  // halves
      // halves of 64 keys: the other half's PV and next S run under this one's softmax
      const int tiles = ALT ? (n > gr ? (n - gr + 1) / 2 : 0) : n;
      for (int m = 0; m < 2 * tiles; ++m, ++done) {
        const int i = ALT ? gr + 2 * (m >> 1) : (m >> 1), h = m & 1;
        const int kf = (it.t0 + i) * KT + 64 * h;
        const uint32_t cv = vc + i, tH = tS + 64 * h;
        ok = wait(&ms.s_done[gr][h], ns & 1);
        if (ok && !h) ok = wait(&ms.v_full[cv & 1], (cv >> 1) & 1);
        ok = __all_sync(FULL_MASK, ok);
        if (!ok) break;
        tc_fence_after();
        [[maybe_unused]] const float4 *kn4 = reinterpret_cast<const float4 *>(ms.kn[(kc + i) & 3]) + 16 * h;
        [[maybe_unused]] const float4 *nv4 = reinterpret_cast<const float4 *>(ms.nv[cv & 1]) + 16 * h;
        [[maybe_unused]] const float4 *nu4 = reinterpret_cast<const float4 *>(ms.nu[cv & 1]) + 16 * h;
        const bool full = kf + 63 <= it.s.base + q0;  // every row sees every key of the half
        // the largest s + log2(value norm, or the power of two in its operand) of the row
        auto row_max = [&]() -> float {
          float bm = -INFINITY;
          if constexpr (!LO) {
#pragma unroll 1
            for (int cc = 0; cc < 2; ++cc) {
              float sv[32];
              tmem_ld32(tH + 32 * cc, sv);
              const float k = ms.ks[(kc + i) & 3][2 * h + cc] * rsc, v = ms.ve[cv & 1][2 * h + cc] - P_SHIFT;
              const int seen = full ? 32 : pos - (kf + 32 * cc) + 1;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float u = fmaf(sv[e], k, v);
                if (e < seen) bm = fmaxf(bm, u);
              }
            }
          } else {
#pragma unroll 1
            for (int cc = 0; cc < 2; ++cc) {
              float sv[32];
              tmem_ld32(tH + 32 * cc, sv);
#pragma unroll
              for (int c4 = 0; c4 < 8; ++c4) {
                const float4 kn = kn4[8 * cc + c4], nu = nu4[8 * cc + c4];
                const float k_[4] = {kn.x, kn.y, kn.z, kn.w}, u_[4] = {nu.x, nu.y, nu.z, nu.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float u = fmaf(sv[4 * c4 + e] * k_[e], rsc, u_[e]);
                  if (full || kf + 32 * cc + 4 * c4 + e <= pos) bm = fmaxf(bm, u);
                }
              }
            }
          }
          return bm;
        };
        // raise the running maximum of the rows that need it (the warp together); with two parts M is the
        // maximum less W_SHIFT
        auto raise_max = [&](bool now) {
          const float bm = row_max() - (LO ? W_SHIFT : 0);
          const bool raise = bm > M + (now ? 0.f : RESCALE_SLACK);  // also from -inf
          const float half = raise ? exp2_approx(0.5f * (M - bm)) : 1.f, alpha = half * half;
          if (raise) M = bm, l = lower(l, half);
          if (done && __any_sync(FULL_MASK, raise)) {
            // O is whole once the previous half's PV has finished (this half's S was issued after
            // the one before that): half 0 of this tile, or half 1 of the tile before, which
            // shares its barrier with the items' un-rotations
            const uint32_t ph = h ? ns : ns - 1 + (ALT && gr ? 0 : nf);
            ok = __all_sync(FULL_MASK, wait(&ms.pv_done[gr][h ^ 1], ph & 1));
            if (!ok) return;
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc) {
              float o[32];
              tmem_ld32(tO + 32 * cc, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              tmem_st32(tO + 32 * cc, o);
            }
          }
        };
        float lsum;
        if constexpr (LO) {
          raise_max(false);
          const float Mu = (M == -INFINITY) ? 0.f : M;
          const uint64_t nm2 = pk2(-Mu, -Mu);
          uint64_t l2 = pk2(0.f, 0.f);
          // two columns: exponentials into l2, probabilities as fp32; short where every row sees all
          auto pair = [&](auto whole, float s0, float s1, float k0, float k1, float v0, float v1, int c, uint64_t nm2,
                          float &p0, float &p1) {
            const uint64_t sk2 = mul2(pk2(s0, s1), rsc2);
            float d0, d1;
            upk2(fma2(sk2, pk2(k0, k1), nm2), d0, d1);
            float e0 = exp2_approx(d0), e1 = exp2_approx(d1);
            if constexpr (!decltype(whole)::value) e0 = kf + c <= pos ? e0 : 0.f, e1 = kf + c + 1 <= pos ? e1 : 0.f;
            const uint64_t e2 = pk2(e0, e1);
            l2 = add2(l2, e2);
            upk2(mul2(e2, pk2(v0, v1)), p0, p1);
            // a masked value norm may be anything
            if constexpr (!decltype(whole)::value) p0 = kf + c <= pos ? p0 : 0.f, p1 = kf + c + 1 <= pos ? p1 : 0.f;
          };
          auto two_parts = [&](auto whole) {
#pragma unroll 1
            for (int cc = 0; cc < 2; ++cc) {
              float sv[32];
              tmem_ld32(tH + 32 * cc, sv);
              uint32_t pw[32];  // the chunk's hi words, then its lo words, over its own columns
#pragma unroll
              for (int c4 = 0; c4 < 8; ++c4) {
                const float4 kn = kn4[8 * cc + c4], nv = nv4[8 * cc + c4];
                float p0, p1;
                pair(whole, sv[4 * c4], sv[4 * c4 + 1], kn.x, kn.y, nv.x, nv.y, 32 * cc + 4 * c4, nm2, p0, p1);
                split_half2(p0, p1, pw[2 * c4], pw[16 + 2 * c4]);
                pair(whole, sv[4 * c4 + 2], sv[4 * c4 + 3], kn.z, kn.w, nv.z, nv.w, 32 * cc + 4 * c4 + 2, nm2, p0, p1);
                split_half2(p0, p1, pw[2 * c4 + 1], pw[16 + 2 * c4 + 1]);
              }
              tmem_st32(tH + 32 * cc, pw);
            }
          };
          if (full) two_parts(std::true_type());
          else two_parts(std::false_type());
          float l0, l1;
          upk2(l2, l0, l1);
          lsum = l0 + l1;
        } else {
          uint32_t pw[32];
          const float2 vi2 = *reinterpret_cast<const float2 *>(&ms.vi[cv & 1][2 * h]);
          const float vi[2] = {vi2.x, vi2.y};
          const float2 ve2 = *reinterpret_cast<const float2 *>(&ms.ve[cv & 1][2 * h]);
          const float2 ks2 = *reinterpret_cast<const float2 *>(&ms.ks[(kc + i) & 3][2 * h]);
          const float ve[2] = {ve2.x, ve2.y}, ks[2] = {ks2.x, ks2.y};
          bool need = live && M == -INFINITY && kf <= pos;
          for (int turn = 0;; ++turn) {
            if (__any_sync(FULL_MASK, need)) raise_max(need);
            const float Mu = (M == -INFINITY) ? 0.f : M;
            float ps = 0.f;
            lsum = 0.f;
            auto one_part = [&](auto whole) {
              uint32_t sw[2][32];
#pragma unroll
              for (int cc = 0; cc < 2; ++cc) {
                if (!cc) {
                  tmem_ld32_start(tH, sw[0]);
                  tmem_ld32_wait(sw[0]);
                  tmem_ld32_start(tH + 32, sw[1]);
                } else {
                  tmem_ld32_wait(sw[1]);
                }
                const float k = ks[cc] * rsc, mv = ve[cc] - Mu;
                const uint64_t k2 = pk2(k, k), mv2 = pk2(mv, mv);
                const int seen = pos - (kf + 32 * cc) + 1;  // keys of the 32 that the row sees
                uint64_t ps2[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                  float d0, d1;
                  upk2(fma2(pk2(__uint_as_float(sw[cc][c]), __uint_as_float(sw[cc][c + 1])), k2, mv2), d0, d1);
                  float p0 = exp2_approx(d0), p1 = exp2_approx(d1);
                  if constexpr (!decltype(whole)::value) p0 = c < seen ? p0 : 0.f, p1 = c + 1 < seen ? p1 : 0.f;
                  pw[16 * cc + c / 2] = pack_half2(p0, p1);
                  ps2[(c >> 1) & 1] = add2(ps2[(c >> 1) & 1], pk2(p0, p1));
                }
                float p0, p1;
                upk2(add2(ps2[0], ps2[1]), p0, p1);
                p0 += p1;
                ps += p0;
                lsum = fmaf(p0, fabsf(vi[cc]), lsum);
              }
            };
            if (full) one_part(std::true_type());
            else one_part(std::false_type());
            // A probability past 2^15 shows in their sum (at most 2^13 under the current maximum): a
            // maximum would take the slower ALU.  The redo then takes the tile's own maximum.
            need = live && !(ps <= 32768.f);
            if (turn || !__any_sync(FULL_MASK, need)) break;
          }
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            if (vi[cc] > 0.f) continue;  // values without a finite norm among the 32
            const uint32_t bad = ms.vbad[cv & 1][2 * h + cc];
            const int seen = pos - (kf + 32 * cc) + 1;
            if (seen > 0 && (bad & (0xFFFFFFFFu >> (32 - min(seen, 32))))) lsum = NAN;
          }
          tmem_st32(tH, pw);
        }
        l += lsum;
        tc_fence_before();
        if (!ok) break;  // (a failed wait while raising the maximum)
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_ready[gr][h]);
        ns += h;
      }
      kc += n, vc += n + R_TILES;

      // ---- end of the item: O / l as fp16 with a power-of-two row scale, times R
      if (ok && done) {
        // ALT: group 1's un-rotation is group 0's, so its own barrier counts its tiles alone
        ok = __all_sync(FULL_MASK, wait(&ms.pv_done[gr][1], (ns - 1 + (ALT && gr ? 0 : nf)) & 1));
        tc_fence_after();
      }
      float amax = 0.f;
      if (ok && done) {
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          float o[32];
          tmem_ld32(tO + 32 * cc, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) amax = fmaxf(amax, fabsf(o[e]));
        }
      }
      float fw = 1.f;
      if (ALT) {  // the two groups' states of a row, merged
        ms.xm[gr][r] = M, ms.xl[gr][r] = l, ms.xa[gr][r] = amax;
        if (softmax_sync_or(!ok)) {
          alive = false;
          break;
        }
        const float M0 = ms.xm[0][r], M1 = ms.xm[1][r], l0 = ms.xl[0][r], l1 = ms.xl[1][r];
        const float a0 = ms.xa[0][r], a1 = ms.xa[1][r];
        (void)softmax_sync_or(false);  // read: the next item may write them
        const float Mx = fmaxf(M0, M1);
        const float f0 = M0 == -INFINITY ? 0.f : exp2f(M0 - Mx), f1 = M1 == -INFINITY ? 0.f : exp2f(M1 - Mx);
        fw = gr ? f1 : f0;
        // (without a maximum a group's sum is 0, or NaN where its scores are)
        l = (M0 == -INFINITY ? l0 : lower_by(l0, M0 - Mx)) + (M1 == -INFINITY ? l1 : lower_by(l1, M1 - Mx));
        amax = fmaxf(f0 ? f0 * a0 : 0.f, f1 ? f1 * a1 : 0.f);
        M = Mx;
      } else if (!ok) {
        break;
      }
      const float fo = l == 0.f ? 0.f : p.inv_vscale / l;
      const float am = amax * fo;
      const int ex = scale_exp(am);
      // (a row without a maximum holds zeros here: a NaN sum reaches it through the scale)
      const float mul = fo * fw * pow2i(-ex), back = isnan(l) ? l : pow2i(ex);
      const bool zero = done == 0 || fw == 0.f || fo == 0.f;  // O holds nothing (of the row)
#pragma unroll 1
      for (int c2 = 0; c2 < (LO ? 4 : 2); ++c2) {
        uint32_t pw[32];
        if constexpr (LO) {
          float o[32];
          tmem_ld32(tO + 32 * c2, o);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            split_half2(zero ? 0.f : o[2 * e] * mul, zero ? 0.f : o[2 * e + 1] * mul, pw[e], pw[16 + e]);
        } else {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float o[32];
            tmem_ld32(tO + 64 * c2 + 32 * hf, o);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              pw[16 * hf + e] = pack_half2(zero ? 0.f : o[2 * e] * mul, zero ? 0.f : o[2 * e + 1] * mul);
          }
        }
        tmem_st32(tS + 32 * c2, pw);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.p_ready[gr][0]);
      if (ALT && gr == 1) continue;
      ok = __all_sync(FULL_MASK, wait(&ms.pv_done[gr][1], (ns + nf) & 1));
      ++nf;
      if (!ok) {
        if (ALT) continue;
        break;
      }
      tc_fence_after();

      // ---- the unit's rows, or this CTA's partial of them
      const Start st = p.start[blockIdx.x];
      const int first = share_of(it.vstart, st.V, st.G);
      const int n_split = share_of(it.vstart + it.tiles - 1, st.V, st.G) - first + 1;
      if (tid == 0 && (int)blockIdx.x != first)
        p.join[blockIdx.x] = JoinInfo{it.s.row + it.qt * p.qpu, it.s.T - it.qt * p.qpu, 0, it.h, first, n_split};
      if (n_split > 1) {
        float *part = p.split + ((size_t)(blockIdx.x * 2 + ((int)blockIdx.x == first ? 1 : 0)) * (ALT ? 1 : 2) + gr) * PART;
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          float o[32];
          tmem_ld32(tO + 32 * cc, o);
          if (live) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<float4 *>(part)[(8 * cc + e) * 128 + r] =
                  make_float4(o[4 * e] * back, o[4 * e + 1] * back, o[4 * e + 2] * back, o[4 * e + 3] * back);
          }
          __syncwarp();
        }
        if (live) part[128 * D + r] = M, part[128 * D + 128 + r] = l;
        continue;
      }
      const DiffView &df = p.o.diff;
      float scale = back, lam = 0.f;
      int64_t at = qrow * D;
      bool store = live;
      if (df.lambda) {  // rows r and r ^ 1 are a pair: the even lane finishes it
        const int pair_i = head >> 1;
        at = (brow * (p.Hq / 2) + pair_i) * D;
        store = live && !(r & 1);
        if (live) lam = df.lambda[brow * df.lambda_stride + pair_i];
        scale = df.out_scale;
        if (df.gain) {
          float ss = 0.f;
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            float o[32];
            tmem_ld32(tO + 32 * cc, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float a = o[e] * back, b = __shfl_xor_sync(FULL_MASK, a, 1), d = fmaf(-lam, b, a);
              ss = fmaf(d, d, ss);
            }
          }
          scale = diff_factor(ss, df);
        }
      }
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        float o[32];
        tmem_ld32(tO + 32 * cc, o);
        if (df.lambda) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float a = o[e] * back, b = __shfl_xor_sync(FULL_MASK, a, 1);
            o[e] = fmaf(-lam, b, a) * scale * (df.gain ? df.gain[32 * cc + e] : 1.f);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= scale;
        }
        if (store && p.o.dtype == TQ_DTYPE_F32) {
          float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.o.out) + at + 32 * cc);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else if (store) {
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.o.out) + at + 32 * cc);
          const bool bf = p.o.dtype == TQ_DTYPE_BF16;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t x[4];
#pragma unroll
            for (int m = 0; m < 4; ++m)
              x[m] = bf ? pack_bf162(o[8 * e + 2 * m], o[8 * e + 2 * m + 1]) : pack_half2(o[8 * e + 2 * m], o[8 * e + 2 * m + 1]);
            dst[e] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, TM_COLS);
}

// ------------------------------------------------------------------------------ join
struct JoinParams {
  PagedOut o;
  int Hq, gq, qpt, unit_rows, grid;
  const JoinInfo *join;
  const float *split;
};
constexpr int JOIN_WARPS = 8, JOIN_ROWS = 16;

// CTA (c, y): 16 rows of the unit whose second share is CTA c's: o = sum w_s o_s / sum w_s with
// w_s = l_s 2^(m_s - m*).  Lane (e, r) of a warp takes row r of eight and two float4 of the 32, so that loads
// follow the partials' layout; four warps make up the rows, four parts of each are in flight.
__global__ void __launch_bounds__(JOIN_WARPS * 32) k_paged_join(const JoinParams p) {
  __shared__ float sums[JOIN_WARPS][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x;
  const JoinInfo j = p.join[c];
  if (j.n < 2 || j.first != c - 1) return;
  const int ns = min(j.n, p.grid - j.first);
  const bool diff = p.o.diff.lambda != nullptr;
  const int r = JOIN_ROWS * blockIdx.y + 8 * (warp >> 2) + (lane & 7), rr = r & 127, rq = rr / p.gq;
  const int qi = (r >> 7) * p.qpt + rq, head = j.h * p.gq + rr - rq * p.gq, e0 = 8 * (warp & 3) + (lane >> 3);
  const bool live = rq < p.qpt && qi < j.T;
  auto part_of = [&](int s) {
    return p.split + ((size_t)((j.first + s) * 2 + (s == 0 ? 1 : 0)) * (p.unit_rows / 128) + (r >> 7)) * PART;
  };
  constexpr int FLY = 4;
  float a[2][4] = {}, top = -INFINITY, sum = 0.f;
  for (int s0 = 0; s0 < ns; s0 += FLY) {
    float mx[FLY], lx[FLY];
    float4 v[FLY][2];
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      mx[i] = lx[i] = 0.f, v[i][0] = v[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (live && s0 + i < ns) {
        const float *part = part_of(s0 + i);
        mx[i] = __ldcg(part + 128 * D + rr), lx[i] = __ldcg(part + 128 * D + 128 + rr);
#pragma unroll
        for (int h = 0; h < 2; ++h) v[i][h] = __ldcg(reinterpret_cast<const float4 *>(part) + (e0 + 4 * h) * 128 + rr);
      }
    }
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      if (lx[i] == 0.f) continue;
      const float mn = fmaxf(top, mx[i]), fh = exp2f(0.5f * (top - mn)), f = fh * fh, wx = lower_by(lx[i], mx[i] - mn);
      top = mn;
      sum = lower(sum, fh) + wx;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[h][0] = fmaf(a[h][0], f, wx * v[i][h].x), a[h][1] = fmaf(a[h][1], f, wx * v[i][h].y);
        a[h][2] = fmaf(a[h][2], f, wx * v[i][h].z), a[h][3] = fmaf(a[h][3], f, wx * v[i][h].w);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e) a[h][e] *= inv;
  const int64_t row = j.row + qi;
  if (!diff) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (live) store_lane4(p.o.out, p.o.dtype, (row * p.Hq + head) * D, e0 + 4 * h, a[h]);
    return;
  }
  // rows r and r ^ 1 are a pair, finished by the even one
  const DiffView &d = p.o.diff;
  const float lam = live ? d.lambda[row * d.lambda_stride + (head >> 1)] : 0.f;
  float ss = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[h][e] = fmaf(-lam, __shfl_xor_sync(FULL_MASK, a[h][e], 1), a[h][e]);
      ss = fmaf(a[h][e], a[h][e], ss);
    }
  float f = d.out_scale;
  if (d.gain) {
    ss += __shfl_xor_sync(FULL_MASK, ss, 8);
    ss += __shfl_xor_sync(FULL_MASK, ss, 16);
    if (lane < 8) sums[warp][lane] = ss;
    __syncthreads();
    const int w0 = warp & ~3, q = lane & 7;
    ss = (sums[w0][q] + sums[w0 + 1][q]) + (sums[w0 + 2][q] + sums[w0 + 3][q]);
    f = diff_factor(ss, d);
  }
  if (!live || (r & 1)) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 g = d.gain ? reinterpret_cast<const float4 *>(d.gain)[e0 + 4 * h] : make_float4(1.f, 1.f, 1.f, 1.f);
    a[h][0] *= f * g.x, a[h][1] *= f * g.y, a[h][2] *= f * g.z, a[h][3] *= f * g.w;
    store_lane4(p.o.out, p.o.dtype, (row * (p.Hq / 2) + (head >> 1)) * D, e0 + 4 * h, a[h]);
  }
}

struct Layout {
  int gq, qpt, qpu, grid, unit_rows;
  QImage qi;
  bool alt, lo;
  size_t qsc, prefix, start, join, split, bytes;
};
bool layout(const tq_ctx *k, const PagedView &pv, int Hq, int out_dtype, Layout *l) {
  l->gq = Hq / pv.Hkv;
  l->qpt = 128 / l->gq;
  l->lo = out_dtype != TQ_DTYPE_BF16;
  // one row tile: both groups on it, else half of the softmax would idle
  l->alt = l->lo || pv.max_q <= l->qpt;
  l->qpu = l->alt ? l->qpt : 2 * l->qpt;
  l->unit_rows = l->alt ? 128 : 256;
  l->grid = k->num_sms;
  const int64_t units = ((int64_t)pv.n_tokens / l->qpu + pv.B + 1) * pv.Hkv;
  const int64_t tiles = units * (((int64_t)pv.max_len + KT - 1) / KT + UNIT_TILES);
  if (tiles > INT32_MAX || (int64_t)pv.n_tokens * Hq > INT32_MAX) return false;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const int tr = (l->qpt * l->gq + 7) & ~7;
  const int64_t plane = (int64_t)pv.n_tokens / l->qpt * tr + (int64_t)(pv.n_tokens % l->qpt) * l->gq + 8 + 8 * ((int64_t)pv.B + 1);
  if (plane * pv.Hkv > INT32_MAX) return false;
  l->qi = QImage{l->gq, l->qpt, tr, (int)plane};
  l->qsc = up((size_t)pv.Hkv * (l->lo ? 2 : 1) * plane * D * 2);
  l->prefix = l->qsc + up((size_t)pv.Hkv * plane * 4);
  l->start = l->prefix + up((size_t)(pv.B + 1) * 4);
  l->join = l->start + up((size_t)l->grid * sizeof(Start));
  l->split = l->join + up((size_t)l->grid * sizeof(JoinInfo));
  l->bytes = l->split + up((size_t)l->grid * 2 * (l->unit_rows / 128) * PART * 4);
  return true;
}

template <bool ALT, bool LO>
cudaError_t launch_main(const PrefillParams &p, int grid, cudaStream_t st) {
  cudaError_t e = kernel_smem_attr((const void *)k_paged_prefill<ALT, LO>, (int)SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_paged_prefill<ALT, LO>, dim3(grid), dim3(THREADS), SMEM, st, p);
}

}  // namespace

bool paged_prefill_workspace(const tq_ctx *k, const PagedView &pv, int Hq, size_t *bytes) {
  Layout a, b;  // the size does not depend on the output's type
  if (!layout(k, pv, Hq, TQ_DTYPE_BF16, &a) || !layout(k, pv, Hq, TQ_DTYPE_F32, &b)) return false;
  *bytes = a.bytes > b.bytes ? a.bytes : b.bytes;
  return true;
}

cudaError_t launch_paged_prefill(const tq_ctx *k, const tq_ctx *v, const PagedView &pv, const uint8_t *kp,
                                 const uint8_t *vp, const RowsView &q, int Hq, const RopeView &rope, float scale,
                                 const PagedOut &o, void *ws, cudaStream_t st) {
  Layout l;
  if (!layout(k, pv, Hq, o.dtype, &l)) return cudaErrorInvalidValue;
  uint8_t *base = static_cast<uint8_t *>(ws);
  PrepParams a{};
  a.pv = pv, a.q = q, a.rope = rope, a.o = o;
  a.Hq = Hq, a.qpu = l.qpu, a.grid = l.grid, a.qi = l.qi;
  a.qmul = LOG2E * scale / k->f16.alpha;
  a.kfrag = k->d_rfrag;
  a.qh = reinterpret_cast<uint16_t *>(base);
  a.qsc = reinterpret_cast<float *>(base + l.qsc);
  a.prefix = reinterpret_cast<int32_t *>(base + l.prefix);
  a.start = reinterpret_cast<Start *>(base + l.start);
  a.join = reinterpret_cast<JoinInfo *>(base + l.join);
  a.lo = l.lo;
  const int64_t rows = (int64_t)pv.n_tokens * Hq;
  cudaError_t e = kernel_smem_attr((const void *)k_paged_prep, (int)sizeof(PrepSmem));
  if (e != cudaSuccess) return e;
  const int64_t tiles = (rows + 15) / 16, most = k->num_sms - 1;
  e = launch_pdl(k_paged_prep, dim3(1 + (unsigned)(tiles < most ? tiles : most)), dim3(PREP_WARPS * 32), sizeof(PrepSmem),
                 st, a);
  if (e != cudaSuccess) return e;
  PrefillParams p{};
  p.pv = pv, p.kp = kp, p.vp = vp, p.o = o;
  p.Hq = Hq, p.gq = l.gq, p.qpt = l.qpt, p.qpu = l.qpu;
  p.qh = a.qh, p.qsc = a.qsc, p.qi = l.qi, p.start = a.start, p.join = a.join;
  p.split = reinterpret_cast<float *>(base + l.split);
  for (int i = 0; i < 2; ++i) {
    p.klo[i] = k->f16.lo[i], p.khi[i] = k->f16.hi[i];
    p.vlo[i] = v->f16.lo[i], p.vhi[i] = v->f16.hi[i];
  }
  p.inv_vscale = 1.0f / (exp2f(P_SHIFT + (l.lo ? -W_SHIFT : NORM_EXP)) * v->f16.alpha);
  p.vr = reinterpret_cast<const uint8_t *>(v->d_rtile);
  e = l.lo ? launch_main<true, true>(p, l.grid, st)
           : (l.alt ? launch_main<true, false>(p, l.grid, st) : launch_main<false, false>(p, l.grid, st));
  if (e != cudaSuccess) return e;
  JoinParams j{};
  j.o = o;
  j.Hq = Hq, j.gq = l.gq, j.qpt = l.qpt, j.unit_rows = l.unit_rows, j.grid = l.grid;
  j.join = p.join, j.split = p.split;
  return launch_pdl(k_paged_join, dim3(l.grid, l.unit_rows / JOIN_ROWS), dim3(JOIN_WARPS * 32), 0, st, j);
}

}  // namespace tq
