// Single-row attention over the paged cache: split-K decode through a block table, in two
// launches.
//
//   k_paged_partial  persistent, one CTA per SM.  The key tiles (240 keys; 224 where a unit has
//                    more than four heads) of all units
//                    (sequence, KV head, group of 4 or 8 q-heads) lie end to end in one
//                    virtual sequence, each unit preceded by a few empty tiles that stand
//                    for the cost of starting it; CTA c takes the c-th equal share, so
//                    ragged lengths balance.  The shares come from the lengths on the
//                    device, so a captured launch follows them.  Per item the consumer
//                    warps rotate the unit's q by its position (fp32) and by R (a WHT in the
//                    warp, a dense R as bf16 parts on the tensor cores,
//                    tq_rotmma.cuh) themselves, while the producer
//                    warp already streams the first tiles: a tile is one bulk copy per
//                    page it meets (K by lanes 0-15, V by lanes 16-31, the page ids of the
//                    next tile loaded one tile ahead) on a four-stage ring.  The products
//                    are those of the contiguous decode: nibble pairs become fp16x2
//                    centroid pairs through a shared-memory table, scores and PV run as
//                    m16n8k16 MMAs with q and the probabilities in fp16 hi + lo parts.
//   k_paged_combine  merges the shares of each unit, R^T o on the tensor cores, the
//                    differential pair and its norm, rounding to the output type.
//
// Measured (GB300): 8 sequences of 24K .. 32K tokens, 32 q-heads on 8: 58 us for 238 MB; 64 ragged
// sequences up to 16K, 12 on 2: 28.9 us; one of 733 tokens: 9.6 us.  A tile takes 1 us (1.9 us of five
// to eight heads), bound by 64 table lookups a warp and 16 keys on the shared-memory path (63%) and by issue
// (61%); an item's start and merge take 2.5 us, the launch's start 3.5 us.
#include <math.h>

#include "tq_decode_common.cuh"
#include "tq_paged.cuh"
#include "tq_rotmma.cuh"
#include "tq_t4_tile.cuh"

namespace tq {

namespace {

// Consumer warps, keys of a pipeline stage and threads (with the producer warp).  GROUPS = 1: units of
// up to four heads, a warp per 16 keys.  GROUPS = 2: up to eight, two warps per 32 keys.
template <int GROUPS>
struct Shape {
  static constexpr int CW = GROUPS == 1 ? 15 : 14, TILE = 16 * CW, NT = (CW + 1) * 32;
  // Cost of an item ahead of its tiles, in tiles, as measured: 3 of 1 us (differential decode of 16: 29.5 us
  // with 3, 29.9 with 4, 30.4 with 5), 1 of 1.9 us (64 ragged sequences of 6 heads: 28.6 us with 1, 29.2
  // with 2, 30.8 with 3).
  static constexpr int ITEM_TILES = GROUPS == 1 ? 3 : 1;
};
constexpr int MAX_CW = Shape<1>::CW, MAX_TILE = Shape<1>::TILE;
constexpr int NSTAGE = 4;
constexpr int STAGE = MAX_TILE * PG_ROW + 32;  // 16,352 bytes, a multiple of 32
constexpr int PROW = D + 4;          // floats of a partial: acc[128], max (less W_SHIFT), sum, 2 spare

struct DecodeParams {
  PagedView pv;
  const uint8_t *kp, *vp;
  RowsView q;
  RopeView rope;
  int Hq, gq, n_hg, hpc;   // q-heads; per KV head; head groups per KV head; heads of a unit
  float qmul;              // log2(e) * scale / alpha_K
  const uint4 *kfrag;      // dense R of the keys (null: WHT, signs in wht_neg)
  uint32_t wht_neg[4];
  uint32_t kc16[8], vc16[8];
  uint32_t klo[2], khi[2], vlo[2], vhi[2];
  float *split;            // [CTA][2][8] partials of units that several CTAs share
  float *whole;            // [row][Hq] partials of units one CTA finished
  int32_t *unit;           // per unit: first CTA | CTAs << 16
};

struct Head {
  union {
    float osm[MAX_CW][4][D];   // the warps' accumulators of 4 heads, for the merge
    struct {
      RotColumns x;        // the item's q
      float y[8][D + 4];   // R q
    } prep;
  };
  uint64_t full[NSTAGE], empty[NSTAGE];
  float mw[MAX_CW][4], lw[MAX_CW][4];
  float mh[8], lh[8];      // the item's maxima and sums
  int abort_flag;
  int V, G;                // the V virtual tiles are shared by G CTAs
  int first, n_split;      // the CTAs that share the item's unit
};
struct Tail {
  uint32_t q[8][D];        // fp16 hi then lo of the item's rotated q
  float qs[8];             // and its power-of-two scales
};
constexpr uint32_t A_OFF = (sizeof(Head) + 15) & ~15u;
constexpr uint32_t LUT_OFF = LUT_WINDOW - RESERVED_SMEM;
constexpr uint32_t B_OFF = LUT_OFF + 256 * 64 * 4;
constexpr int BELOW = 2;   // stage buffers below the table
constexpr uint32_t TAIL_OFF = B_OFF + (2 * NSTAGE - BELOW) * STAGE;
constexpr uint32_t SMEM = TAIL_OFF + sizeof(Tail);
static_assert(A_OFF + BELOW * STAGE <= LUT_OFF, "the head and two stage buffers below the table");
static_assert(SMEM + RESERVED_SMEM <= 228 * 1024, "shared memory of one SM");

// Stage buffer i: K of stage i (i < 4), V of stage i - 4.
__device__ __forceinline__ uint8_t *stage_at(uint8_t *sm, int i) {
  return sm + (i < BELOW ? A_OFF + i * STAGE : B_OFF + (i - BELOW) * STAGE);
}

// Barrier over the first N threads, apart from that of all the consumers.
template <int N>
__device__ __forceinline__ void named_sync2() {
  asm volatile("bar.sync 2, %0;" ::"n"(N) : "memory");
}

// A head's R q (elements 4l .. 4l + 3 of lane l) times mul, scaled by a power of two 2^-e so that
// the largest element lies in [2^13, 2^14), as fp16 hi and lo: word w of a part (elements 2w,
// 2w + 1) at 16 (w / 16) + ((w % 16) ^ x), x of the part and block, so that the consumers' lanes,
// which read word w % 16 of 16 (part, block) pairs of a bank each, hit 32 banks.
__device__ __forceinline__ void split_q(float (&v)[4], float mul, Tail &tl, int slot, int lane) {
  float amax = 0.f;
#pragma unroll
  for (int m = 0; m < 4; ++m) v[m] *= mul, amax = fmaxf(amax, fabsf(v[m]));
  amax = __uint_as_float(__reduce_max_sync(FULL_MASK, __float_as_uint(amax)));  // ordered like the floats
  const int e = scale_exp(amax);
  const float down = pow2i(-e);
  const int t = lane >> 3, at = 16 * t + 2 * (lane & 7), x = 4 * (slot & 3) + (t >> 1);
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    uint32_t hi, lo;
    split_half2(v[2 * m] * down, v[2 * m + 1] * down, hi, lo);
    tl.q[slot][(at + m) ^ x] = hi;               // part 0: 2 g + t / 2 with g = 2 (slot % 4)
    tl.q[slot][64 + ((at + m) ^ (x + 2))] = lo;  // part 1: g + 1
  }
  if (lane == 0) tl.qs[slot] = pow2i(e);
}

// H D x of a row held as elements 4l .. 4l + 3 of lane l (without the 1 / sqrt(128)).
__device__ __forceinline__ void wht_lane4(float (&x)[4], const uint32_t (&neg)[4], int lane) {
  const uint32_t n = neg[lane >> 3] >> (4 * (lane & 7));
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = (n >> e) & 1u ? -x[e] : x[e];
  const float a = x[0] + x[1], b = x[0] - x[1], c = x[2] + x[3], d = x[2] - x[3];
  x[0] = a + c, x[1] = b + d, x[2] = a - c, x[3] = b - d;
#pragma unroll
  for (int h = 1; h <= 16; h <<= 1) {
    const float sg = (lane & h) ? -1.f : 1.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fmaf(sg, x[e], __shfl_xor_sync(FULL_MASK, x[e], h));
  }
}

// Keys that sequence b's row sees and the row (-1: none).
__device__ __forceinline__ int seq_keys(const PagedView &v, int b, int *row, bool flag) {
  const int n = paged_len(v, b, flag);
  if (!v.cu_q) {
    *row = b;
    return n;
  }
  const int a = v.cu_q[b], e = v.cu_q[b + 1];
  if (a < 0 || a >= v.n_tokens || e <= a) {
    *row = -1;
    return 0;
  }
  if (flag && e - a > 1) atomicExch(v.status, (int32_t)DEVERR_SEQLEN);  // rows past max_q = 1
  *row = a;
  return max(n - (e - a) + 1, 0);
}
template <int GROUPS>
__device__ __forceinline__ int key_tiles(int keys) {
  return (keys + Shape<GROUPS>::TILE - 1) / Shape<GROUPS>::TILE;
}

// Walks a CTA's share: per unit met, the tiles [t0, t1) of it.
struct Walk {
  int b, u, off, left;  // sequence, unit within it, virtual offset within the unit, tiles left
  int v;                // virtual position
  int keys, row, tiles;
};
struct Item {
  int b, u, t0, t1, keys, row, tiles, vstart;
};

// One warp: the total of virtual tiles (flagging bad lengths), then this CTA's share.
template <int GROUPS>
__device__ __forceinline__ int total_tiles(const DecodeParams &p, int lane, bool flag) {
  const int upb = p.pv.Hkv * p.n_hg;
  int sum = 0;
  for (int b = lane; b < p.pv.B; b += 32) {
    int row;
    const int t = key_tiles<GROUPS>(seq_keys(p.pv, b, &row, flag));
    sum += t ? t + Shape<GROUPS>::ITEM_TILES : 0;
  }
#pragma unroll
  for (int h = 16; h >= 1; h >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, h);
  return sum * upb;
}
// One warp: the sequence that holds virtual tile v and the offset within it.
template <int GROUPS>
__device__ __forceinline__ void seek(const DecodeParams &p, int v, int lane, int *b_out, int *off_out) {
  const int upb = p.pv.Hkv * p.n_hg;
  int base = 0;
  for (int b0 = 0;; b0 += 32) {
    const int b = b0 + lane;
    int row, t = 0;
    if (b < p.pv.B) {
      t = key_tiles<GROUPS>(seq_keys(p.pv, b, &row, false));
      t = t ? (t + Shape<GROUPS>::ITEM_TILES) * upb : 0;
    }
    int inc = t;
#pragma unroll
    for (int h = 1; h < 32; h <<= 1) {
      const int o = __shfl_up_sync(FULL_MASK, inc, h);
      if (lane >= h) inc += o;
    }
    const uint32_t hit = __ballot_sync(FULL_MASK, base + inc > v);
    if (hit || b0 + 32 >= p.pv.B) {
      const int l = hit ? __ffs(hit) - 1 : 31;
      *b_out = b0 + l;
      *off_out = v - (base + __shfl_sync(FULL_MASK, inc - t, l));
      return;
    }
    base += __shfl_sync(FULL_MASK, inc, 31);
  }
}

template <int GROUPS>
__device__ __forceinline__ void walk_load(const DecodeParams &p, Walk &w) {
  w.keys = w.b < p.pv.B ? seq_keys(p.pv, w.b, &w.row, false) : 0;
  w.tiles = key_tiles<GROUPS>(w.keys);
}
// The next sequence with keys, looked for 32 at a time by the whole warp (idle slots may be many).
template <int GROUPS>
__device__ __forceinline__ bool walk_next(const DecodeParams &p, Walk &w) {
  for (int b0 = w.b + 1; b0 < p.pv.B; b0 += 32) {
    const int b = b0 + (int)(threadIdx.x & 31);
    int row = -1;
    const int keys = b < p.pv.B ? seq_keys(p.pv, b, &row, false) : 0;
    const uint32_t m = __ballot_sync(FULL_MASK, keys > 0);
    if (m) {
      const int src = __ffs(m) - 1;
      w.b = b0 + src, w.keys = __shfl_sync(FULL_MASK, keys, src), w.row = __shfl_sync(FULL_MASK, row, src);
      w.tiles = key_tiles<GROUPS>(w.keys);
      return true;
    }
  }
  return false;
}
// The next item of the share (false: done).  The whole warp calls.
template <int GROUPS>
__device__ __forceinline__ bool next_item(const DecodeParams &p, Walk &w, Item &it) {
  const int upb = p.pv.Hkv * p.n_hg;
  while (w.left > 0) {
    if (w.b >= p.pv.B) return false;
    if (w.tiles == 0 || w.u >= upb) {
      w.u = 0, w.off = 0;
      if (!walk_next<GROUPS>(p, w)) return false;
      continue;
    }
    const int vt = w.tiles + Shape<GROUPS>::ITEM_TILES, n = min(vt - w.off, w.left);
    it.b = w.b, it.u = w.u, it.keys = w.keys, it.row = w.row, it.tiles = w.tiles;
    it.t0 = max(w.off - Shape<GROUPS>::ITEM_TILES, 0), it.t1 = w.off + n - Shape<GROUPS>::ITEM_TILES;
    it.vstart = w.v - w.off + Shape<GROUPS>::ITEM_TILES;
    w.v += n, w.left -= n, w.off += n;
    if (w.off == vt) ++w.u, w.off = 0;
    if (it.t1 > it.t0) return true;
  }
  return false;
}

// GROUPS = 1: at most four heads; warps 2i and 2i + 1 take 16 keys of the i-th 32 each.  GROUPS = 2: five to
// eight heads in two halves; warp i of either half takes all of the i-th 32 keys.  Both halves decode
// every key, but a warp holds the state of four heads only: one that held eight decoded once, spilled, and
// took 2.2 us a tile against 1.9.
template <int GROUPS, bool FIXED>
__global__ void __maxnreg__(128) k_paged_partial(const DecodeParams p) {
  constexpr int CW = Shape<GROUPS>::CW, TILE = Shape<GROUPS>::TILE, NT = Shape<GROUPS>::NT;
  constexpr int ITEM_TILES = Shape<GROUPS>::ITEM_TILES;
  auto consumers_sync = [] { named_sync1<CW * 32>(); };
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Head &sm = *reinterpret_cast<Head *>(smem_raw);
  Tail &tl = *reinterpret_cast<Tail *>(smem_raw + TAIL_OFF);
  uint32_t *lut = reinterpret_cast<uint32_t *>(smem_raw + LUT_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (FIXED && smem_addr(smem_raw) != RESERVED_SMEM) {  // layout assumption broken: refuse
    if (threadIdx.x == 0) atomicExch(p.pv.status, (int32_t)DEVERR_LAYOUT);
    return;
  }
  if (warp == CW) {
    // ---------------- producer: the CTA's share, then every tile's copies
    if (lane == 0) {
      for (int s = 0; s < NSTAGE; ++s) {
        mbar_init(&sm.full[s], 1);
        mbar_init(&sm.empty[s], CW);
      }
      sm.abort_flag = 0;
      fence_mbar_init();
    }
    pdl_wait();
    const int V = total_tiles<GROUPS>(p, lane, blockIdx.x == 0);
    const int G = min((int)gridDim.x, V);
    Walk w{0, 0, 0, 0, 0, 0, 0, 0};
    if ((int)blockIdx.x < G) {
      w.v = share_start(blockIdx.x, V, G);
      w.left = share_start(blockIdx.x + 1, V, G) - w.v;
      seek<GROUPS>(p, w.v, lane, &w.b, &w.off);
      walk_load<GROUPS>(p, w);
      const int vt = w.tiles + ITEM_TILES;
      w.u = w.off / vt;
      w.off -= w.u * vt;
    }
    if (lane == 0) {
      sm.V = V, sm.G = G;
      *reinterpret_cast<Walk *>(tl.q[0]) = w;
    }
    __syncwarp();
    named_arrive0<NT>();  // the barriers and the share are set up
    const int psh = p.pv.page_shift, P = 1 << psh;
    const bool side = lane >= 16;  // lanes 0-15: K, 16-31: V
    const int seg = lane & 15;
    const uint8_t *pages = side ? p.vp : p.kp;
    int ctr = 0;
    Item it;
    bool ok = true;
    while (ok && next_item<GROUPS>(p, w, it)) {
      const int kvh = it.u / p.n_hg;
      // the page of this lane's segment of tile j
      auto page_of = [&](int j) -> int {
        const int pi = ((j * TILE) >> psh) + seg;
        if (j >= it.t1 || (pi << psh) >= min((j + 1) * TILE, it.keys)) return -1;
        return max(paged_page(p.pv, it.b, pi << psh, !side), 0);
      };
      int pg = page_of(it.t0);
      for (int j = it.t0; j < it.t1; ++j) {
        const int kf = j * TILE, nk = min(TILE, it.keys - kf), s = ctr % NSTAGE;
        const int pg_next = page_of(j + 1);
        const bool up = ctr < NSTAGE || mbar_wait_bounded(&sm.empty[s], ((ctr / NSTAGE) - 1) & 1, WAIT_LIMIT_NS);
        if (!__all_sync(FULL_MASK, up)) {  // (the warp together: the walk takes all its lanes)
          if (lane == 0) {
            atomicExch(&sm.abort_flag, 1);
            atomicExch(p.pv.status, (int32_t)DEVERR_TIMEOUT);
          }
          ok = false;
          break;
        }
        // rows of a tile rounded up to four (16-byte copies; they stay inside the page)
        if (lane == 0) mbar_arrive_expect_tx(&sm.full[s], 2u * ((nk + 3) & ~3) * PG_ROW);
        __syncwarp();
        if (pg >= 0) {
          const int k0 = max((((kf >> psh) + seg) << psh), kf);           // first key of the segment
          const int k1 = min(((k0 >> psh) + 1) << psh, kf + ((nk + 3) & ~3));
          bulk_g2s(stage_at(smem_raw, s + (side ? NSTAGE : 0)) + (k0 - kf) * PG_ROW,
                   pages + paged_row(p.pv, pg, kvh, k0 & (P - 1)), (uint32_t)(k1 - k0) * PG_ROW, &sm.full[s]);
        }
        pg = pg_next;
        ++ctr;
      }
    }
    // Let every issued copy land before the CTA can exit (only matters after a bounded wait
    // gave up; otherwise the consumers have consumed them all).
    if (!ok || *reinterpret_cast<volatile int *>(&sm.abort_flag)) {
      for (int c = (ctr > NSTAGE ? ctr - NSTAGE : 0); c < ctr; ++c)
        (void)mbar_wait_bounded(&sm.full[c % NSTAGE], (c / NSTAGE) & 1, WAIT_LIMIT_NS);
    }
    return;
  }

  // ---------------- consumers: the table (entry b: centroids of nibbles b & 15, b >> 4)
  for (int piece = threadIdx.x; piece < 256 * 8; piece += CW * 32) {
    const int byte = piece >> 3, chunk = piece & 7;  // chunks 0-3: key slots, 4-7: value slots
    const uint32_t *c16 = (chunk & 4) ? p.vc16 : p.kc16;
    const uint32_t lo = (c16[(byte & 15) >> 1] >> (16 * (byte & 1))) & 0xFFFFu;
    const uint32_t hi = (c16[(byte >> 4) >> 1] >> (16 * ((byte >> 4) & 1))) & 0xFFFFu;
    const uint32_t e = lo | (hi << 16);
    uint4 *dst = reinterpret_cast<uint4 *>(lut + byte * 64 + chunk * 8);
    dst[0] = make_uint4(e, e, e, e);
    dst[1] = make_uint4(e, e, e, e);
  }
  pdl_wait();  // the pages, q and the workspace may be written by the previous kernel
  named_sync0<NT>();
  Walk w = *reinterpret_cast<const Walk *>(tl.q[0]);
  const int V = sm.V, G = sm.G;

  const int g = lane >> 2, t = lane & 3;
  const uint32_t lut_base = smem_addr(lut);
  const uint32_t kword = 4u * lane, vword = 128u + 4u * lane;
  const uint32_t klo[2] = {p.klo[0], p.klo[1]}, khi[2] = {p.khi[0], p.khi[1]};
  const uint32_t vlo[2] = {p.vlo[0], p.vlo[1]}, vhi[2] = {p.vhi[0], p.vhi[1]};
  const int grp = GROUPS == 2 && warp >= CW / 2 ? 1 : 0, wi = warp - grp * (CW / 2);
  // Tile row of key k of the warp's 16 (the first of two such blocks, eight rows apart, in a half):
  // rows 16 apart start 16 banks apart, so that the packed words and norms are read without bank conflicts.
  const bool paired = GROUPS == 2 || warp < 2 * (CW / 2);  // (the 15th warp's rows lie together)
  const int r0 = GROUPS == 2 ? 32 * wi : (paired ? 32 * (warp >> 1) + 8 * (warp & 1) : 16 * warp);
  auto row_of = [&](int k) { return paired ? r0 + (k & 7) + 16 * (k >> 3) : r0 + k; };
  const int pk0 = row_of(key_of_row(g)), pk1 = row_of(key_of_row(g + 8)), pat = row_of((t & 1) | ((t & 2) << 2));
  const int hs = g >> 1;
  const int src0 = 4 * t + hs, src1 = 4 * (4 + t) + hs;
  const float lo_sel = (g & 1) ? 1.f : 0.f;

  int ctr = 0;
  Item it, nx;
  bool aborted = false;
  // an item's first q-head and heads; warp h < heads loads head h's row and its angles
  auto heads_of = [&](const Item &i, int &head0, int &GH) {
    const int kvh = p.n_hg == 1 ? i.u : i.u / p.n_hg, hg = i.u - kvh * p.n_hg;
    head0 = kvh * p.gq + hg * p.hpc, GH = min(p.hpc, p.gq - hg * p.hpc);
  };
  uint4 q_raw = make_uint4(0u, 0u, 0u, 0u);
  LaneAngles q_ang;
  auto fetch_q = [&](const Item &i) {
    int head0, GH;
    heads_of(i, head0, GH);
    if (warp >= GH) return;
    q_raw = load_lane4_raw(p.q.data + i.row * p.q.token_bytes + (head0 + warp) * p.q.head_bytes, p.q.dtype, lane);
    if (p.rope.rot_dim) q_ang = rope_angles(lane, p.rope, rope_pos(p.rope, i.keys - 1, p.pv.status, lane == 0));
  };
  bool have = next_item<GROUPS>(p, w, it);
  if (have) fetch_q(it);
  consumers_sync();  // tl.q (the share) has been read
  while (have) {
    int head0, GH;
    heads_of(it, head0, GH);

    if (warp == CW - 1) {  // (it prepares no q)
      const int f = share_of(it.vstart, V, G), n = share_of(it.vstart + it.tiles - 1, V, G) - f + 1;
      if (lane == 0) sm.first = f, sm.n_split = n;
    }
    // ---- q of the item: position rotation, R q, scale, fp16 hi + lo.  The WHT runs in a warp per
    // head; a dense R takes its 64 KB from L2 and two barriers more (1.4 us).
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (warp < GH) {
      lane4_floats(q_raw, p.q.dtype, x);
      if (p.rope.rot_dim) rope_turn(x, lane, p.rope, q_ang);
    }
    if (!p.kfrag) {
      if (warp < GH) {
        wht_lane4(x, p.wht_neg, lane);
        split_q(x, p.qmul * 0.08838834764831845f, tl, warp, lane);
      }
    } else if (warp < 8) {
      uint4 rh[8], rl[8];  // this warp's 16 rows of R
      rot_load(rh, p.kfrag, 0, 0, warp, lane);
      rot_load(rl, p.kfrag, 0, 1, warp, lane);
      rot_put(sm.prep.x, warp, lane, x);
      named_sync2<8 * 32>();
      rot_tile(rh, rl, warp, lane, sm.prep.x, &sm.prep.y[0][0], D + 4);
      named_sync2<8 * 32>();
      if (warp < GH) {
        const float4 v = *reinterpret_cast<const float4 *>(&sm.prep.y[warp][4 * lane]);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        split_q(x, p.qmul, tl, warp, lane);
      }
    }
    consumers_sync();
    uint32_t qb[8][2];
    float qs;
    {
      const int slot = grp * 4 + hs, sw = 2 * g + (t >> 1);
      const uint32_t *qw = tl.q[slot] + (g & 1) * 64 + 16 * t, held = slot < GH ? ~0u : 0u;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) qb[kk][0] = qw[(2 * kk) ^ sw] & held, qb[kk][1] = qw[(2 * kk + 1) ^ sw] & held;
      const int my = grp * 4 + t;  // the head whose scores this lane holds
      qs = my < GH ? tl.qs[my] : 0.f;
    }
    float O[8][4];
    float M = -INFINITY, lsum = 0.f;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) O[mt][0] = O[mt][1] = O[mt][2] = O[mt][3] = 0.f;

    const bool more = next_item<GROUPS>(p, w, nx);  // its lengths are loaded under the tiles
    for (int j = it.t0; j < it.t1; ++j) {
      const int s = ctr % NSTAGE;
      if (!mbar_wait_bounded(&sm.full[s], (ctr / NSTAGE) & 1, WAIT_LIMIT_NS)) {
        if (lane == 0) {
          atomicExch(p.pv.status, (int32_t)DEVERR_TIMEOUT);
          atomicExch(&sm.abort_flag, 1);
        }
        aborted = true;
        break;
      }
      const int nk = min(TILE, it.keys - j * TILE);
      const uint8_t *Ks = stage_at(smem_raw, s), *Vs = stage_at(smem_raw, NSTAGE + s);
#pragma unroll 1
      for (int b8 = 0; b8 < 8 * GROUPS; b8 += 8) {
        if (r0 + b8 >= nk) break;  // the block's first row is its lowest: no valid key
        // ---- scores S^T[16 keys x 8] = K_hat Q^T, two accumulator chains
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
        const int k0 = pk0 + b8, k1 = pk1 + b8;
        const uint8_t *kr0 = Ks + k0 * PG_ROW + 4 + 16 * t;
        const uint8_t *kr1 = Ks + k1 * PG_ROW + 4 + 16 * t;
#pragma unroll
        for (int w4 = 0; w4 < 4; ++w4) {
          uint32_t d0[4], d1[4];
          const uint32_t x0 = ld_u32(kr0 + 4 * w4), x1 = ld_u32(kr1 + 4 * w4);
          decode4<false, FIXED>(lut_base, kword, x0, klo, khi, d0);
          decode4<false, FIXED>(lut_base, kword, x1, klo, khi, d1);
          const uint32_t a0[4] = {d0[0], d1[0], d0[1], d1[1]};
          const uint32_t a1[4] = {d0[2], d1[2], d0[3], d1[3]};
          mma_f16(sa, a0, qb[2 * w4][0], qb[2 * w4][1]);
          mma_f16(sb, a1, qb[2 * w4 + 1][0], qb[2 * w4 + 1][1]);
        }
        // ---- online softmax over the two keys of this lane, head t of each group; the running
        // max is of s + log2(value norm), so that the probability operand 2^7 e^s n_v stays in
        // fp16's range whatever the norms
        const float nk0 = *reinterpret_cast<const float *>(Ks + k0 * PG_ROW);
        const float nk1 = *reinterpret_cast<const float *>(Ks + k1 * PG_ROW);
        const float nv0 = *reinterpret_cast<const float *>(Vs + k0 * PG_ROW);
        const float nv1 = *reinterpret_cast<const float *>(Vs + k1 * PG_ROW);
        const bool ok0 = k0 < nk, ok1 = k1 < nk;
        const float pv0 = ok0 ? nv0 * NORM_FACTOR : 0.f, pv1 = ok1 ? nv1 * NORM_FACTOR : 0.f;
        uint32_t pb[2];
        const float d0 = (sa[0] + sa[1]) + (sb[0] + sb[1]);
        const float d1 = (sa[2] + sa[3]) + (sb[2] + sb[3]);
        const float s0 = ok0 ? d0 * (nk0 * qs) : -INFINITY;
        const float s1 = ok1 ? d1 * (nk1 * qs) : -INFINITY;
        float e0 = exp2_approx(s0 - M), e1 = exp2_approx(s1 - M);
        // An operand past 2^15, a weight past W_MOST (a value of no norm has operand 0, or NaN of an
        // infinite weight, which fmaxf drops), or no maximum yet (e then infinite or NaN): the maximum is
        // raised.  One vote a tile, where the maximum itself takes three exchanges.
        if (__any_sync(FULL_MASK, !(fmaxf(e0 * pv0, e1 * pv1) <= 32768.f) || !(fmaxf(e0, e1) <= W_MOST) ||
                                      M == -INFINITY)) {
          const float u0 = s0 + (ok0 ? fmaxf(log2_approx(nv0), -64.f) : 0.f);
          const float u1 = s1 + (ok1 ? fmaxf(log2_approx(nv1), -64.f) : 0.f);
          float bm = fmaxf(u0, u1);
          bm = fmaxf(bm, __shfl_xor_sync(FULL_MASK, bm, 4));
          bm = fmaxf(bm, __shfl_xor_sync(FULL_MASK, bm, 8));
          bm = fmaxf(bm, __shfl_xor_sync(FULL_MASK, bm, 16)) - W_SHIFT;  // M is the maximum less W_SHIFT
          if (bm > M + RESCALE_SLACK) {  // also taken while M is -inf
            const float half = exp2_approx(0.5f * (M - bm)), alpha = half * half;
            M = bm;
            lsum = lower(lsum, half);
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
              O[mt][0] *= alpha, O[mt][1] *= alpha, O[mt][2] *= alpha, O[mt][3] *= alpha;
          }
          const float Mu = (M == -INFINITY) ? 0.f : M;
          e0 = exp2_approx(s0 - Mu), e1 = exp2_approx(s1 - Mu);
        }
        lsum += e0 + e1;
        p_operand(e0 * pv0, e1 * pv1, src0, src1, lo_sel, pb);
        // ---- O^T[dims x cols] += V_hat^T[dims x keys] P^T
        const uint8_t *va_p = Vs + (pat + b8) * PG_ROW + 4 + 8 * g;  // key a_t; a_t+2, +4, +6 follow
#pragma unroll
        for (int w2 = 0; w2 < 2; ++w2) {
          const uint32_t xa = ld_u32(va_p + 4 * w2), xb = ld_u32(va_p + 2 * PG_ROW + 4 * w2);
          const uint32_t xc = ld_u32(va_p + 4 * PG_ROW + 4 * w2), xd = ld_u32(va_p + 6 * PG_ROW + 4 * w2);
          // byte i of zlo = (low nibble of key a, low nibble of key b) of byte 8g + 4w + i
          const uint32_t zlo_ab = (xa & 0x0F0F0F0Fu) | ((xb << 4) & 0xF0F0F0F0u);
          const uint32_t zhi_ab = ((xa >> 4) & 0x0F0F0F0Fu) | (xb & 0xF0F0F0F0u);
          const uint32_t zlo_cd = (xc & 0x0F0F0F0Fu) | ((xd << 4) & 0xF0F0F0F0u);
          const uint32_t zhi_cd = ((xc >> 4) & 0x0F0F0F0Fu) | (xd & 0xF0F0F0F0u);
          uint32_t r0w[4], r1w[4], r2w[4], r3w[4];
          decode4<false, FIXED>(lut_base, vword, zlo_ab, vlo, vhi, r0w);
          decode4<false, FIXED>(lut_base, vword, zhi_ab, vlo, vhi, r1w);
          decode4<false, FIXED>(lut_base, vword, zlo_cd, vlo, vhi, r2w);
          decode4<false, FIXED>(lut_base, vword, zhi_cd, vlo, vhi, r3w);
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) {
            const uint32_t a[4] = {r0w[jj], r1w[jj], r2w[jj], r3w[jj]};
            mma_f16(O[4 * w2 + jj], a, pb[0], pb[1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[s]);
      ++ctr;
    }
    // A warp that gave up waiting has set the flag before any warp can get here past the
    // same tile, so either every consumer warp enters the merge barriers or none.
    if (aborted || *reinterpret_cast<volatile int *>(&sm.abort_flag)) return;

    have = more;
    if (have) fetch_q(nx);  // under the merge

    // ---- merge the warps' states and write the item's partial
    lsum += __shfl_xor_sync(FULL_MASK, lsum, 4);
    lsum += __shfl_xor_sync(FULL_MASK, lsum, 8);
    lsum += __shfl_xor_sync(FULL_MASK, lsum, 16);
    if (g == 0) sm.mw[warp][t] = M, sm.lw[warp][t] = lsum;
    const int first = sm.first, n_split = sm.n_split;
    const int cta = blockIdx.x;
    float *dst0 = n_split == 1 ? p.whole + ((size_t)it.row * p.Hq + head0) * PROW
                               : p.split + (size_t)(cta * 2 + (cta == first ? 1 : 0)) * 8 * PROW;
    if (threadIdx.x == 0 && cta == first) p.unit[it.b * p.pv.Hkv * p.n_hg + it.u] = first | (n_split << 16);
    consumers_sync();
    {
      // the head's max and sum over its warps: lane (g, t) takes warps g and g + 8 of them
      constexpr int WPG = CW / GROUPS;
      const int wb = grp * WPG;
      const bool has0 = g < WPG, has1 = g + 8 < WPG;
      const float m0 = has0 ? sm.mw[wb + g][t] : -INFINITY, l0 = has0 ? sm.lw[wb + g][t] : 0.f;
      const float m1 = has1 ? sm.mw[wb + g + 8][t] : -INFINITY, l1 = has1 ? sm.lw[wb + g + 8][t] : 0.f;
      float ms = fmaxf(m0, m1);
      ms = fmaxf(ms, __shfl_xor_sync(FULL_MASK, ms, 4));
      ms = fmaxf(ms, __shfl_xor_sync(FULL_MASK, ms, 8));
      ms = fmaxf(ms, __shfl_xor_sync(FULL_MASK, ms, 16));
      // (without a maximum a warp's sum is 0, or NaN where its scores are)
      float ls = (m0 == -INFINITY ? l0 : lower(l0, exp2_approx(0.5f * (m0 - ms)))) +
                 (m1 == -INFINITY ? l1 : lower(l1, exp2_approx(0.5f * (m1 - ms))));
      ls += __shfl_xor_sync(FULL_MASK, ls, 4);
      ls += __shfl_xor_sync(FULL_MASK, ls, 8);
      ls += __shfl_xor_sync(FULL_MASK, ls, 16);
      if (wi == 0 && g == 0) sm.mh[grp * 4 + t] = ms, sm.lh[grp * 4 + t] = ls;
      const float fac = (M == -INFINITY) ? 0.f : exp2_approx(M - ms);
      // rows g and g + 8 of m-tile mt: dims 16g + 2mt, + 1, in blocks of 16 permuted so that the
      // warp's lanes hit 32 banks
      float *orow = &sm.osm[warp][t][16 * g];
      const int sw = 4 * (g >> 1) + t;
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        orow[(2 * mt) ^ sw] = (O[mt][0] + O[mt][1]) * fac;
        orow[(2 * mt + 1) ^ sw] = (O[mt][2] + O[mt][3]) * fac;
      }
      consumers_sync();
      for (int idx = threadIdx.x; idx < GH * D; idx += CW * 32) {
        const int h = idx / D, jd = idx % D, h4 = h & 3, w0 = GROUPS == 2 ? (h >> 2) * WPG : 0;
        const float ms2 = sm.mh[h], ls2 = sm.lh[h];
        float acc = 0.f;
#pragma unroll
        for (int ww = 0; ww < WPG; ++ww) acc += sm.osm[w0 + ww][h4][jd ^ (4 * (jd >> 5) + h4)];
        float *dst = dst0 + h * PROW;
        dst[jd] = (ms2 == -INFINITY) ? 0.f : acc;
        if (jd < 2) dst[D + jd] = jd == 0 ? ms2 : ls2;
      }
      consumers_sync();
    }
    it = nx;
  }
}

// ------------------------------------------------------------------------------ combine
struct CombineParams {
  PagedView pv;
  PagedOut o;
  int Hq, gq, n_hg, hpc, units, grid;
  float inv_vscale;        // 2^W_SHIFT / (2^P_SHIFT * alpha_V)
  const uint4 *vfrag;      // R and R^T of the values
  const float *split, *whole;
  const int32_t *unit;
};

constexpr int CB_WARPS = 8;

// A unit per CTA and turn: warp h merges head h's partials (m* = max m_s, l* = sum l_s
// 2^(m_s - m*), o = sum acc_s 2^(m_s - m*) / l*), the eight warps multiply by R^T, then warp h
// (or pair h) finishes the row.
__global__ void __launch_bounds__(CB_WARPS * 32) k_paged_combine(const CombineParams p) {
  __shared__ RotColumns x;
  __shared__ __align__(16) float y[8][D + 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  uint4 ahi[8], alo[8];  // this warp's 16 rows of R^T
  rot_load(ahi, p.vfrag, 1, 0, warp, lane);
  rot_load(alo, p.vfrag, 1, 1, warp, lane);
  pdl_wait();
  const int upb = p.pv.Hkv * p.n_hg;
  // The CTA's units 32 at a time: a lane finds one's row (idle slots have none, and cost nothing more).
  for (int u0 = blockIdx.x; u0 < p.units; u0 += 32 * gridDim.x) {
    const int of_lane = u0 + lane * gridDim.x;
    int lane_row = -1;
    const int lane_keys = of_lane < p.units ? seq_keys(p.pv, of_lane / upb, &lane_row, false) : 0;
    for (uint32_t todo = __ballot_sync(FULL_MASK, lane_row >= 0); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1, unit = u0 + src * gridDim.x;
      const int row = __shfl_sync(FULL_MASK, lane_row, src), keys = __shfl_sync(FULL_MASK, lane_keys, src);
      const int b = unit / upb, u = unit - b * upb, kvh = u / p.n_hg, hg = u - kvh * p.n_hg;
      const int head0 = kvh * p.gq + hg * p.hpc, GH = min(p.hpc, p.gq - hg * p.hpc);
      float a[4] = {0.f, 0.f, 0.f, 0.f};
      if (warp < GH && keys > 0) {
        const uint32_t info = (uint32_t)p.unit[unit];
        const int first = min((int)(info & 0xFFFFu), p.grid - 1), n = min((int)(info >> 16), p.grid - first);
        float ms = -INFINITY, ls = 0.f;
        for (int s0 = 0; s0 < n; s0 += 8) {
          float m8[8], l8[8];
          float4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int s = min(s0 + i, n - 1);
            const float *src = n == 1 ? p.whole + ((size_t)row * p.Hq + head0 + warp) * PROW
                                      : p.split + (size_t)(((first + s) * 2 + (s == 0 ? 1 : 0)) * 8 + warp) * PROW;
            m8[i] = __ldcg(src + D), l8[i] = __ldcg(src + D + 1);
            v[i] = __ldcg(reinterpret_cast<const float4 *>(src) + lane);
          }
          float mc = -INFINITY;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (s0 + i < n && l8[i] != 0.f) mc = fmaxf(mc, m8[i]);
          if (mc > ms) {
            const float h = (ms == -INFINITY) ? 0.f : exp2f(0.5f * (ms - mc)), f = h * h;
            ls = lower(ls, h);
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] *= f;
            ms = mc;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (s0 + i < n && l8[i] != 0.f) {
              const float h = exp2f(0.5f * (m8[i] - ms)), f = h * h;
              ls += lower(l8[i], h);
              a[0] = fmaf(f, v[i].x, a[0]), a[1] = fmaf(f, v[i].y, a[1]);
              a[2] = fmaf(f, v[i].z, a[2]), a[3] = fmaf(f, v[i].w, a[3]);
            }
          }
        }
        const float f = ls == 0.f ? 0.f : p.inv_vscale / ls;  // (NaN stays)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] *= f;
      }
      rot_put(x, warp, lane, a);
      __syncthreads();
      {
        float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
        rot_mul<true>(acc, ahi, x, lane);
        rot_mul<false>(acc2, alo, x, lane);
        float *d = &y[2 * (lane & 3)][16 * warp + (lane >> 2)];
        d[0] = acc[0] + acc2[0], d[D + 4] = acc[1] + acc2[1];
        d[8] = acc[2] + acc2[2], d[D + 12] = acc[3] + acc2[3];
      }
      __syncthreads();
      if (!p.o.diff.lambda) {
        if (warp < GH) {
          const float4 r = *reinterpret_cast<const float4 *>(&y[warp][4 * lane]);
          const float v4[4] = {r.x, r.y, r.z, r.w};
          store_lane4(p.o.out, p.o.dtype, ((size_t)row * p.Hq + head0 + warp) * D, lane, v4);
        }
      } else if (2 * warp < GH) {
        const float4 r = *reinterpret_cast<const float4 *>(&y[2 * warp][4 * lane]);
        const float4 r2 = *reinterpret_cast<const float4 *>(&y[2 * warp + 1][4 * lane]);
        float v4[4] = {r.x, r.y, r.z, r.w};
        const float w4[4] = {r2.x, r2.y, r2.z, r2.w};
        diff_finish(v4, w4, p.o.diff, row, (head0 >> 1) + warp, lane);
        store_lane4(p.o.out, p.o.dtype, ((size_t)row * (p.Hq / 2) + (head0 >> 1) + warp) * D, lane, v4);
      }
      __syncthreads();  // x and y are free again
    }
  }
}

template <int GROUPS>
cudaError_t launch_partial_ng(const DecodeParams &p, bool fixed, int grid, cudaStream_t st) {
  auto kern = fixed ? k_paged_partial<GROUPS, true> : k_paged_partial<GROUPS, false>;
  cudaError_t e = kernel_smem_attr((const void *)kern, (int)SMEM, true);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(Shape<GROUPS>::NT), SMEM, st, p);
}

struct Layout {
  int hpc, n_hg, grid;
  size_t split, whole, unit, bytes;
};
bool layout(const tq_ctx *k, const PagedView &pv, int Hq, Layout *l) {
  const int gq = Hq / pv.Hkv;
  l->hpc = gq > 4 ? 8 : 4;
  l->n_hg = (gq + l->hpc - 1) / l->hpc;
  l->grid = k->num_sms;
  const int64_t units = (int64_t)pv.B * pv.Hkv * l->n_hg;
  const bool two = l->hpc == 8;
  const int tile = two ? Shape<2>::TILE : Shape<1>::TILE, item = two ? Shape<2>::ITEM_TILES : Shape<1>::ITEM_TILES;
  const int64_t tiles = units * ((pv.max_len + tile - 1) / tile + item);
  if (l->grid > 65535 || tiles > INT32_MAX || (int64_t)pv.n_tokens * Hq > INT32_MAX) return false;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  l->split = 0;
  l->whole = up((size_t)l->grid * 2 * 8 * PROW * 4);
  l->unit = l->whole + up((size_t)pv.n_tokens * Hq * PROW * 4);
  l->bytes = l->unit + up((size_t)units * 4);
  return true;
}

}  // namespace

bool paged_decode_workspace(const tq_ctx *k, const PagedView &pv, int Hq, size_t *bytes) {
  Layout l;
  if (!layout(k, pv, Hq, &l)) return false;
  *bytes = l.bytes;
  return true;
}

cudaError_t launch_paged_decode(const tq_ctx *k, const tq_ctx *v, const PagedView &pv, const uint8_t *kp,
                                const uint8_t *vp, const RowsView &q, int Hq, const RopeView &rope, float scale,
                                const PagedOut &o, void *ws, cudaStream_t st) {
  Layout l;
  if (!layout(k, pv, Hq, &l)) return cudaErrorInvalidValue;
  uint8_t *base = static_cast<uint8_t *>(ws);
  DecodeParams p{};
  p.pv = pv, p.kp = kp, p.vp = vp, p.q = q, p.rope = rope;
  p.Hq = Hq, p.gq = Hq / pv.Hkv, p.n_hg = l.n_hg, p.hpc = l.hpc;
  p.qmul = LOG2E * scale / k->f16.alpha;
  p.kfrag = k->p.rotation == TQ_ROT_DENSE ? k->d_rfrag : nullptr;
  for (int i = 0; i < 4; ++i) p.wht_neg[i] = k->wht_neg[i];
  for (int i = 0; i < 8; ++i) p.kc16[i] = k->f16.c16[i], p.vc16[i] = v->f16.c16[i];
  for (int i = 0; i < 2; ++i) {
    p.klo[i] = k->f16.lo[i], p.khi[i] = k->f16.hi[i];
    p.vlo[i] = v->f16.lo[i], p.vhi[i] = v->f16.hi[i];
  }
  p.split = reinterpret_cast<float *>(base + l.split);
  p.whole = reinterpret_cast<float *>(base + l.whole);
  p.unit = reinterpret_cast<int32_t *>(base + l.unit);
  const bool fixed = k->reserved_smem == (int)RESERVED_SMEM;
  cudaError_t e = l.hpc == 8 ? launch_partial_ng<2>(p, fixed, l.grid, st) : launch_partial_ng<1>(p, fixed, l.grid, st);
  if (e != cudaSuccess) return e;
  CombineParams c{};
  c.pv = pv, c.o = o;
  c.Hq = Hq, c.gq = p.gq, c.n_hg = l.n_hg, c.hpc = l.hpc, c.grid = l.grid;
  c.units = pv.B * pv.Hkv * l.n_hg;
  c.inv_vscale = 1.0f / (exp2f(P_SHIFT - W_SHIFT) * v->f16.alpha);
  c.vfrag = v->d_rfrag;
  c.split = p.split, c.whole = p.whole, c.unit = p.unit;
  int blocks = 1;
  if ((e = kernel_occupancy((const void *)k_paged_combine, CB_WARPS * 32, 0, &blocks)) != cudaSuccess) return e;
  const int most = k->num_sms * blocks;
  return launch_pdl(k_paged_combine, dim3(c.units < most ? c.units : most), dim3(CB_WARPS * 32), 0, st, c);
}

}  // namespace tq
