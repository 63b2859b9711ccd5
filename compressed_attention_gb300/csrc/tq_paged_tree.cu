// Attention of drafted trees over the paged cache on the 5th-generation tensor cores, in two launches.
//
// Node i of a sequence sees the context, its ancestors and itself:
//   out = R_V^T sum_t p_t n_t c_t / sum_t p_t,  p_t = exp(scale n_t <R_K rope(q, context + depth), c_t>),
// with n_t the norms and c_t the centroids of the fp16 table of the packed rows.
// A unit is a sequence's KV head with as many of its nodes as fit R columns (a column is a node's q-head).
// Few columns against long contexts: so the products are laid with the keys in the rows,
//   S^T [128 keys x R] = C_K Q^T,   O^T [128 dims x N] += C_V^T P^T,
// and the time of a tile goes with its 128 keys and its columns, where rows of 128 queries (the chunk kernel's
// form) would compute 128 exponentials a key whatever the tree holds.  (For trees of some hundred columns a KV head that does
// not hold: they are cut into units of 64, which decode every tile again, and the chunk kernel spends about as much
// on a tile of 128 rows as this one on 64 columns; it takes no trees.)  A softmax thread is a key: its norms are two
// scalars, and the sums of weights stay in its registers until the item's end.
//
//   k_tree_partial  persistent, one CTA per SM; the key tiles of all units lie end to end (each unit after a few
//                   empty tiles that stand for its start) and are shared out evenly, as in the paged decode.  An
//                   item is a unit's tiles in one CTA's share.  Specialised warps:
//                     loaders     keys, values: packed tiles, one bulk copy per page, on rings; the keys' loader
//                                 walks the share for all
//                     K decoders  nibbles -> fp16 centroids (byte permutes) into tensor memory, a key per lane:
//                                 the A operand of S^T, without a trip through shared memory
//                     V decoders  the same into 128-byte swizzled tiles, the MN-major A operand of O^T
//                     issuers     one thread for S^T, as far ahead as its buffers go, one for O^T; the first
//                                 one's warp finds the next item's positions
//                     softmax     two groups of four warps on alternate key tiles, each with its own O^T.  An
//                                 item starts with q: rows turned (fp32), times R in bf16 parts (m16n8k16), as fp16 parts
//                                 in the operand's image.  Then S^T from tensor memory, weights against the columns'
//                                 running maxima, P as the MN-major B operand in shared memory.  A maximum is raised
//                                 (and O rescaled) only when a weight would leave the operand's range: one vote a tile.
//   k_tree_combine  the log-sum-exp merge of a column's shares, R^T o on the tensor cores, rounding.
//
// Parts: for bf16 outputs q and P enter as one fp16 each (off by 2^-11 of the value at most); for fp16 and fp32 outputs as hi + lo,
// the lo parts as more columns.  Sums, maxima and O are fp32.
//
// Measured: 8 sequences of 24,000 to 32,768 tokens, 8 nodes each, 32 heads on 8, bf16: 114 us for both launches, 2.2 TB/s of
// packed rows (37 us at the copy rate), 2,100 cycles per 128 keys and SM.  The decoders' byte permutes keep the ALU at 69%
// of its rate, issue 65%, tensor pipe 12%; with the decoders' arithmetic taken out (scratch build, when this took 117) it
// was 99 us, with the copies too 83: what is left is the chain decode -> S -> softmax -> P -> O and its barriers.  Table
// lookups in place of the permutes, deeper packed rings and fewer raise barriers changed nothing.  An item's start and end
// take 9.5 us wherever they are hidden by nothing: one user's 8 nodes on 733 tokens 16.4 us, where an empty kernel takes 3
// and the combine 4; of the 9.5 more than half is q (position, turn, R), a chain of short dependent steps.  R is applied as a
// product under a WHT too, where the single-row decode turns q by a butterfly in the warp.  Positions and ancestors are walks
// along the parents, a load a step, at every item's start: on those 733 tokens a chain of 32, 64 and 128 nodes takes 23, 33
// and 49 us where trees of the same sizes and a few levels take 19, 24 and 31.
#include <math.h>

#include "tq_decode_common.cuh"
#include "tq_paged.cuh"
#include "tq_rotmma.cuh"
#include "tq_tc.cuh"

namespace tq {

namespace {

constexpr int KT = 128;          // keys per tile
// Cost of an item ahead of its tiles (q, the first maxima, the partials), in tiles.  With 6, 8 and 12: 8 sequences towards 32K
// take 115, 114 and 116 us, short chains 34.6, 35.5 and 38.2, mixed trees 33.0, 31.9 and 32.9, wide trees 173, 172 and 171.
constexpr int ITEM_TILES = 8;
constexpr int RAW = KT * PG_ROW; // a packed tile
constexpr int PROW = D + 4;      // floats of a partial: acc[128], max (less W_SHIFT), sum, 2 spare
constexpr int NITEM = 4;         // items known ahead

// R columns of a unit, PARTS fp16 parts of q and P.
template <int R_, int PARTS_>
struct Cfg {
  static constexpr int R = R_, PARTS = PARTS_;
  static constexpr int N = R * PARTS;   // columns of P and O
  // Warps: softmax, K and V decoders, the issuer of O^T, the loaders of keys and values, the issuer of S^T.  Two groups of
  // decoders each, on alternate tiles, where the softmax is quicker than one (8 sequences towards 32K 117 us, with one
  // group 129, before K had three stages); with 64 columns it is not, and takes the registers instead, for a sum per
  // column and 32 scores (four trees of 40 to 64 nodes 172 us, with two groups 206).
  static constexpr int GROUPS = R == 64 ? 1 : 2;
  static constexpr int W_KDEC = 8, W_VDEC = 8 + 4 * GROUPS, W_PV = 8 + 8 * GROUPS, W_LOAD = W_PV + 1, W_S = W_PV + 3;
  static constexpr int THREADS = (W_S + 1) * 32;
  // Spilled, for those registers (stores): R = 32 44 B (one part) and 62 (two), R = 64 300 and 352, all where items start
  // and end and where maxima rise.
  static constexpr int REGS_LAUNCH = GROUPS == 1 ? 96 : 72, REGS_SOFTMAX = GROUPS == 1 ? 144 : 128, REGS_OTHER = GROUPS == 1 ? 64 : 48;
  static_assert(256 * REGS_SOFTMAX + (THREADS - 256) * REGS_OTHER <= THREADS * REGS_LAUNCH, "the launch's registers");
  static constexpr int CH = 32;         // columns a thread takes at a time
  // Stages: packed tiles on their way (more of the values', which the K decoders need for their norms long before
  // the V decoders come to them), decoded K (tensor memory) and V (shared memory), scores, P: what shared and tensor memory
  // hold.  For 32 columns six packed stages against one decoded V less, or half the P, were slower (117 -> 121 to 125 us), a
  // fourth decoded K too (114 -> 117: decoders that run further ahead take the issue slots of what is waited for).
  static constexpr int NRAW_K = N == 32 ? 4 : 2, NRAW_V = 4;
  // A stage of packed tiles always falls to the same group of decoders: copies may land out of order, and a group that
  // had not waited for a stage's last phase could take its parity for the next one's.  The decoded stages (three) and the
  // scores' buffers (five, or three) pass from group to group, so that a waiter meets a buffer's barrier every other phase
  // only.  They hold because one thread issues their products and commits them in order: a commit arrives when all
  // products before it are done.  A K decoder that waits for tile n - NK to be scored has waited for tile n - NK - 2 (its
  // own last tile's wait), so that of the same stage's phase before, tile n - 2 NK, it knows that it has passed: the phase it
  // waits for is the open one or the one just closed, and parity tells them apart.  The same holds for the values'
  // stages (O^T's commits), and for a softmax group at the scores of tile n, which has waited for those of tile n - 2, issued
  // after or with its buffer's last ones, of tile n - NS (NS >= 2).  With another order of commits, or with several issuers, these rings would
  // have to be even as the packed ones are.
  static_assert(GROUPS == 1 || (NRAW_K % 2 == 0 && NRAW_V % 2 == 0), "packed stages");
  static constexpr int NK = N == 128 ? 2 : 3, NV = N == 128 ? 2 : 3;
  static constexpr int NS = N == 128 ? 2 : (R == 64 ? 3 : 5), NP = N == 32 ? 4 : 2;
  static constexpr int NKN = NS + NK + 2;  // tiles whose norms are kept: see Misc
  static constexpr uint32_t TM_S = 0, TM_O = NS * R, TM_K = TM_O + 2 * N;
  static_assert(TM_K + NK * 64 <= 512, "tensor memory");
  // A row of P: 64 bytes where it has 32 columns, else 128 (a second half for more than 64)
  static constexpr uint32_t P_ROW = N == 32 ? 64 : 128, P_BYTES = N * KT * 2;
  static constexpr uint32_t Q_HALF = N * 128, Q_BYTES = 2 * Q_HALF;
  static constexpr uint32_t OFF_V = 0, OFF_P = NV * SW_TILE_BYTES, OFF_Q = OFF_P + NP * P_BYTES;
  static constexpr uint32_t OFF_RAW = OFF_Q + Q_BYTES;
  static constexpr uint32_t OFF_RAW_V = OFF_RAW + NRAW_K * RAW, OFF_MISC = OFF_RAW_V + NRAW_V * RAW;
  static constexpr uint32_t IDESC_S = (1u << 4) | (uint32_t(R >> 3) << 17) | ((128u >> 4) << 24);
  static constexpr uint32_t IDESC_PV = (1u << 4) | (1u << 15) | (1u << 16) | (uint32_t(N >> 3) << 17) | ((128u >> 4) << 24);
  // Byte of P's (key, column): rows of 128 bytes swizzled as the other operands, rows of 64 with 16-byte chunk c of
  // row r at c ^ (r / 2 % 4), eight rows to 512 bytes.
  static __device__ __forceinline__ uint32_t p_at(uint32_t key, uint32_t col) {
    return N == 32 ? key * 64 + (((col >> 3) ^ ((key >> 1) & 3)) << 4) + (col & 7) * 2 : sw128_offset(key, col);
  }
};
// Descriptor of P's 64-byte rows as the MN-major B operand (32 columns): eight rows 512 bytes apart; K-step s of 16 rows
// starts 1024 s bytes in.
__device__ __forceinline__ uint64_t sw64_mn_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1 << 16;                         // leading offset (unused: one atom of columns)
  d |= (uint64_t)((512u >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;                         // descriptor version
  d |= (uint64_t)4 << 61;                         // 64-byte swizzle
  return d;
}

struct TreeView {
  PagedView pv;
  const int32_t *parents;
  int npu, n_qt, gq;  // nodes of a unit, units of a sequence and KV head (for max_q nodes), q-heads per KV head
  uint32_t by_grid;        // floor((2^32 - 1) / CTAs)
  uint32_t by_npu, by_gq;  // floor(2^16 / .) + 1: x / y = x * by_y >> 16 for x < 256, y <= 64
};
__device__ __forceinline__ int node_of(const TreeView &v, int col) { return (int)((uint32_t)col * v.by_gq >> 16); }

// A sequence's nodes and keys.
struct Seq {
  int row, T, base, len;  // first row, nodes taken, slot of node 0 (negative: some have none), keys
};
__device__ __forceinline__ Seq seq_of(const TreeView &v, int b, bool flag) {
  Seq s{0, 0, 0, 0};
  if (b >= v.pv.B) return s;
  const int n = paged_len(v.pv, b, flag);
  int a = b, e = b + 1;
  if (v.pv.cu_q) a = v.pv.cu_q[b], e = v.pv.cu_q[b + 1];
  if (a < 0 || a >= v.pv.n_tokens || e <= a) return s;
  s.row = a, s.base = n - (e - a), s.len = n;
  s.T = min(min(e, v.pv.n_tokens) - a, v.pv.max_q);
  if (flag && e - a > s.T) atomicExch(v.pv.status, (int32_t)DEVERR_SEQLEN);
  return s;
}
__device__ __forceinline__ int seq_tiles(const Seq &s) { return s.T ? (s.len + KT - 1) / KT : 0; }
__device__ __forceinline__ int seq_qt(const TreeView &v, const Seq &s) { return (int)((uint32_t)(s.T + v.npu - 1) * v.by_npu >> 16); }
// Virtual tiles of the sequence.
__device__ __forceinline__ int seq_vtiles(const TreeView &v, const Seq &s) {
  const int t = seq_tiles(s);
  return t ? seq_qt(v, s) * v.pv.Hkv * (t + ITEM_TILES) : 0;
}
// x / y: an estimate in fp32, put right.
__device__ __forceinline__ int div_near(uint32_t x, uint32_t y) {
  uint32_t t = (uint32_t)__fdividef((float)x, (float)y);
  while (t * y > x) --t;
  while ((t + 1) * y <= x) ++t;
  return (int)t;
}
// Units of a sequence lie KV head by KV head, the tiles of nodes of one next to each other.
__device__ __forceinline__ int unit_index(const TreeView &v, int b, int h, int qt) { return (b * v.pv.Hkv + h) * v.n_qt + qt; }

struct Walk {
  int b, u, off, left, v, tiles, units;  // sequence, unit within it, virtual offset within the unit, tiles left, position
  Seq s;
};
struct Item {
  int b, h, qt, t0, t1, tiles, vstart;
  Seq s;
};
// The next sequence with keys, looked for 32 at a time by the whole warp (idle slots may be many).
__device__ __forceinline__ bool walk_next(const TreeView &v, Walk &w) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int b0 = w.b + 1; b0 < v.pv.B; b0 += 32) {
    const Seq s = seq_of(v, b0 + lane, false);
    const uint32_t m = __ballot_sync(FULL_MASK, seq_tiles(s) > 0);
    if (m) {
      const int l = __ffs(m) - 1;
      w.b = b0 + l;
      w.s = Seq{__shfl_sync(FULL_MASK, s.row, l), __shfl_sync(FULL_MASK, s.T, l), __shfl_sync(FULL_MASK, s.base, l),
                __shfl_sync(FULL_MASK, s.len, l)};
      w.tiles = seq_tiles(w.s);
      w.units = seq_qt(v, w.s) * v.pv.Hkv;
      return true;
    }
  }
  return false;
}
// The next item of the share (false: done).  The whole warp calls.
__device__ __forceinline__ bool next_item(const TreeView &v, Walk &w, Item &it) {
  while (w.left > 0) {
    if (w.b >= v.pv.B) return false;
    if (w.tiles == 0 || w.u >= w.units) {
      w.u = 0, w.off = 0;
      if (!walk_next(v, w)) return false;
      continue;
    }
    const int vt = w.tiles + ITEM_TILES, n = min(vt - w.off, w.left), nq = seq_qt(v, w.s);
    it.b = w.b, it.h = div_near(w.u, nq), it.qt = w.u - it.h * nq, it.s = w.s, it.tiles = w.tiles;
    it.t0 = max(w.off - ITEM_TILES, 0), it.t1 = w.off + n - ITEM_TILES;
    it.vstart = w.v - w.off + ITEM_TILES;
    w.v += n, w.left -= n, w.off += n;
    if (w.off == vt) ++w.u, w.off = 0;
    if (it.t1 > it.t0) return true;
  }
  return false;
}
// V virtual tiles over G CTAs in equal shares, as share_start and share_of of the other paged kernels, in 32 bits and
// without divisions (they lie on the way to a CTA's first tile): floor(c V / G) = c (V / G) + floor(c (V % G) / G).
struct Shares {
  uint32_t G, by_grid, q, r;
  float inv;  // G / V
  // x / grid: the product falls short by one at most
  __device__ __forceinline__ uint32_t over_grid(uint32_t x) const {
    const uint32_t t = __umulhi(x, by_grid);
    return t + (x - t * G >= G ? 1 : 0);
  }
  __device__ __forceinline__ void set(int V, const TreeView &v) {
    G = gridDim.x, by_grid = v.by_grid;
    if (V < (int)G) G = V, q = 1, r = 0;
    else q = over_grid(V), r = V - q * G;
    inv = V ? __fdividef((float)G, (float)V) : 0.f;
  }
  __device__ __forceinline__ int start(uint32_t c) const { return c * q + (r ? over_grid(c * r) : 0); }  // (grid < 2^16)
  __device__ __forceinline__ int of(int v) const {  // the CTA whose share holds virtual tile v; the estimate is near
    int c = min((int)((float)v * inv), (int)G - 1);
    while (start(c) > v) --c;
    while (c + 1 < (int)G && start(c + 1) <= v) ++c;
    return c;
  }
};
// One warp: all virtual tiles (flagging bad lengths), then where this CTA's share of them starts.
__device__ __forceinline__ void find_share(const TreeView &v, int lane, Walk &w, Shares &sh) {
  const bool flag = blockIdx.x == 0;
  Seq s;
  int t = 0, sum = 0, b0 = 0;
#pragma unroll 1
  for (int b = lane; b0 < v.pv.B; b += 32, b0 += 32) {
    s = seq_of(v, b, flag);
    t = seq_vtiles(v, s);
    sum += t;
  }
  sh.set(__reduce_add_sync(FULL_MASK, sum), v);
  w = Walk{};
  if (blockIdx.x >= sh.G) return;
  w.v = sh.start(blockIdx.x);
  w.left = sh.start(blockIdx.x + 1) - w.v;
  int base = 0;
#pragma unroll 1
  for (int at = 0;; at += 32) {
    if (b0 > 32) s = seq_of(v, at + lane, false), t = seq_vtiles(v, s);  // (up to 32 sequences: still here)
    int inc = t;
#pragma unroll
    for (int h = 1; h < 32; h <<= 1) {
      const int o = __shfl_up_sync(FULL_MASK, inc, h);
      if (lane >= h) inc += o;
    }
    const uint32_t hit = __ballot_sync(FULL_MASK, base + inc > w.v);
    if (hit || at + 32 >= v.pv.B) {
      const int l = hit ? __ffs(hit) - 1 : 31;
      w.b = at + l;
      w.off = w.v - (base + __shfl_sync(FULL_MASK, inc - t, l));
      w.s = Seq{__shfl_sync(FULL_MASK, s.row, l), __shfl_sync(FULL_MASK, s.T, l), __shfl_sync(FULL_MASK, s.base, l),
                __shfl_sync(FULL_MASK, s.len, l)};
      break;
    }
    base += __shfl_sync(FULL_MASK, inc, 31);
  }
  w.tiles = seq_tiles(w.s);
  w.units = seq_qt(v, w.s) * v.pv.Hkv;
  const int vt = w.tiles + ITEM_TILES;
  w.u = div_near(w.off, vt);
  w.off -= w.u * vt;
}

// ------------------------------------------------------------------------------ attention
struct PartialParams {
  TreeView v;
  const uint8_t *kp, *vp;
  RowsView q;
  RopeView rope;
  int Hq;
  float qmul;          // log2(e) * scale / alpha_K
  const uint4 *kfrag;  // R of the keys
  uint32_t klo[2], khi[2], vlo[2], vhi[2];
  float *split;   // [CTA][2][R] partials of units that several CTAs share
  float *whole;   // [row][Hq] partials of units one CTA finished
  int32_t *unit;  // per unit: first CTA | CTAs << 16
  int late;       // failure test: the first item is known once a wait for it has run out
};

template <int NKN>
struct Misc {
  uint64_t raw_full[2][4], raw_empty[2][4];  // [side][stage]
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_done[5], s_free[5];      // [buffer]
  uint64_t p_ready[4], pv_done[4];    // [buffer of P]
  uint64_t q_known, q_full, o_free, drain[2];
  // Norms of the last tiles, both written by the K decoders, so that the softmax waits for no values.  Tile j is
  // decoded once the scores of tile j - NK are done, and those once the softmax has read the scores, and with them the
  // norms, of tile j - NK - NS.
  float kn[NKN][KT], nv[NKN][KT];
  alignas(16) float nm[2][64];  // [group] minus the running maxima (less W_SHIFT; none yet: 0)
  uint64_t q_src[64];     // the columns' rows of q (0 without a node) and the positions they are turned by
  int q_turn[64];
  float qs[64], qd[64];   // the columns' powers of two (0 without a node), what R q is held times
  uint32_t anc[64][TREE_MAX / 32];  // the unit's nodes: ancestors and the node itself
  float4 move[2][32];     // and, where maxima are raised: what the scores fall by, the square root of O's factor
  float mx[2][64];        // the running maxima, -infinity without one
  float red[2][4][64];    // [group][warp][column]
  float4 end[64];         // per column at the item's end: factors of the groups' O^T, place of the partial (two words)
  uint32_t tmem;
  int abort_flag;
  uint64_t item_full[NITEM], item_empty[NITEM];
  Item item[NITEM];       // found by the keys' loader, one without tiles at the end
  Shares shares;
};

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

// Barrier of softmax group gr (128 threads) that ORs a flag across them.
__device__ __forceinline__ bool group_or(int gr, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(1 + gr)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void prefetch_l1(const void *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }
// Barrier of both softmax groups that ORs a flag across them.
__device__ __forceinline__ bool both_or(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " bar.red.or.pred q, 3, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
// 16 consecutive columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&x)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16_start(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&x)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(x[i]);
  tmem_st16_start(taddr, r);
  tmem_st_wait();
}
// The larger of three, and of a warp's (NaN counts as none).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void acc2(uint64_t &a, uint64_t b) { asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b)); }

template <int R, int PARTS>
__global__ void __launch_bounds__(Cfg<R, PARTS>::THREADS, 1) k_tree_partial(const PartialParams p) {
  using F = Cfg<R, PARTS>;
  constexpr int W_KDEC = F::W_KDEC, W_VDEC = F::W_VDEC, W_PV = F::W_PV, W_LOAD = F::W_LOAD, W_S = F::W_S, THREADS = F::THREADS;
  constexpr int CH = F::CH, NRAW_K = F::NRAW_K, NRAW_V = F::NRAW_V, NK = F::NK, NV = F::NV, NS = F::NS, NP = F::NP, NKN = F::NKN;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t *smem = smem_dyn + ((1024u - (smem_addr(smem_dyn) & 1023u)) & 1023u);
  Misc<NKN> &ms = *reinterpret_cast<Misc<NKN> *>(smem + F::OFF_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) tmem_alloc(smem_addr(&ms.tmem), 512);
  if (tid == 0) {
    for (int s = 0; s < 2; ++s)
      for (int i = 0; i < (s ? NRAW_V : NRAW_K); ++i) mbar_init(&ms.raw_full[s][i], 1), mbar_init(&ms.raw_empty[s][i], s ? 8 : 4);
    for (int i = 0; i < NK; ++i) mbar_init(&ms.k_full[i], 4), mbar_init(&ms.k_empty[i], 1);
    for (int i = 0; i < NV; ++i) mbar_init(&ms.v_full[i], 4), mbar_init(&ms.v_empty[i], 1);
    for (int i = 0; i < NS; ++i) mbar_init(&ms.s_done[i], 1), mbar_init(&ms.s_free[i], 4);
    for (int i = 0; i < NP; ++i) mbar_init(&ms.p_ready[i], 4), mbar_init(&ms.pv_done[i], 1);
    mbar_init(&ms.q_known, 1), mbar_init(&ms.q_full, 8), mbar_init(&ms.o_free, 8);
    mbar_init(&ms.drain[0], 1), mbar_init(&ms.drain[1], 1);
    for (int i = 0; i < NITEM; ++i) mbar_init(&ms.item_full[i], 1), mbar_init(&ms.item_empty[i], THREADS / 32 - 1);
    ms.abort_flag = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();  // (what ran before is done: the combine reads lengths and offsets ahead of its own wait)
  const uint32_t tmem = ms.tmem;
  // Bounded wait, in few instructions (they are on every role's path); fails when another thread has given up.
  auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
    uint64_t t0 = 0;
    while (!mbar_try_wait(bar, parity)) {
      const uint64_t t = global_timer_ns();
      if (!t0) t0 = t;
      if (t - t0 > WAIT_LIMIT_NS) {
        atomicExch(&ms.abort_flag, 1);
        atomicExch(p.v.pv.status, (int32_t)DEVERR_TIMEOUT);
      }
      if (*reinterpret_cast<volatile int *>(&ms.abort_flag)) return false;
    }
    return true;
  };
  Item it;
  bool ok = true;
  uint32_t n_items = 0;
  auto next = [&]() -> bool {  // the next item, as the keys' loader found it
    const uint32_t i = n_items % NITEM;
    if (!__all_sync(FULL_MASK, wait(&ms.item_full[i], (n_items / NITEM) & 1))) return ok = false;
    it = ms.item[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms.item_empty[i]);
    ++n_items;
    return it.t1 > it.t0;
  };
  if (warp >= W_KDEC) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F::REGS_OTHER));
    if (warp == W_LOAD || warp == W_LOAD + 1) {
      // ================ loaders: a warp for the keys, one for the values; a lane per page of a tile
      const int psh = p.v.pv.page_shift, P = 1 << psh, side = warp - W_LOAD;
      const uint8_t *pages = side ? p.vp : p.kp;
      Walk w;
      if (!side) {
        Shares sh;
        find_share(p.v, lane, w, sh);
        if (lane == 0) ms.shares = sh;
      }
      auto publish = [&]() -> bool {  // the keys' loader walks its share for all
        const uint32_t i = n_items % NITEM;
        if (!next_item(p.v, w, it)) it.t0 = it.t1 = 0;
        if (p.late && n_items == 0)
          for (const uint64_t t0 = global_timer_ns();
               !*reinterpret_cast<volatile int *>(&ms.abort_flag) && global_timer_ns() - t0 < 2 * WAIT_LIMIT_NS;) {
          }
        if (n_items >= NITEM && !__all_sync(FULL_MASK, wait(&ms.item_empty[i], ((n_items / NITEM) - 1) & 1))) return ok = false;
        if (lane == 0) {
          ms.item[i] = it;
          mbar_arrive(&ms.item_full[i]);
        }
        __syncwarp();
        ++n_items;
        return it.t1 > it.t0;
      };
      const uint32_t nr = side ? NRAW_V : NRAW_K, raw = side ? F::OFF_RAW_V : F::OFF_RAW;
      uint32_t n = 0, s = 0, turn = 0;  // tiles loaded; the next one's stage, and rounds of the stages
      while (ok && (side ? next() : publish())) {
        auto page_of = [&](int j) -> int {
          const int pi = ((j * KT) >> psh) + lane;
          if (j >= it.t1 || lane >= 8 || (pi << psh) >= min((j + 1) * KT, it.s.len)) return -1;
          return max(paged_page(p.v.pv, it.b, pi << psh, !side), 0);
        };
        int pg = page_of(it.t0);
        for (int j = it.t0; ok && j < it.t1; ++j, ++n) {
          const int kf = j * KT, nk4 = (min(KT, it.s.len - kf) + 3) & ~3;
          const int pg_next = page_of(j + 1);
          if (turn && !(ok = __all_sync(FULL_MASK, wait(&ms.raw_empty[side][s], (turn - 1) & 1)))) break;
          // rows of a tile rounded up to four (16-byte copies; they stay inside the page)
          if (lane == 0) mbar_arrive_expect_tx(&ms.raw_full[side][s], nk4 * PG_ROW);
          __syncwarp();
          if (pg >= 0) {
            const int k0 = max((((kf >> psh) + lane) << psh), kf), k1 = min(((k0 >> psh) + 1) << psh, kf + nk4);
            bulk_g2s(smem + raw + s * RAW + (k0 - kf) * PG_ROW,
                     pages + paged_row(p.v.pv, pg, it.h, k0 & (P - 1)), (uint32_t)(k1 - k0) * PG_ROW, &ms.raw_full[side][s]);
          }
          pg = pg_next;
          if (++s == nr) s = 0, ++turn;
        }
      }
      // after a failed wait: let the copies in flight land before the CTA ends
      if (*reinterpret_cast<volatile int *>(&ms.abort_flag))
        for (uint32_t c = n > nr ? n - nr : 0; c < n; ++c)
          (void)mbar_wait_bounded(&ms.raw_full[side][c % nr], (c / nr) & 1, WAIT_LIMIT_NS);
    } else if (warp < W_PV) {
      // ================ decoders: one or two groups of four warps for the keys, as many for the values, the two on
      // alternate tiles; thread = key of the tile
      const int row = tid & 127;
      const bool side = warp >= W_VDEC;
      uint32_t lo2[2], hi2[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) lo2[i] = side ? p.vlo[i] : p.klo[i], hi2[i] = side ? p.vhi[i] : p.khi[i];
      const uint32_t tK = tmem + ((uint32_t)((warp & 3) * 32) << 16) + F::TM_K;
      const uint32_t to_v = smem_addr(smem + F::OFF_V) + row * 128 + 16 * (row & 7);  // chunk 0 of the row
      uint32_t n = 0;
      while (ok && next()) {
        for (int j = it.t0; ok && j < it.t1; ++j, ++n) {
          if (F::GROUPS == 2 && (n & 1) != (uint32_t)((warp >> 2) & 1)) continue;
          const uint32_t rv = n % NRAW_V, rs = side ? rv : n % NRAW_K, ns = side ? NV : NK, st = n % ns;
          if (n >= ns) ok = wait(side ? &ms.v_empty[st] : &ms.k_empty[st], ((n / ns) - 1) & 1);
          if (ok) ok = wait(&ms.raw_full[side][rs], (n / (side ? NRAW_V : NRAW_K)) & 1);
          if (!(ok = __all_sync(FULL_MASK, ok))) break;
          const uint32_t *src = reinterpret_cast<const uint32_t *>(smem + (side ? F::OFF_RAW_V : F::OFF_RAW) + rs * RAW + row * PG_ROW);
          // Short loops (the warps of an SM run six different ones), the next words loaded ahead of the stores of these.
          if (side) {
            const uint32_t to = to_v + st * SW_TILE_BYTES;
            uint32_t word[4], next[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) word[i] = src[1 + i];
#pragma unroll 1
            for (int q4 = 0; q4 < 4; ++q4) {
#pragma unroll
              for (int i = 0; i < 4; ++i) next[i] = src[1 + 4 * min(q4 + 1, 3) + i];
              // chunk 4 (q4 % 2) + i of half q4 / 2, at its place ^ (row % 8)
              const uint32_t at = (to + (q4 >> 1) * SW_HALF_BYTES) ^ (64u * (q4 & 1));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t d[4];
                decode8<0x5140u, 0x7362u>(word[i], lo2, hi2, d);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (16u * i)), "r"(d[0]), "r"(d[1]), "r"(d[2]), "r"(d[3]) : "memory");
                word[i] = next[i];
              }
            }
            fence_async_smem();
          } else {
            tc_fence_after();  // the product that read the stage
#pragma unroll 1
            for (int q2 = 0; q2 < 4; ++q2) {
              uint32_t d[16];
#pragma unroll
              for (int ch = 0; ch < 4; ++ch) {
                uint32_t x[4];
                decode8<0x5140u, 0x7362u>(src[1 + 4 * q2 + ch], lo2, hi2, x);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[4 * ch + e] = x[e];
              }
              tmem_st16_start(tK + 64 * st + 16 * q2, d);
            }
            tmem_st_wait();
            const bool live = j * KT + row < it.s.len;
            ms.kn[n % NKN][row] = live ? __uint_as_float(src[0]) : 0.f;
            ok = __all_sync(FULL_MASK, wait(&ms.raw_full[1][rv], (n / NRAW_V) & 1));
            if (!ok) break;
            ms.nv[n % NKN][row] = live ? *reinterpret_cast<const float *>(smem + F::OFF_RAW_V + rv * RAW + row * PG_ROW) : 0.f;
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(side ? &ms.v_full[st] : &ms.k_full[st]), mbar_arrive(&ms.raw_empty[side][rs]);
            if (!side) mbar_arrive(&ms.raw_empty[1][rv]);
          }
        }
      }
    } else if (warp == W_S) {
      // ================ issuer of the scores, as far ahead as their buffers go
      const bool lead = elect_lane();
      const uint32_t tb = __shfl_sync(FULL_MASK, tmem, 0), tS = tb + F::TM_S, tK = tb + F::TM_K;
      const uint64_t dq = sw128_desc(smem_addr(smem + F::OFF_Q));
      uint32_t n = 0, items = 0;
      bool issued = false;
      while (ok && next()) {
        // where the columns' rows of q lie and their positions: found ahead of the softmax warps, which are still on
        // the last item, with the rows and the angles sent for
        const int n0 = it.qt * p.v.npu, cols = min(it.s.T - n0, p.v.npu) * p.v.gq;
#pragma unroll 1
        for (int c = lane; c < R; c += 32) {
          const int local = node_of(p.v, c), node = n0 + local;
          uint64_t src = 0;
          int turn = 0;
          if (c < cols && it.s.base + node >= 0) {
            const uint8_t *row = p.q.data + (it.s.row + node) * p.q.token_bytes + (it.h * p.v.gq + c - local * p.v.gq) * p.q.head_bytes;
            src = (uint64_t)(uintptr_t)row;
            prefetch_l1(row), prefetch_l1(row + 128);
            if (p.q.dtype == TQ_DTYPE_F32) prefetch_l1(row + 256), prefetch_l1(row + 384);
            if (p.rope.rot_dim) {  // (a walk per column: see the deep chains in the header)
              turn = rope_pos(p.rope, tree_pos(p.v.pv, p.v.parents, it.b, it.s.row + node, it.s.base + node, true), p.v.pv.status, true);
              const size_t at = (size_t)turn * (p.rope.rot_dim >> 1);
              prefetch_l1(p.rope.cos_t + at), prefetch_l1(p.rope.sin_t + at);
              if (p.rope.rot_dim == 128) prefetch_l1(p.rope.cos_t + at + 32), prefetch_l1(p.rope.sin_t + at + 32);
            }
          }
          ms.q_src[c] = src, ms.q_turn[c] = turn;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.q_known);
        ok = __all_sync(FULL_MASK, wait(&ms.q_full, items & 1));
        for (int j = it.t0; ok && j < it.t1; ++j, ++n) {
          const uint32_t st = n % NK, sb = n % NS;
          if (n >= NS) ok = wait(&ms.s_free[sb], ((n / NS) - 1) & 1);
          if (ok) ok = wait(&ms.k_full[st], (n / NK) & 1);
          if (!(ok = __all_sync(FULL_MASK, ok))) break;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
              for (int s = 0; s < 8; ++s)
                umma_ts<F::IDESC_S>(tS + R * sb, tK + 64 * st + 8 * s,
                                    desc_step(dq, (s >> 2) * F::Q_HALF + part * R * 128 + (s & 3) * 32), (part || s) ? 1u : 0u);
            umma_commit(&ms.s_done[sb]);
            umma_commit(&ms.k_empty[st]);
          }
          __syncwarp();
          issued = true;
        }
        ++items;
      }
      if (issued && lead && *reinterpret_cast<volatile int *>(&ms.abort_flag))
        umma_commit(&ms.drain[0]), (void)mbar_wait_bounded(&ms.drain[0], 0, WAIT_LIMIT_NS);
    } else if (warp == W_PV) {
      // ================ issuer of O^T
      const bool lead = elect_lane();
      const uint32_t tO = __shfl_sync(FULL_MASK, tmem, 0) + F::TM_O;
      const uint64_t dv = sw128_mn_desc(smem_addr(smem + F::OFF_V)), dp = F::N == 32 ? sw64_mn_desc(smem_addr(smem + F::OFF_P)) : sw128_mn_desc(smem_addr(smem + F::OFF_P));
      uint32_t n = 0, items = 0;
      bool issued = false;
      while (ok && next()) {
        for (int j = it.t0; ok && j < it.t1; ++j, ++n) {
          const uint32_t vs = n % NV, ps = n % NP;
          ok = wait(&ms.p_ready[ps], (n / NP) & 1);
          if (ok) ok = wait(&ms.v_full[vs], (n / NV) & 1);
          if (ok && j == it.t0 && items) ok = wait(&ms.o_free, (items - 1) & 1);
          if (!(ok = __all_sync(FULL_MASK, ok))) break;
          tc_fence_after();
          if (lead) {
            const uint64_t a = desc_step(dv, vs * SW_TILE_BYTES), b = desc_step(dp, ps * F::P_BYTES);
#pragma unroll
            for (int s = 0; s < 8; ++s)  // (each group's first tile of the item starts its accumulator)
              umma<F::IDESC_PV>(tO + F::N * (n & 1), desc_step(a, 2048 * s), desc_step(b, 16 * F::P_ROW * s), (j >= it.t0 + 2 || s) ? 1u : 0u);
            umma_commit(&ms.pv_done[ps]);
            umma_commit(&ms.v_empty[vs]);
          }
          __syncwarp();
          issued = true;
        }
        ++items;
      }
      if (issued && lead && *reinterpret_cast<volatile int *>(&ms.abort_flag))
        umma_commit(&ms.drain[1]), (void)mbar_wait_bounded(&ms.drain[1], 0, WAIT_LIMIT_NS);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F::REGS_SOFTMAX));
    // ================ softmax: group gr takes the tiles n with n % 2 == gr, thread = key
    const int gr = warp >> 2, key = tid & 127, wq = warp & 3;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + F::TM_S, tO = tmem + lane_off + F::TM_O + F::N * gr;
    float *const nm = ms.nm[gr];
    float4 *const mv = ms.move[gr];
    uint32_t n = 0;  // tiles before the item
    for (uint32_t items = 0;; ++items) {
      // The eight warps meet at named barriers, so they leave together or not at all: a warp that found no item left,
      // or gave up while another may still have seen one come, says so in the vote that the others take next, below.  (One
      // vote for both: 80 B more of spills, eight sequences towards 32K 114 -> 119 us, wide trees 172 -> 203.)
      if (!next()) {
        (void)both_or(true);
        break;
      }
      const int unit = unit_index(p.v, it.b, it.h, it.qt), n0 = it.qt * p.v.npu;
      const int cols = min(it.s.T - n0, p.v.npu) * p.v.gq;  // columns with a node
      // ---- q: rows turned by their nodes' positions, split into bf16 parts in P's buffers (free between items),
      // times R on the tensor cores (m16n8k16, three products of parts), as fp16 parts in the image of the operand
      {
        constexpr int RW = R / 8;  // columns of a warp
        uint8_t *const xs = smem + F::OFF_P;  // bf16 hi of the columns, then lo; 16-byte chunk c of column r at c ^ (r % 8)
        ok = __all_sync(FULL_MASK, wait(&ms.q_known, items & 1));
        if (both_or(!ok)) break;
        constexpr int W = 2;  // rows at a time (one: short chat 0.5 us more; four spill: four wide trees 30 us more)
        uint64_t src[W], src_next[W];
        uint4 raw[W], raw_next[W];
        LaneAngles an[W], an_next[W];
        auto fetch = [&](int i) {  // the next rows, while some are worked on
#pragma unroll
          for (int r = 0; r < W; ++r) {
            src_next[r] = ms.q_src[warp * RW + i + r];
            raw_next[r] = make_uint4(0u, 0u, 0u, 0u);
            if (src_next[r]) raw_next[r] = load_lane4_raw(reinterpret_cast<const uint8_t *>((uintptr_t)src_next[r]), p.q.dtype, lane);
            if (p.rope.rot_dim) an_next[r] = rope_angles(lane, p.rope, ms.q_turn[warp * RW + i + r]);
          }
        };
        fetch(0);
#pragma unroll 1
        for (int i = 0; i < RW; i += W) {
          float x[W][4], big[W];
#pragma unroll
          for (int r = 0; r < W; ++r) src[r] = src_next[r], raw[r] = raw_next[r], an[r] = an_next[r];
          if (i + W < RW) fetch(i + W);
#pragma unroll
          for (int r = 0; r < W; ++r) lane4_floats(raw[r], p.q.dtype, x[r]);
          if (p.rope.rot_dim) {
#pragma unroll
            for (int r = 0; r < W; ++r) rope_turn(x[r], lane, p.rope, an[r]);
          }
#pragma unroll
          for (int r = 0; r < W; ++r) {
            big[r] = fmaxf(fmaxf(fabsf(x[r][0]), fabsf(x[r][1])), fmaxf(fabsf(x[r][2]), fabsf(x[r][3])));
            big[r] = __uint_as_float(__reduce_max_sync(FULL_MASK, __float_as_uint(big[r])));  // ordered like the floats
          }
#pragma unroll
          for (int r = 0; r < W; ++r) {
            const int c = warp * RW + i + r;
            // R q is at most sqrt(128) times the largest element: held times a power of two that brings that to
            // [2^10, 2^11); times none where it lies between, of ordinary size, so that one part drops what is below
            // 2^-14 of the row's norm, two parts what is below 2^-20 of it.
            const float m = big[r] * fabsf(p.qmul);
            const int e = m >= (PARTS == 2 ? 0x1p-4f : 0x1p-8f) && m < 0x1p11f ? 0 : scale_exp(m) + 3;
            if (lane == 0) ms.qs[c] = src[r] ? pow2i(e) : 0.f, ms.qd[c] = p.qmul * pow2i(-e);
            uint32_t hi[2], lo[2];
            float f[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              hi[k] = pack_bf162(x[r][2 * k], x[r][2 * k + 1]);
              f[2 * k] = __uint_as_float(hi[k] << 16), f[2 * k + 1] = __uint_as_float(hi[k] & 0xFFFF0000u);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = isinf(f[k]) ? x[r][k] = 0.f : f[k];  // an infinite part has no rest
#pragma unroll
            for (int k = 0; k < 2; ++k) lo[k] = pack_bf162(x[r][2 * k] - f[2 * k], x[r][2 * k + 1] - f[2 * k + 1]);
            uint8_t *dst = xs + c * 256 + (((lane >> 1) ^ (c & 7)) << 4) + 8 * (lane & 1);
            *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2 *>(dst + R * 256) = make_uint2(lo[0], lo[1]);
          }
        }
        // whom the nodes see of one another: only a share with the last tiles asks
        if (it.t1 * KT > it.s.base && tid < p.v.npu) {
          uint32_t word[TREE_MAX / 32] = {};
          for (int m = n0 + tid < it.s.T ? n0 + tid : -1; m >= 0; m = tree_parent(p.v.parents, it.s.row, m, p.v.pv.status, true)) {
#pragma unroll
            for (int i = 0; i < TREE_MAX / 32; ++i) word[i] |= (m >> 5) == i ? 1u << (m & 31) : 0u;
          }
          *reinterpret_cast<uint4 *>(ms.anc[tid]) = make_uint4(word[0], word[1], word[2], word[3]);
        }
        uint4 rh[8], rl[8];  // this warp's 16 rows of R (sooner, they would take the registers of the rows of q)
        rot_load(rh, p.kfrag, 0, 0, warp, lane), rot_load(rl, p.kfrag, 0, 1, warp, lane);
        (void)both_or(false);
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll 1
        for (int c0 = 0; c0 < R; c0 += 8) {
          // No node: zeros, in this warp's 16 dims of eight columns two 16-byte chunks of each (chains of 5 columns 36.2 ->
          // 35.3 us; with 64 columns, mostly live, the test costs more than it saves: 171 -> 174).
          if (R == 32 && c0 >= cols) {
            const int c = c0 + (lane & 7), ch = 2 * (warp & 3) + ((lane >> 3) & 1), part = lane >> 4;
            if (part < PARTS)
              *reinterpret_cast<uint4 *>(smem + F::OFF_Q + (warp >> 2) * F::Q_HALF + (part * R + c) * 128 + ((ch ^ (c & 7)) << 4)) =
                  make_uint4(0u, 0u, 0u, 0u);
            continue;
          }
          float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
          const uint8_t *col = xs + (c0 + g) * 256 + 4 * t4;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t o0 = (uint32_t)((2 * k) ^ g) << 4, o1 = (uint32_t)((2 * k + 1) ^ g) << 4;
            const uint32_t h0 = *reinterpret_cast<const uint32_t *>(col + o0), h1 = *reinterpret_cast<const uint32_t *>(col + o1);
            const uint32_t l0 = *reinterpret_cast<const uint32_t *>(col + R * 256 + o0), l1 = *reinterpret_cast<const uint32_t *>(col + R * 256 + o1);
            mma_bf16(acc, rh[k], h0, h1), mma_bf16(acc2, rh[k], l0, l1), mma_bf16(acc2, rl[k], h0, h1);
          }
          // dims 16 warp + g and + 8, columns c0 + 2 t4 and the next
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int c = c0 + 2 * t4 + i;
            const float mul = ms.qd[c];
            const float a = (acc[i] + acc2[i]) * mul, b = (acc[2 + i] + acc2[2 + i]) * mul;
            uint32_t hi, lo;
            split_half2(a, b, hi, lo);
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
              const uint32_t w = part ? lo : hi;
              uint8_t *dst = smem + F::OFF_Q + (warp >> 2) * F::Q_HALF + (part * R + c) * 128;
              const int ch = 2 * (warp & 3);
              *reinterpret_cast<uint16_t *>(dst + ((ch ^ (c & 7)) << 4) + 2 * g) = (uint16_t)w;
              *reinterpret_cast<uint16_t *>(dst + (((ch + 1) ^ (c & 7)) << 4) + 2 * g) = (uint16_t)(w >> 16);
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.q_full);
      }
      // no column has a maximum yet; those without a node keep 0
      bool scale = false;
      if (key < R) {
        const float sc = ms.qs[key];
        nm[key] = 0.f;
        ms.mx[gr][key] = sc == 0.f ? 0.f : -INFINITY;
        scale = sc != 0.f && sc != 1.f;
      }
      bool fresh = true;  // some column has no maximum yet
      uint64_t l2[R / 2];
#pragma unroll
      for (int i = 0; i < R / 2; ++i) l2[i] = 0;
      const bool scaled = group_or(gr, scale);  // some column's q is held times a power of two
      const int tiles = it.t1 - it.t0;
      const int first_m = (n & 1) == (uint32_t)gr ? 0 : 1;
      bool held = false;  // O^T holds something of the item
      for (int m = first_m; m < tiles; m += 2) {
        const uint32_t c = n + m, sb = c % NS, ps = c % NP;
        const int t = (it.t0 + m) * KT + key, j = t - it.s.base;
        ok = wait(&ms.s_done[sb], (c / NS) & 1);
        if (ok && c >= NP) ok = wait(&ms.pv_done[ps], ((c / NP) - 1) & 1);  // the P buffer is free
        ok = __all_sync(FULL_MASK, ok);
        tc_fence_after();
        const float kn = ms.kn[c % NKN][key], nv = ms.nv[c % NKN][key], nvf = nv * NORM_FACTOR;
        const uint64_t kn2 = pk2(kn, kn), nvf2 = pk2(nvf, nvf);
        // a score past this leaves the operand's range (2^15), or its weight passes W_MOST
        const float most = fminf(15.f - log2_approx(nvf), 96.f);
        const bool whole = (it.t0 + m + 1) * KT <= it.s.base;  // every column sees every key of the tile
        uint32_t see[R / 32];
#pragma unroll
        for (int i = 0; i < R / 32; ++i) see[i] = ~0u;
        if (!whole && j >= 0) {  // a node's key: the columns of the nodes that have it among their ancestors
          uint64_t bits = 0;
          if (t < it.s.len && j < TREE_MAX) {
            const uint64_t node_cols = p.v.gq < 64 ? (1ull << p.v.gq) - 1 : ~0ull;
#pragma unroll 1
            for (int i = 0, c2 = 0; c2 < cols; ++i, c2 += p.v.gq)
              if ((ms.anc[i][j >> 5] >> (j & 31)) & 1u) bits |= node_cols << c2;
          }
#pragma unroll
          for (int i = 0; i < R / 32; ++i) see[i] = (uint32_t)(bits >> (32 * i));
        }
        bool some = false;
        uint8_t *const pb = smem + F::OFF_P + ps * F::P_BYTES;
#pragma unroll
        for (int cc = 0; cc < R; cc += CH) {
          const uint32_t bits = see[cc / 32];
          // scores less the running maxima, and the largest
          float d[CH], top = -INFINITY;
          tmem_ld32(tS + R * sb + cc, d);
          if (cc + CH == R) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.s_free[sb]);
          }
          if (scaled) {
#pragma unroll
            for (int e = 0; e < CH; ++e) d[e] *= ms.qs[cc + e];
          }
#pragma unroll
          for (int e = 0; e < CH; e += 2) {
            const float2 x = *reinterpret_cast<const float2 *>(&nm[cc + e]);
            upk2(fma2(pk2(d[e], d[e + 1]), kn2, pk2(x.x, x.y)), d[e], d[e + 1]);
          }
          if (!whole) {
#pragma unroll
            for (int e = 0; e < CH; ++e) d[e] = (bits >> e) & 1u ? d[e] : -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < CH; e += 2) top = max3(top, d[e], d[e + 1]);
          if (group_or(gr, fresh || top > most || !ok)) {
            // ---- the columns' maxima over the tile's keys of score + log2(value norm); raise those that need it
            if (group_or(gr, !ok)) {
              ok = false;
              break;
            }
            const float lv = fmaxf(log2_approx(nv), -64.f);
#pragma unroll
            for (int e = 0; e < CH; ++e) {
              const float u = warp_max(d[e] + lv);
              if (lane == e) ms.red[gr][wq][e] = u;
            }
            (void)group_or(gr, false);
            bool none = false, raised = false;
            if (key < CH) {
              const int col = cc + key;
              const float bm = fmaxf(fmaxf(ms.red[gr][0][key], ms.red[gr][1][key]),
                                     fmaxf(ms.red[gr][2][key], ms.red[gr][3][key])) - W_SHIFT;
              const float old = ms.mx[gr][col];
              float by = 0.f, root = 1.f;  // the maximum rises by `by` (from 0 without one)
              if (bm > (old == -INFINITY ? -INFINITY : RESCALE_SLACK)) {
                by = bm;
                ms.mx[gr][col] = old == -INFINITY ? bm : old + bm;
                nm[col] = -ms.mx[gr][col];
                raised = old != -INFINITY;
                if (raised) root = exp2_approx(-0.5f * by);
              } else {
                none = old == -INFINITY;
              }
              float *x = reinterpret_cast<float *>(&mv[col >> 1]);
              x[col & 1] = by, x[2 + (col & 1)] = root;
            }
            if (group_or(gr, none)) some = true;
#pragma unroll
            for (int e = 0; e < CH; e += 2) {
              const float4 x = mv[(cc + e) >> 1];
              d[e] -= x.x, d[e + 1] -= x.y;
            }
            if (group_or(gr, raised)) {
#pragma unroll
              for (int e = 0; e < CH; e += 2) {
                const float4 x = mv[(cc + e) >> 1];
                const uint64_t f2 = pk2(x.z, x.w);
                l2[(cc + e) / 2] = mul2(mul2(l2[(cc + e) / 2], f2), f2);
              }
              if (held) {
                // O^T is whole once the group's last product is done
                ok = __all_sync(FULL_MASK, wait(&ms.pv_done[(c - 2) % NP], ((c - 2) / NP) & 1));
                if (group_or(gr, !ok)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
#pragma unroll
                for (int at = 0; at < PARTS * CH; at += 16) {
                  float o[16];
                  const int col = cc + at % CH;
                  tmem_ld16(tO + at / CH * R + col, o);
#pragma unroll
                  for (int e = 0; e < 16; e += 2) {
                    const float4 x = mv[(col + e) >> 1];
                    o[e] *= x.z * x.z, o[e + 1] *= x.w * x.w;
                  }
                  tmem_st16(tO + at / CH * R + col, o);
                }
              }
            }
          }
          // ---- weights, their sums and the operand P
#pragma unroll
          for (int e = 0; e < CH; e += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const uint64_t e2 = pk2(exp2_approx(d[e + i]), exp2_approx(d[e + i + 1]));
              acc2(l2[(cc + e + i) / 2], e2);
              float p0, p1;
              upk2(mul2(e2, nvf2), p0, p1);
              if (PARTS == 2) split_half2(p0, p1, hi[i / 2], lo[i / 2]);
              else hi[i / 2] = pack_half2(p0, p1);
            }
            *reinterpret_cast<uint4 *>(pb + F::p_at(key, cc + e)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (PARTS == 2) *reinterpret_cast<uint4 *>(pb + F::p_at(key, R + cc + e)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        if (!ok) break;
        // A norm that is not finite makes NaN of a weight of 0 too: not for the columns that do not see the key.
        if (!whole && !(fabsf(nvf) < INFINITY)) {
#pragma unroll 1
          for (int c2 = 0; c2 < R * PARTS; ++c2) {
            const int col = c2 % R;
            if (!(((R == 64 && col >= 32 ? see[R / 32 - 1] : see[0]) >> (col & 31)) & 1u))
              *reinterpret_cast<uint16_t *>(pb + F::p_at(key, c2)) = 0;
          }
        }
        fresh = some;
        held = true;
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_ready[ps]);
      }
      n += tiles;

      // ---- end of the item: the groups' states merged; O^T: thread = dim
      if (ok && held) {  // the group's last tile
        const uint32_t c = n - 1 - (((n - 1) ^ gr) & 1);
        ok = __all_sync(FULL_MASK, wait(&ms.pv_done[c % NP], (c / NP) & 1));
      }
#pragma unroll
      for (int cc = 0; cc < R; cc += 32) {  // sums over the warp's keys: column cc + l to lane l
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; e += 2) upk2(l2[(cc + e) / 2], x[e], x[e + 1]);
#pragma unroll
        for (int h = 16; h >= 1; h >>= 1) {
          const bool up = lane & h;
#pragma unroll
          for (int e = 0; e < h; ++e) {
            const float mine = up ? x[e + h] : x[e], other = up ? x[e] : x[e + h];
            x[e] = mine + __shfl_xor_sync(FULL_MASK, other, h);
          }
        }
        ms.red[gr][wq][cc + lane] = x[0];
      }
      tc_fence_before();
      if (both_or(!ok)) break;
      tc_fence_after();
      const int first = ms.shares.of(it.vstart), n_split = ms.shares.of(it.vstart + it.tiles - 1) - first + 1, cta = blockIdx.x;
      if (tid == 0 && cta == first) p.unit[unit] = first | (n_split << 16);
      if (tid < cols) {
        auto sum = [&](int g2) {
          return (ms.red[g2][0][tid] + ms.red[g2][1][tid]) + (ms.red[g2][2][tid] + ms.red[g2][3][tid]);
        };
        const float m0 = ms.mx[0][tid], m1 = ms.mx[1][tid], mx = fmaxf(m0, m1), l0 = sum(0), l1 = sum(1);
        const float f0 = m0 == -INFINITY ? 0.f : exp2_approx(m0 - mx), f1 = m1 == -INFINITY ? 0.f : exp2_approx(m1 - mx);
        const int local = node_of(p.v, tid);
        float *dst = n_split > 1 ? p.split + ((size_t)(cta * 2 + (cta == first ? 1 : 0)) * R + tid) * PROW
                                 : p.whole + ((size_t)(it.s.row + n0 + local) * p.Hq + it.h * p.v.gq + tid - local * p.v.gq) * PROW;
        // (without a maximum a group's sum is 0, or NaN where its scores are)
        dst[D] = mx;
        dst[D + 1] = (m0 == -INFINITY ? l0 : lower_by(l0, m0 - mx)) + (m1 == -INFINITY ? l1 : lower_by(l1, m1 - mx));
        const uint64_t at = (uint64_t)(uintptr_t)dst;
        ms.end[tid] = make_float4(f0, f1, __uint_as_float((uint32_t)at), __uint_as_float((uint32_t)(at >> 32)));
      }
      (void)both_or(false);
      // group gr writes the columns gr R / 2 .. of both accumulators
      const bool has0 = tiles > 1 || first_m == (gr == 0 ? 0 : 1), has1 = tiles > 1 || !has0;
#pragma unroll 1
      for (int cc = gr * (R / 2); cc < min((gr + 1) * (R / 2), cols); cc += 16) {
        float o[2][16];
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2) {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[g2][e] = 0.f;
          if (g2 ? has1 : has0) {
            const uint32_t at = tmem + lane_off + F::TM_O + F::N * g2 + cc;
            tmem_ld16(at, o[g2]);
            if (PARTS == 2) {
              float x[16];
              tmem_ld16(at + R, x);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[g2][e] += x[e];
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (cc + e < cols) {
            const float4 f = ms.end[cc + e];
            float *dst = reinterpret_cast<float *>((uintptr_t)(((uint64_t)__float_as_uint(f.w) << 32) | __float_as_uint(f.z)));
            dst[32 * wq + lane] = (f.x == 0.f ? 0.f : o[0][e] * f.x) + (f.y == 0.f ? 0.f : o[1][e] * f.y);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.o_free);
      if (both_or(false)) break;  // the maxima and sums are read: the next item may write them
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------------------ combine
struct CombineParams {
  TreeView v;
  PagedOut o;
  int Hq, R, grid, groups;
  float inv_vscale;    // 2^W_SHIFT / (2^P_SHIFT * alpha_V)
  const uint4 *vfrag;  // R and R^T of the values
  const float *split, *whole;
  const int32_t *unit;
};
constexpr int CB_WARPS = 16, CB_COLS = 32;

// The sequence of row i as paged_seq's, the whole warp looking at 32 offsets at a time.
__device__ __forceinline__ int warp_seq(const PagedView &v, int i, int lane) {
  if (!v.cu_q) return i;
  int lo = 0, n = v.B;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const uint32_t m = __ballot_sync(FULL_MASK, lane == 0 || (lane * step < n && v.cu_q[at] <= i));
    const int k = __popc(m) - 1;
    lo += k * step, n = min(step, n - k * step);
  }
  return lo;
}

// Ends 4 to 6 us behind the partials of short batches, which is latency: its rows and sequences are found ahead of its wait,
// then come the unit's entry, the partials, the products.  6,656 columns (four wide trees) take 15 us, two turns of a CTA.
// 8 `groups` columns (a node's q-head each) per CTA and turn: a warp merges a column's partials, two columns at a time
// (m* = max m_s, l* = sum l_s 2^(m_s - m*), o = sum acc_s 2^(m_s - m*) / l*), the first eight warps multiply by R^T's hi
// parts, the others by its lo parts (16 rows of it in a warp's registers), then the rows are summed and rounded.
__global__ void __launch_bounds__(CB_WARPS * 32) k_tree_combine(const CombineParams p) {
  __shared__ RotColumns x[CB_COLS / 8];
  __shared__ __align__(16) float y[2][CB_COLS][D + 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp >> 3, mt = warp & 7;
  pdl_trigger();
  uint4 a[8];
  rot_load(a, p.vfrag, 1, part, mt, lane);
  const TreeView &v = p.v;
  const uint32_t n = (uint32_t)paged_rows(v.pv) * p.Hq, turn = 8 * p.groups;  // (31 bits)
  bool taken[2];
  uint32_t row[2];
  int unit[2], col[2];  // (-1: zeros)
  // whose columns c0 = r0 + warp and r0 + warp + 16 are
  auto locate = [&](uint32_t r0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t c0 = warp + CB_WARPS * i;
      row[i] = r0 + c0, taken[i] = false, unit[i] = -1;
      if (c0 >= turn || row[i] >= n) continue;
      const int tok = (int)(row[i] / (uint32_t)p.Hq), head = (int)row[i] - tok * p.Hq;
      const int b = warp_seq(v.pv, tok, lane);
      const Seq s = seq_of(v, b, false);
      const int node = tok - s.row;
      taken[i] = node >= 0 && node < s.T;  // (rows past max_q are left as they were)
      if (!taken[i] || s.base + node < 0) continue;
      const int qt = (int)((uint32_t)node * v.by_npu >> 16), h = head / v.gq;
      unit[i] = unit_index(v, b, h, qt), col[i] = (node - qt * v.npu) * v.gq + head - h * v.gq;
    }
  };
  locate(blockIdx.x * turn);
  pdl_wait();
  for (uint32_t r0 = blockIdx.x * turn; r0 < n; r0 += gridDim.x * turn) {
    if (r0 != blockIdx.x * turn) locate(r0);
    const float *src[2] = {nullptr, nullptr};  // the column's first partial
    int ns[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (unit[i] < 0) continue;
      const uint32_t info = (uint32_t)__ldcg(p.unit + unit[i]);
      const int first = min((int)(info & 0xFFFFu), p.grid - 1);
      ns[i] = min((int)(info >> 16), p.grid - first);
      src[i] = ns[i] == 1 ? p.whole + (size_t)row[i] * PROW : p.split + ((size_t)first * 2 * p.R + col[i]) * PROW;
    }
    // (the first CTA's share is its second partial, the others' their first)
    auto part_of = [&](int i, int k) { return ns[i] == 1 ? src[i] : src[i] + ((size_t)k * 2 + (k == 0 ? 1 : 0)) * p.R * PROW; };
    float o[2][4] = {}, ms[2] = {-INFINITY, -INFINITY}, ls[2] = {0.f, 0.f};
    constexpr int FLY = 4;
    for (int s0 = 0; s0 < max(ns[0], ns[1]); s0 += FLY) {
      float m4[2][FLY], l4[2][FLY];
      float4 v4[2][FLY];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < FLY; ++k) {
          m4[i][k] = l4[i][k] = 0.f, v4[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (s0 + k < ns[i]) {
            const float *at = part_of(i, s0 + k);
            m4[i][k] = __ldcg(at + D), l4[i][k] = __ldcg(at + D + 1);
            v4[i][k] = __ldcg(reinterpret_cast<const float4 *>(at) + lane);
          }
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mc = ms[i];
#pragma unroll
        for (int k = 0; k < FLY; ++k)
          if (l4[i][k] != 0.f) mc = fmaxf(mc, m4[i][k]);
        if (mc > ms[i]) {
          const float hf = ms[i] == -INFINITY ? 0.f : exp2f(0.5f * (ms[i] - mc)), f = hf * hf;
          ls[i] = lower(ls[i], hf);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= f;
          ms[i] = mc;
        }
#pragma unroll
        for (int k = 0; k < FLY; ++k) {
          if (l4[i][k] != 0.f) {
            const float hf = exp2f(0.5f * (m4[i][k] - ms[i])), f = hf * hf;
            ls[i] += lower(l4[i][k], hf);
            o[i][0] = fmaf(f, v4[i][k].x, o[i][0]), o[i][1] = fmaf(f, v4[i][k].y, o[i][1]);
            o[i][2] = fmaf(f, v4[i][k].z, o[i][2]), o[i][3] = fmaf(f, v4[i][k].w, o[i][3]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c0 = warp + CB_WARPS * i;
      if (c0 >= turn) break;
      const float f = ls[i] == 0.f ? 0.f : p.inv_vscale / ls[i];  // (NaN stays)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] *= f;
      rot_put(x[c0 >> 3], c0 & 7, lane, o[i]);
    }
    __syncthreads();
#pragma unroll 1
    for (int g = 0; g < p.groups; ++g) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      if (part) rot_mul<false>(acc, a, x[g], lane);
      else rot_mul<true>(acc, a, x[g], lane);
      float *d = &y[part][8 * g + 2 * (lane & 3)][16 * mt + (lane >> 2)];
      d[0] = acc[0], d[D + 4] = acc[1], d[8] = acc[2], d[D + 12] = acc[3];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!taken[i]) continue;
      const float4 h4 = *reinterpret_cast<const float4 *>(&y[0][warp + CB_WARPS * i][4 * lane]);
      const float4 l4 = *reinterpret_cast<const float4 *>(&y[1][warp + CB_WARPS * i][4 * lane]);
      const float z[4] = {h4.x + l4.x, h4.y + l4.y, h4.z + l4.z, h4.w + l4.w};
      store_lane4(p.o.out, p.o.dtype, (size_t)row[i] * D, lane, z);
    }
    // (the next turn's x is written behind its loads; y behind the next barrier)
  }
}

struct Layout {
  int R, parts, npu, n_qt, gq, grid;
  int64_t units;
  size_t unit, split, whole, bytes;
};
// Columns of a unit, 32 or 64, from what the host knows of the batch: a tile of 64 takes 1.45 times the time of one of 32 and an
// item 19 tiles' where one of 32 takes 8, so 64 pay where trees fill them over long contexts, 32 where trees are smaller
// than their bound or contexts short.  Trees are taken to lie evenly about their mean up to max_q.  The time
// is the CTAs' even share of the items and half an item for the split ends.  Measured, 64 against 32 (4 query heads per KV
// head, bf16): 4 sequences of 16,000 tokens with 9 nodes 62 / 74 us, 24 nodes 100 / 107, 64 nodes 182 / 265, 1 to 16 nodes
// 62 / 53; 8 of 1,500 with 9 nodes 32 / 33, 24 nodes 54 / 49, 64 nodes 100 / 112, 1 to 16 nodes 32 / 27; 32 of 16 to
// 8,000 with up to 20 nodes, 6 query heads, f16: 39 / 31.  What the host knows are bounds: a batch padded to full trees, or with
// the block table's width for max_len, is taken for what it could hold, which can cost it that difference.
int columns(const PagedView &pv, int gq, int grid) {
  if (gq > 32) return 64;
  if (pv.max_q * gq <= 32 || pv.B == 0) return 32;
  const double hi = pv.max_q, mean = fmin((double)pv.n_tokens / pv.B, hi), lo = fmax(2 * mean - hi, 1.0);
  const double tiles = (pv.max_len + KT - 1) / KT;
  auto time = [&](int R, double item, double tile) {
    const int npu = R / gq;
    double units = 0;
    for (int i = 0; i < 16; ++i) {
      const int T = (int)fmin(lo + (hi - lo + 1) * (i + 0.5) / 16, hi);
      units += (T + npu - 1) / npu / 16.0;
    }
    return pv.B * pv.Hkv * units / grid * (item + tile * tiles) + item / 2;
  };
  return time(64, 19, 1.45) < time(32, 8, 1) ? 64 : 32;
}
bool layout(const tq_ctx *k, const PagedView &pv, int Hq, int out_dtype, Layout *l) {
  l->gq = Hq / pv.Hkv;
  l->parts = out_dtype == TQ_DTYPE_BF16 ? 1 : 2;
  l->R = columns(pv, l->gq, k->num_sms);
  l->npu = l->R / l->gq;  // at least one: 64 heads per KV head at most
  l->n_qt = (pv.max_q + l->npu - 1) / l->npu;
  l->grid = k->num_sms;
  // the larger of both widths' needs, so that no smaller batch of trees needs more than a larger one
  const int least = l->gq <= 32 ? 32 / l->gq : 1;
  l->units = (int64_t)pv.B * pv.Hkv * ((pv.max_q + least - 1) / least);
  const int64_t tiles = l->units * (((int64_t)pv.max_len + KT - 1) / KT + ITEM_TILES);
  if (l->grid > 65535 || tiles > INT32_MAX || (int64_t)pv.n_tokens * Hq > INT32_MAX) return false;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  l->unit = 0;
  l->split = up((size_t)l->units * 4);
  l->whole = l->split + up((size_t)l->grid * 2 * 64 * PROW * 4);
  l->bytes = l->whole + up((size_t)pv.n_tokens * Hq * PROW * 4);
  return true;
}

template <int R, int PARTS>
cudaError_t launch_partial(const PartialParams &p, int grid, cudaStream_t st) {
  constexpr uint32_t smem = Cfg<R, PARTS>::OFF_MISC + sizeof(Misc<Cfg<R, PARTS>::NKN>) + 1024;  // + slack to align to 1024
  static_assert(smem <= 227 * 1024, "shared memory budget");
  const cudaError_t e = kernel_smem_attr((const void *)k_tree_partial<R, PARTS>, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_tree_partial<R, PARTS>, dim3(grid), dim3(Cfg<R, PARTS>::THREADS), smem, st, p);
}

}  // namespace

// One node per sequence sees all of its sequence's keys: a single row of the paged decode, which takes 9.5 us for two
// sequences of 733 tokens and 59 for eight towards 32K, where the kernels above take 15.0 and 110 (captured).
static bool is_decode(const PagedView &pv, int Hq) { return pv.max_q == 1 && Hq / pv.Hkv <= 16; }

bool paged_tree_workspace(const tq_ctx *k, const PagedView &pv, int Hq, size_t *bytes) {
  if (is_decode(pv, Hq)) return paged_decode_workspace(k, pv, Hq, bytes);
  Layout a, b;  // the size does not depend on the output's type
  if (!layout(k, pv, Hq, TQ_DTYPE_BF16, &a) || !layout(k, pv, Hq, TQ_DTYPE_F32, &b)) return false;
  *bytes = a.bytes > b.bytes ? a.bytes : b.bytes;
  return true;
}

int paged_tree_columns(const tq_ctx *k, const PagedView &pv, int Hq) {
  Layout l;
  return !is_decode(pv, Hq) && layout(k, pv, Hq, TQ_DTYPE_BF16, &l) ? l.R : 0;
}

cudaError_t launch_paged_tree(const tq_ctx *k, const tq_ctx *v, const PagedView &pv, const int32_t *parents,
                              const uint8_t *kp, const uint8_t *vp, const RowsView &q, int Hq, const RopeView &rope,
                              float scale, const PagedOut &o, void *ws, cudaStream_t st, bool late) {
  if (is_decode(pv, Hq)) return launch_paged_decode(k, v, pv, kp, vp, q, Hq, rope, scale, o, ws, st);
  Layout l;
  if (!layout(k, pv, Hq, o.dtype, &l)) return cudaErrorInvalidValue;
  uint8_t *base = static_cast<uint8_t *>(ws);
  const TreeView tv{pv, parents, l.npu, l.n_qt, l.gq, UINT32_MAX / (uint32_t)l.grid, 65536u / l.npu + 1, 65536u / l.gq + 1};
  PartialParams p{};
  p.v = tv, p.kp = kp, p.vp = vp, p.q = q, p.rope = rope, p.Hq = Hq;
  p.qmul = LOG2E * scale / k->f16.alpha;
  p.kfrag = k->d_rfrag;
  for (int i = 0; i < 2; ++i) {
    p.klo[i] = k->f16.lo[i], p.khi[i] = k->f16.hi[i];
    p.vlo[i] = v->f16.lo[i], p.vhi[i] = v->f16.hi[i];
  }
  p.split = reinterpret_cast<float *>(base + l.split);
  p.whole = reinterpret_cast<float *>(base + l.whole);
  p.unit = reinterpret_cast<int32_t *>(base + l.unit);
  p.late = late;
  cudaError_t e;
  if (l.parts == 1)
    e = l.R == 32 ? launch_partial<32, 1>(p, l.grid, st) : launch_partial<64, 1>(p, l.grid, st);
  else
    e = l.R == 32 ? launch_partial<32, 2>(p, l.grid, st) : launch_partial<64, 2>(p, l.grid, st);
  if (e != cudaSuccess) return e;
  CombineParams c{};
  c.v = tv, c.o = o, c.Hq = Hq, c.R = l.R, c.grid = l.grid;
  c.inv_vscale = 1.0f / (exp2f(P_SHIFT - W_SHIFT) * v->f16.alpha);
  c.vfrag = v->d_rfrag;
  c.split = p.split, c.whole = p.whole, c.unit = p.unit;
  // Eight columns a turn while that leaves no SM two turns, up to 32: short chat 16.5 us, with 32 always 18.7; four wide
  // trees 172, with 8 always 178.
  const int64_t cols = (int64_t)pv.n_tokens * Hq;
  c.groups = 1;
  while (c.groups < CB_COLS / 8 && cols > (int64_t)8 * c.groups * k->num_sms) c.groups <<= 1;
  const int64_t want = (cols + 8 * c.groups - 1) / (8 * c.groups);
  return launch_pdl(k_tree_combine, dim3((unsigned)(want < k->num_sms ? want : k->num_sms)), dim3(CB_WARPS * 32), 0, st, c);
}

}  // namespace tq
