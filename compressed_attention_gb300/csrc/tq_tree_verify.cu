// Verification of drafted tokens: a walk along each sequence's tree from given random numbers.
//
// A cluster of CTAs per sequence, each over its slice of the vocabulary.  Every CTA reads the nodes
// (parent, token, the two probabilities of the token behind its parent: a node per thread, two dependent loads)
// and walks alike: a test needs single weights only.  The vocabulary is read where a test fails against a
// draft's row (the residual's sum) and once at the end, for the weights that the next token is drawn from; the sums meet
// over distributed shared memory and a cluster barrier.  Residuals are not stored: r after k failed tests is
// recomputed from p, q and the k sums so far, max(... max(p - q, 0) - Z_1 q ...), so that no vocabulary is too
// large.  The CTA that holds the threshold finds the token in one of its warps' segments.
//
// Weights are whole multiples of 2^-62 in 64 bits: sums do not depend on their order, so neither does the
// outcome, and a comparison is off by 2^-62 where fp32 sums over 10^5 weights would move the borders between tokens by
// 10^-7, as much as a rare token has.
//
// Measured: 64 chains over 131,072 tokens (fp32, two rows of each: 67 MB) 22.3 us, 3.0 TB/s; bound by the ALU (51%; whole
// groups loaded without a look at the row's ends and the first residual by comparing floats: 31 -> 23 us) and by SMs with two
// CTAs beside SMs with one.  One chain 7.5 us: launch, two dependent loads of the nodes, one pass, the token's segment
// again.  16 trees of several failed tests 20 us: a pass over the rows and a cluster barrier each.  32 trees of 20 to 32
// likeliest tokens over 65,537 (bf16) 12 us: one pass, then the walk's chain of tests.
#include <cooperative_groups.h>
#include <limits.h>

#include <type_traits>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

namespace cg = cooperative_groups;

constexpr int VT = 512, VW = VT / 32;  // threads, warps of a CTA
constexpr int MAX_CLUSTER = 16;
constexpr uint64_t ONE = 1ull << 62;

// A probability in multiples of 2^-62: [0, 1], NaN as 0.  Its 24 bits in a word's upper end are 2^(e - 128) of 64 bits
// with biased exponent e: shifts, where the conversion instruction to 64 bits has a fraction of their rate.
__device__ __forceinline__ float clamp01(float p) { return fminf(fmaxf(p, 0.f), 1.f); }
__device__ __forceinline__ uint64_t fix01(float p) {  // p in [0, 1]
  const uint32_t b = __float_as_uint(p);
  uint64_t r;  // (a shift past 64 leaves 0: exponents below 64, and 0)
  asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"((uint64_t)((b << 8) | 0x80000000u) << 32), "r"(128u - (b >> 23)));
  return r;
}
__device__ __forceinline__ uint64_t fix(float p) { return fix01(clamp01(p)); }
// floor(a b / 2^62), a < 2^63, b <= 2^62.
__device__ __forceinline__ uint64_t mul62(uint64_t a, uint64_t b) { return __umul64hi(a << 1, b << 1); }
// A random number in multiples of 2^-64.
__device__ __forceinline__ uint64_t fix_u(float u) { return __float2ull_rz(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f) * 0x1p64f); }

template <int DT>
__device__ __forceinline__ float prob(const void *row, int64_t w) {
  if (DT == TQ_DTYPE_F32) return static_cast<const float *>(row)[w];
  const uint16_t x = static_cast<const uint16_t *>(row)[w];
  return DT == TQ_DTYPE_BF16 ? bf16_bits_to_f32(x) : __half2float(__ushort_as_half(x));
}

// A row in groups of 16 bytes from the last 16-byte boundary at or before it: group g is elements g E - skip .. , of
// which the first group and the last may lack some.
template <int DT>
struct Groups {
  static constexpr int E = DT == TQ_DTYPE_F32 ? 4 : 8;
  static __device__ __forceinline__ int skip(const void *row) {
    return (int)(((uintptr_t)row & 15) / (DT == TQ_DTYPE_F32 ? 4 : 2));
  }
  static __device__ __forceinline__ float at(const uint4 &v, int e) {
    const uint32_t w = DT == TQ_DTYPE_F32 ? (&v.x)[e] : (&v.x)[e >> 1];
    if (DT == TQ_DTYPE_F32) return __uint_as_float(w);
    const uint32_t x = (e & 1) ? w >> 16 : w & 0xFFFFu;
    return DT == TQ_DTYPE_BF16 ? bf16_bits_to_f32(x) : __half2float(__ushort_as_half((uint16_t)x));
  }
  // Group g of a row of V elements with the skip of another row (`with`): one load where the two lie alike and
  // the group is whole, else element by element; zeros outside the row.
  static __device__ __forceinline__ uint4 load(const void *row, int g, int with, bool alike, int V) {
    const int64_t w0 = (int64_t)g * E - with;
    if (alike && w0 >= 0 && w0 + E <= V)
      return __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(row) + w0 * (16 / E)));
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (w0 + e < 0 || w0 + e >= V) continue;
      if (DT == TQ_DTYPE_F32) (&v.x)[e] = static_cast<const uint32_t *>(row)[w0 + e];
      else (&v.x)[e >> 1] |= (uint32_t)static_cast<const uint16_t *>(row)[w0 + e] << (16 * (e & 1));
    }
    return v;
  }
};

struct Shared {
  int32_t token[TREE_MAX];
  int32_t parent[TREE_MAX];
  uint64_t p[TREE_MAX], q[TREE_MAX], u[TREE_MAX];  // of a node's token behind its parent; its random number
  uint64_t z[TREE_MAX];      // draft: Z ahead of the failed tests on the current node
  int32_t gone[TREE_MAX];    // no draft: nodes that failed on the current node
  uint64_t cta[2][MAX_CLUSTER];  // the CTAs' sums of a pass (alternating: a CTA may be one pass ahead)
  uint64_t warp[VW];             // this CTA's warps' sums
  uint64_t scan[VW];
};

template <int DT, bool DRAFT>
__global__ void __launch_bounds__(VT, 2) k_tree_verify(const VerifyArgs a) {
  __shared__ Shared sm;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank(), b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  int lo = b, T = 1;
  if (a.cu_q) {
    lo = a.cu_q[b];
    const int e = min(a.cu_q[b + 1], a.n_tokens);
    T = lo < 0 ? 0 : max(e - lo, 0);
  }
  if (T > a.max_q) {
    if (rank == 0 && tid == 0) atomicExch(a.status, (int32_t)DEVERR_SEQLEN);
    T = a.max_q;
  }
  int32_t *path = a.path + b * a.path_stride;
  if (T == 0) {  // (the whole cluster)
    if (rank == 0) {
      for (int i = tid; i < a.max_q; i += VT) path[i] = -1;
      if (tid == 0) a.n_path[b] = 0, a.next_token[b] = -1;
    }
    return;
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // begun: waited for ahead of the first sums' exchange
  const size_t esz = DT == TQ_DTYPE_F32 ? 4 : 2;
  auto row_of = [&](const void *base, int64_t stride, int node) {
    return static_cast<const void *>(static_cast<const uint8_t *>(base) + (size_t)(lo + node) * stride * esz);
  };
  const int V = a.vocab;
  if (tid < T) {
    int par = a.parents[lo + tid];
    const int x = tid ? a.tokens[lo + tid] : 0;
    bool bad = par < -1 || par >= tid;
    if (bad) par = -1;
    const bool known = (unsigned)x < (unsigned)V;
    bad |= !known;
    if (bad && rank == 0) atomicExch(a.status, (int32_t)DEVERR_TREE);
    const bool child = par >= 0 && known;
    sm.token[tid] = x, sm.parent[tid] = child ? par : -1;  // (a token outside the vocabulary: never tested)
    sm.p[tid] = child ? fix(prob<DT>(row_of(a.target, a.target_stride, par), x)) : 0;
    sm.q[tid] = DRAFT && child ? fix(prob<DT>(row_of(a.draft, a.draft_stride, par), x)) : 0;
    sm.u[tid] = tid ? fix_u(a.u_accept[lo + tid]) : 0;
  }
  __syncthreads();
  int par4[TREE_MAX / 32];  // a warp's lanes hold all parents
#pragma unroll
  for (int i = 0; i < TREE_MAX / 32; ++i) par4[i] = 32 * i + lane < T ? sm.parent[32 * i + lane] : -1;
  // the next child of node v behind node `last` (TREE_MAX: none); the whole warp calls
  auto next_child = [&](int v, int last) {
    int at = TREE_MAX;
#pragma unroll
    for (int i = TREE_MAX / 32 - 1; i >= 0; --i) {
      const uint32_t m = __ballot_sync(FULL_MASK, par4[i] == v && 32 * i + lane > last);
      if (m) at = 32 * i + __ffs(m) - 1;
    }
    return at;
  };

  // The rows that the walk stands on, this CTA's groups of them, and a warp's: whole runs of 32 groups.
  using Gr = Groups<DT>;
  int cur = 0, n_path = 1, fails = 0, pass = 0;
  const void *prow, *qrow;
  int skip, lo_g, hi_g, seg;
  bool alike;
  auto stand = [&](int node) {
    prow = row_of(a.target, a.target_stride, node);
    skip = Gr::skip(prow);
    alike = true;
    if (DRAFT) qrow = row_of(a.draft, a.draft_stride, node), alike = Gr::skip(qrow) == skip;
    const int64_t n = ((int64_t)V + skip + Gr::E - 1) / Gr::E;
    lo_g = (int)(n * rank / C), hi_g = (int)(n * (rank + 1) / C);
    seg = ((hi_g - lo_g + VW - 1) / VW + 31) & ~31;
  };
  stand(0);
  // r of one element after `fails` failed tests (no draft: the tokens taken out are the caller's); p and q in [0, 1]
  auto weight = [&](float p, float q) -> uint64_t {
    uint64_t r = fix01(p);
    if (DRAFT && fails) {
      const uint64_t x = fix01(q);
      r -= fix01(fminf(p, q));  // the first test's Z is 1, and of two floats the lesser has the lesser multiple
      for (int k = 1; k < fails; ++k) {
        const uint64_t c = mul62(sm.z[k], x);
        r = r > c ? r - c : 0;
      }
    }
    return r;
  };
  auto warp_sum = [](uint64_t x) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(FULL_MASK, x, m);
    return x;
  };
  // sum r over the vocabulary, with the CTAs' sums and the warps' sums left in shared memory
  auto total = [&]() -> uint64_t {
    const int g0 = lo_g + warp * seg, g1 = min(g0 + seg, hi_g);
    uint64_t sum = 0;
    auto add_up = [&](auto fly, auto with_q, auto f) {  // `fly` groups of a thread in flight
      constexpr int FLY = decltype(fly)::value;
      constexpr bool Q = decltype(with_q)::value;
      auto take = [&](const uint4 &p4, const uint4 &q4) {
        float x[Gr::E], y[Gr::E];
        uint32_t most = 0;
#pragma unroll
        for (int e = 0; e < Gr::E; ++e) {
          x[e] = Gr::at(p4, e), y[e] = Q ? Gr::at(q4, e) : 0.f;
          most = max(most, max(__float_as_uint(x[e]), __float_as_uint(y[e])));
        }
        if (most > 0x3F800000u) {  // past 1, negative or NaN
#pragma unroll
          for (int e = 0; e < Gr::E; ++e) x[e] = clamp01(x[e]), y[e] = clamp01(y[e]);
        }
        f(x, y);
      };
      const uint4 none = make_uint4(0u, 0u, 0u, 0u);
      // whole groups first: their loads need no look at the row's ends
      const bool plain = !Q || alike;
      const int end = (V + skip) / Gr::E, a = max(g0, skip ? 1 : 0), e = min(g1, end);
      if (plain) {
        const uint4 *pg = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(prow) - skip * (16 / Gr::E)) + a + lane;
        const uint4 *qg = Q ? reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(qrow) - skip * (16 / Gr::E)) + a + lane : nullptr;
#pragma unroll 1
        for (int g = a + lane; g < e; g += 32 * FLY, pg += 32 * FLY, qg += 32 * FLY) {
          uint4 p4[FLY], q4[FLY];
#pragma unroll
          for (int i = 0; i < FLY; ++i) {
            p4[i] = q4[i] = none;
            if (g + 32 * i < e) {
              p4[i] = __ldg(pg + 32 * i);
              if (Q) q4[i] = __ldg(qg + 32 * i);
            }
          }
#pragma unroll
          for (int i = 0; i < FLY; ++i) take(p4[i], q4[i]);
        }
      }
      // the row's first and last group where they are not whole (a lane each); all of them where p's and q's do not pair
      int g = g0 + lane;
      if (plain) g = lane == 0 && skip ? 0 : lane == 1 && !(skip && end == 0) ? end : INT_MAX;
#pragma unroll 1
      for (; g < g1; g += 32) {
        if (g >= g0) take(Gr::load(prow, g, skip, true, V), Q ? Gr::load(qrow, g, skip, alike, V) : none);
        if (plain) break;
      }
    };
    using Fly = std::integral_constant<int, DT == TQ_DTYPE_F32 ? 4 : 2>;
    using Row = const float (&)[Gr::E];
    if (!DRAFT || !fails) {
      add_up(Fly(), std::false_type(), [&](Row x, Row) {
#pragma unroll
        for (int e = 0; e < Gr::E; ++e) sum += fix01(x[e]);
      });
    } else if (fails == 1) {
      add_up(Fly(), std::true_type(), [&](Row x, Row y) {
#pragma unroll
        for (int e = 0; e < Gr::E; ++e) sum += fix01(x[e]), sum -= fix01(fminf(x[e], y[e]));
      });
    } else {
      add_up(std::integral_constant<int, 1>(), std::true_type(), [&](Row x, Row y) {
#pragma unroll
        for (int h = 0; h < Gr::E; h += 4) {  // `weight` of four elements at once
          uint64_t r[4], q2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            r[e] = fix01(x[h + e]) - fix01(fminf(x[h + e], y[h + e]));
            q2[e] = fix01(y[h + e]) << 1;
          }
#pragma unroll 1
          for (int k = 1; k < fails; ++k) {
            const uint64_t z2 = sm.z[k] << 1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint64_t c = __umul64hi(z2, q2[e]);
              r[e] = r[e] > c ? r[e] - c : 0;
            }
          }
          sum += (r[0] + r[1]) + (r[2] + r[3]);
        }
      });
    }
    sum = warp_sum(sum);
    if (!DRAFT)  // less the tokens taken out (each once: a token again has failed before)
      for (int k = 0; k < fails; ++k) {
        const int x = (int)(((int64_t)sm.token[sm.gone[k]] + skip) / Gr::E);
        if (x >= g0 && x < g1) sum -= sm.p[sm.gone[k]];
      }
    if (lane == 0) sm.warp[warp] = sum;
    __syncthreads();
    // (the others' shared memory is there once they have begun)
    if (pass == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const int side = pass++ & 1;
    if (warp == 0) {
      const uint64_t t = warp_sum(lane < VW ? sm.warp[lane] : 0);
      if (lane < C) *cl.map_shared_rank(&sm.cta[side][rank], lane) = t;
    }
    cl.sync();
    uint64_t t = 0;
    for (int i = 0; i < C; ++i) t += sm.cta[side][i];
    return t;
  };

  uint64_t Z = ONE, sum = 0;
  bool have = false;  // sum is that of r as it stands
  uint32_t out[TREE_MAX / 32] = {};  // no draft: nodes that failed on the current node (every warp keeps its own: no barrier a test)
  if (rank == 0 && tid == 0) path[0] = 0;
  for (int c = next_child(0, 0);; c = next_child(cur, c)) {
    const bool done = c == TREE_MAX;  // no child left
    if (done && have) break;
    bool refused = false;
    if (!done) {
      uint64_t r = sm.p[c];
      bool take;
      if (DRAFT) {
        for (int k = 0; k < fails; ++k) {
          const uint64_t d = mul62(sm.z[k], sm.q[c]);
          r = r > d ? r - d : 0;
        }
        take = __umul64hi(sm.u[c], mul62(Z, sm.q[c])) < r;
      } else {
        bool again = false;  // a token that has failed on this node
        const int x = sm.token[c];
#pragma unroll
        for (int i = 0; i < TREE_MAX / 32; ++i) again |= ((out[i] >> lane) & 1u) && sm.token[32 * i + lane] == x;
        if (__any_sync(FULL_MASK, again)) r = 0;
        take = __umul64hi(sm.u[c], Z) < r;
      }
      if (take) {
        cur = c, fails = 0, Z = ONE, have = false;
#pragma unroll
        for (int i = 0; i < TREE_MAX / 32; ++i) out[i] = 0;
        if (rank == 0 && tid == 0) path[n_path] = c;
        ++n_path;
        stand(cur);
      } else if (DRAFT) {
        __syncthreads();  // (z is read)
        if (tid == 0) sm.z[fails] = Z;
        __syncthreads();
        ++fails;
        refused = true;
      } else if (r) {
#pragma unroll
        for (int i = 0; i < TREE_MAX / 32; ++i) out[i] |= c >> 5 == i ? 1u << (c & 31) : 0u;
        ++fails;
        Z = Z > r ? Z - r : 0;
      }
    } else if (!DRAFT) {  // the list that the sums look at
      if (warp == 0) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < TREE_MAX / 32; ++i) {
          if ((out[i] >> lane) & 1u) sm.gone[n + __popc(out[i] & ((1u << lane) - 1))] = 32 * i + lane;
          n += __popc(out[i]);
        }
      }
      __syncthreads();
    }
    if (done || refused) {  // (one place: the passes' code is long)
      const uint64_t s = total();
      if (done) {
        sum = s;
        break;
      }
      if (s) Z = s < ONE * 2 ? s : ONE * 2 - 1, sum = s, have = true;
      else --fails, have = false;  // as it was, its sums to be found again
    }
  }
  if (rank == 0) {
    for (int i = n_path + tid; i < a.max_q; i += VT) path[i] = -1;
    if (tid == 0) a.n_path[b] = n_path;
  }
  // ---- the smallest w whose running sum passes the threshold
  uint64_t t = __umul64hi(sum, fix_u(a.u_next[b]));
  const int side = (pass - 1) & 1;
  int owner = C;
  for (int i = 0; i < C; ++i) {
    const uint64_t x = sm.cta[side][i];
    if (owner == C) {
      if (t < x) owner = i;
      else t -= x;
    }
  }
  if (owner == C && rank == 0 && tid == 0) a.next_token[b] = -1;  // no weight
  if (owner != rank) return;
  if (tid == 0) a.next_token[b] = -1;  // (what the scan below always overwrites, unless sums of 2 and more wrapped around)
  int wseg = 0;
  while (wseg < VW - 1 && t >= sm.warp[wseg]) t -= sm.warp[wseg++];
  const int g0 = lo_g + wseg * seg, g1 = min(g0 + seg, hi_g);
  for (int gb = g0; gb < g1; gb += VT) {  // a group per thread
    const int g = gb + tid;
    uint64_t r[Gr::E], mine = 0;
    uint4 p4 = make_uint4(0u, 0u, 0u, 0u), q4 = p4;
    if (g < g1) {
      p4 = Gr::load(prow, g, skip, true, V);
      if (DRAFT && fails) q4 = Gr::load(qrow, g, skip, alike, V);
    }
    const int64_t w0 = (int64_t)g * Gr::E - skip;
#pragma unroll
    for (int e = 0; e < Gr::E; ++e) r[e] = weight(clamp01(Gr::at(p4, e)), clamp01(Gr::at(q4, e)));
    if (!DRAFT) {
#pragma unroll 1
      for (int k = 0; k < fails; ++k) {
        const int64_t at = sm.token[sm.gone[k]] - w0;
#pragma unroll
        for (int e = 0; e < Gr::E; ++e) r[e] = at == e ? 0 : r[e];
      }
    }
#pragma unroll
    for (int e = 0; e < Gr::E; ++e) mine += r[e];
    uint64_t inc = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint64_t o = __shfl_up_sync(FULL_MASK, inc, m);
      if (lane >= m) inc += o;
    }
    if (lane == 31) sm.scan[warp] = inc;
    __syncthreads();
    uint64_t before = inc - mine, all = 0;
    for (int i = 0; i < VW; ++i) {
      if (i < warp) before += sm.scan[i];
      all += sm.scan[i];
    }
    if (t >= before && t - before < mine) {
      uint64_t left = t - before;
#pragma unroll
      for (int e = 0; e < Gr::E; ++e) {
        if (left < r[e]) {
          a.next_token[b] = (int32_t)(w0 + e);
          break;
        }
        left -= r[e];
      }
    }
    if (t < all) return;
    t -= all;
    __syncthreads();
  }
}

template <int DT>
cudaError_t launch(const VerifyArgs &a, int cluster, cudaStream_t st) {
  auto kern = a.draft ? k_tree_verify<DT, true> : k_tree_verify<DT, false>;
  if (cluster > 8) {
    const cudaError_t e = kernel_wide_clusters((const void *)kern);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.B * cluster);
  cfg.blockDim = dim3(VT);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_verify(const VerifyArgs &a, int num_sms, cudaStream_t st) {
  // As many CTAs per sequence as fill the SMs twice, up to a cluster's sixteen: 64 chains take 26 us with four, 36 with
  // two and 35 with eight (as the kernel stood then); 32 trees without a draft 13 with eight, 24 with sixteen.
  int cluster = MAX_CLUSTER;
  while (cluster > 1 && (int64_t)cluster * a.B > 2 * num_sms) cluster >>= 1;
  if (a.dtype == TQ_DTYPE_F32) return launch<TQ_DTYPE_F32>(a, cluster, st);
  if (a.dtype == TQ_DTYPE_BF16) return launch<TQ_DTYPE_BF16>(a, cluster, st);
  return launch<TQ_DTYPE_F16>(a, cluster, st);
}

}  // namespace tq
