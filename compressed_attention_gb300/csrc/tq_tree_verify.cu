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
#include <cooperative_groups.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

namespace cg = cooperative_groups;

constexpr int VT = 512, VW = VT / 32;  // threads, warps of a CTA
constexpr int MAX_CLUSTER = 16;
constexpr uint64_t ONE = 1ull << 62;

// A probability in multiples of 2^-62: [0, 1], NaN as 0.
__device__ __forceinline__ uint64_t fix(float p) { return __float2ull_rz(fminf(fmaxf(p, 0.f), 1.f) * 0x1p62f); }
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
__global__ void __launch_bounds__(VT) k_tree_verify(const VerifyArgs a) {
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

  // this CTA's slice, and a warp's segment of it: whole runs of 32 weights
  const int64_t s0 = (int64_t)V * rank / C, s1 = (int64_t)V * (rank + 1) / C;
  const int seg = (((int)(s1 - s0) + VW - 1) / VW + 31) & ~31;
  int cur = 0, n_path = 1, fails = 0, pass = 0;
  const void *prow = row_of(a.target, a.target_stride, 0), *qrow = DRAFT ? row_of(a.draft, a.draft_stride, 0) : nullptr;
  // weight w of r after `fails` failed tests (no draft: without the taken-out tokens)
  auto weight = [&](int64_t w) -> uint64_t {
    uint64_t r = fix(prob<DT>(prow, w));
    if (DRAFT && fails) {
      const uint64_t q = fix(prob<DT>(qrow, w));
      for (int k = 0; k < fails; ++k) {
        const uint64_t c = mul62(sm.z[k], q);
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
    const int64_t g0 = s0 + (int64_t)warp * seg, g1 = min(g0 + seg, s1);
    uint64_t sum = 0;
#pragma unroll 8
    for (int64_t w = g0 + lane; w < g1; w += 32) sum += weight(w);
    sum = warp_sum(sum);
    if (!DRAFT)  // less the tokens taken out (each once: a token again has failed before)
      for (int k = 0; k < fails; ++k) {
        const int x = sm.token[sm.gone[k]];
        if (x >= g0 && x < g1) sum -= sm.p[sm.gone[k]];
      }
    if (lane == 0) sm.warp[warp] = sum;
    __syncthreads();
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
  if (rank == 0 && tid == 0) path[0] = 0;
  for (int c = next_child(0, 0); c < TREE_MAX;) {
    uint64_t r = sm.p[c];
    bool take;
    if (DRAFT) {
      for (int k = 0; k < fails; ++k) {
        const uint64_t d = mul62(sm.z[k], sm.q[c]);
        r = r > d ? r - d : 0;
      }
      take = __umul64hi(sm.u[c], mul62(Z, sm.q[c])) < r;
    } else {
      bool again = false;
      for (int k = lane; k < fails; k += 32) again |= sm.token[sm.gone[k]] == sm.token[c];
      if (__any_sync(FULL_MASK, again)) r = 0;
      take = __umul64hi(sm.u[c], Z) < r;
    }
    if (take) {
      cur = c, fails = 0, Z = ONE, have = false;
      if (rank == 0 && tid == 0) path[n_path] = c;
      ++n_path;
      prow = row_of(a.target, a.target_stride, cur);
      if (DRAFT) qrow = row_of(a.draft, a.draft_stride, cur);
    } else if (DRAFT) {
      __syncthreads();  // (z is read)
      if (tid == 0) sm.z[fails] = Z;
      __syncthreads();
      ++fails;
      const uint64_t left = total();
      if (left) Z = left < ONE * 2 ? left : ONE * 2 - 1, sum = left, have = true;
      else --fails;  // as it was
    } else if (r) {
      __syncthreads();
      if (tid == 0) sm.gone[fails] = c;
      __syncthreads();
      ++fails;
      Z = Z > r ? Z - r : 0;
    }
    c = next_child(cur, c);
  }
  if (!have) sum = total();
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
  const int64_t g0 = s0 + (int64_t)wseg * seg, g1 = min(g0 + seg, s1);
  for (int64_t w0 = g0; w0 < g1; w0 += VT) {
    const int64_t w = w0 + tid;
    uint64_t r = w < g1 ? weight(w) : 0;
    if (!DRAFT)
      for (int k = 0; k < fails; ++k)
        if (sm.token[sm.gone[k]] == w) r = 0;
    uint64_t inc = r;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint64_t o = __shfl_up_sync(FULL_MASK, inc, m);
      if (lane >= m) inc += o;
    }
    if (lane == 31) sm.scan[warp] = inc;
    __syncthreads();
    uint64_t before = 0, all = 0;
    for (int i = 0; i < VW; ++i) {
      if (i < warp) before += sm.scan[i];
      all += sm.scan[i];
    }
    if (t >= before + inc - r && t < before + inc) a.next_token[b] = (int32_t)w;
    if (t < all) return;
    t -= all;
    __syncthreads();
  }
}

template <int DT>
cudaError_t launch(const VerifyArgs &a, int cluster, cudaStream_t st) {
  auto kern = a.draft ? k_tree_verify<DT, true> : k_tree_verify<DT, false>;
  if (cluster > 8) {
    const cudaError_t e = cudaFuncSetAttribute((const void *)kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
  (void)num_sms;
  const int cluster = 8;
  if (a.dtype == TQ_DTYPE_F32) return launch<TQ_DTYPE_F32>(a, cluster, st);
  if (a.dtype == TQ_DTYPE_BF16) return launch<TQ_DTYPE_BF16>(a, cluster, st);
  return launch<TQ_DTYPE_F16>(a, cluster, st);
}

}  // namespace tq
