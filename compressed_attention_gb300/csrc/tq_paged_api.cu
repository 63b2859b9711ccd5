// The extern "C" entry points of the paged cache: argument checks on the host, then the
// kernel launchers.
#include <cuda_runtime.h>

#include <cmath>

#include "tq_internal.h"

using namespace tq;

namespace {

tq_status fail(tq_status s, const char *msg) {
  set_error("%s", msg);
  return s;
}

tq_status cuda_fail(cudaError_t e, const char *where) {
  set_error("%s: %s", where, cudaGetErrorString(e));
  (void)cudaGetLastError();  // a reported failure does not surface again in a later launch check
  return TQ_ERR_CUDA;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool dtype_ok(int t) { return t == TQ_DTYPE_F32 || t == TQ_DTYPE_BF16 || t == TQ_DTYPE_F16; }

// Contexts, cache and batch of a call; *empty: nothing to do.
tq_status check_paged(const tq_ctx *k, const tq_ctx *v, const tq_paged_kv *kv, const tq_paged_batch *bt,
                      const char *who, PagedView *pv, bool *empty) {
  if (!k || !v) return fail(TQ_ERR_INVALID_ARG, "null context");
  if (!kv || !bt) return fail(TQ_ERR_INVALID_ARG, "null cache or batch");
  if (k->device != v->device) return fail(TQ_ERR_INVALID_ARG, "the key and value contexts belong to different devices");
  tq_status st = check_current_device(k->device, who);
  if (st != TQ_OK) return st;
  if (k->fmt != TQ_FMT_TURBO4 || v->fmt != TQ_FMT_TURBO4 || k->d != D || v->d != D)
    return fail(TQ_ERR_UNSUPPORTED, "the paged cache takes turbo4 keys and values of head dimension 128");
  if (kv->page_size < 16 || kv->page_size > 256 || (kv->page_size & (kv->page_size - 1)))
    return fail(TQ_ERR_INVALID_ARG, "page_size must be 16, 32, 64, 128 or 256");
  if (kv->n_pages < 1 || kv->Hkv < 1 || kv->table_len < 1) return fail(TQ_ERR_INVALID_ARG, "n_pages, Hkv and table_len must be >= 1");
  if (kv->table_stride < kv->table_len) return fail(TQ_ERR_INVALID_ARG, "table_stride below table_len");
  const int64_t cap = (int64_t)kv->table_len * kv->page_size;
  if (bt->B < 0 || bt->n_tokens < 0) return fail(TQ_ERR_INVALID_ARG, "B and n_tokens must be >= 0");
  if (bt->max_q < 1) return fail(TQ_ERR_INVALID_ARG, "max_q must be >= 1");
  if (bt->max_len < 0 || bt->max_len > cap) return fail(TQ_ERR_INVALID_ARG, "max_len must lie in [0, table_len * page_size]");
  if (bt->max_len == 0 && cap > INT32_MAX) return fail(TQ_ERR_INVALID_ARG, "table_len * page_size passes 2^31 - 1: give max_len");
  if (!bt->cu_q && (bt->n_tokens != bt->B || bt->max_q != 1))
    return fail(TQ_ERR_INVALID_ARG, "without cu_q every sequence has one row: n_tokens == B and max_q == 1");
  *empty = bt->B == 0 || bt->n_tokens == 0;
  if (*empty) return TQ_OK;
  if (!kv->k_pages || !kv->v_pages || !kv->block_table || !bt->seq_lens) return fail(TQ_ERR_INVALID_ARG, "null pages, block table or lengths");
  if (!aligned(kv->k_pages, 16) || !aligned(kv->v_pages, 16)) return fail(TQ_ERR_ALIGNMENT, "pages must be 16-byte aligned");
  if (!aligned(kv->block_table, 4) || !aligned(bt->seq_lens, 4) || !aligned(bt->cu_q, 4))
    return fail(TQ_ERR_ALIGNMENT, "block table, lengths and cu_q must be 4-byte aligned");
  if ((int64_t)bt->n_tokens * kv->Hkv > INT32_MAX / 2) return fail(TQ_ERR_INVALID_ARG, "n_tokens * Hkv passes 2^30");
  *pv = PagedView{};
  pv->table = kv->block_table, pv->table_stride = kv->table_stride;
  for (pv->page_shift = 4; (1 << pv->page_shift) < kv->page_size;) ++pv->page_shift;
  pv->n_pages = kv->n_pages, pv->Hkv = kv->Hkv;
  pv->cu_q = bt->cu_q, pv->seq_lens = bt->seq_lens;
  pv->B = bt->B, pv->max_q = bt->max_q < bt->n_tokens ? bt->max_q : bt->n_tokens, pv->n_tokens = bt->n_tokens;
  pv->max_len = bt->max_len ? bt->max_len : (int)cap;
  pv->status = k->d_status;
  return TQ_OK;
}

tq_status check_rows(const tq_rows *r, int heads, RowsView *rv) {
  if (!r || !r->data) return fail(TQ_ERR_INVALID_ARG, "null rows");
  if (!dtype_ok(r->dtype)) return fail(TQ_ERR_INVALID_ARG, "rows must be F32, BF16 or F16");
  const int64_t e = r->dtype == TQ_DTYPE_F32 ? 4 : 2;
  const int64_t most = INT64_MAX / 8 / INT32_MAX;
  if (r->token_stride < 0 || r->head_stride < 0 || r->token_stride > most || r->head_stride > most ||
      (heads > 1 && r->head_stride < D))
    return fail(TQ_ERR_INVALID_ARG, "bad row strides");
  if (!aligned(r->data, 16) || (r->token_stride * e) % 16 || (heads > 1 && (r->head_stride * e) % 16))
    return fail(TQ_ERR_ALIGNMENT, "rows must be 16-byte aligned");
  *rv = RowsView{(const uint8_t *)r->data, r->dtype, r->token_stride * e, r->head_stride * e};
  return TQ_OK;
}

tq_status check_rope(const tq_rope *r, RopeView *rv) {
  *rv = RopeView{};
  if (!r) return TQ_OK;
  if (r->rot_dim != 32 && r->rot_dim != 64 && r->rot_dim != 128) return fail(TQ_ERR_UNSUPPORTED, "rot_dim must be 32, 64 or 128");
  if (!r->cos_table || !r->sin_table) return fail(TQ_ERR_INVALID_ARG, "null rotation table");
  if (r->n_pos < 1) return fail(TQ_ERR_INVALID_ARG, "the rotation table needs a position");
  if (r->interleaved != 0 && r->interleaved != 1) return fail(TQ_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (!aligned(r->cos_table, 16) || !aligned(r->sin_table, 16)) return fail(TQ_ERR_ALIGNMENT, "rotation tables must be 16-byte aligned");
  *rv = RopeView{r->cos_table, r->sin_table, r->n_pos, r->rot_dim, r->interleaved};
  return TQ_OK;
}

tq_status check_heads(const tq_paged_kv *kv, int Hq) {
  if (Hq < 1 || Hq % kv->Hkv) return fail(TQ_ERR_INVALID_ARG, "Hq must be a multiple of Hkv");
  if (Hq / kv->Hkv > 64) return fail(TQ_ERR_UNSUPPORTED, "at most 64 q-heads per KV head");
  return TQ_OK;
}

tq_status check_tree(const tq_paged_batch *bt, const int32_t *parents, bool empty) {
  if (bt->max_q > TREE_MAX) return fail(TQ_ERR_UNSUPPORTED, "at most 128 nodes per sequence");
  if (!parents && !empty) return fail(TQ_ERR_INVALID_ARG, "null parents");
  if (!aligned(parents, 4)) return fail(TQ_ERR_ALIGNMENT, "parents must be 4-byte aligned");
  return TQ_OK;
}

tq_status attention(const tq_ctx *k, const tq_ctx *v, const tq_paged_kv *kv, const tq_paged_batch *bt,
                    const tq_rows *q, int Hq, const tq_rope *rope, const DiffView &diff, float scale, void *out,
                    int out_dtype, void *ws, size_t ws_bytes, tq_stream_t stream, const char *who,
                    bool tree = false, const int32_t *parents = nullptr, bool late = false) {
  PagedView pv;
  bool empty;
  tq_status st = check_paged(k, v, kv, bt, who, &pv, &empty);
  if (st != TQ_OK || (st = check_heads(kv, Hq)) != TQ_OK) return st;
  if (tree && (st = check_tree(bt, parents, empty)) != TQ_OK) return st;
  if (diff.lambda && (Hq / kv->Hkv) % 2) return fail(TQ_ERR_INVALID_ARG, "a head pair shares a KV head: Hq / Hkv must be even");
  if (!dtype_ok(out_dtype)) return fail(TQ_ERR_INVALID_ARG, "the output must be F32, BF16 or F16");
  if (!std::isfinite(scale)) return fail(TQ_ERR_INVALID_ARG, "scale must be finite");
  RopeView rv;
  if ((st = check_rope(rope, &rv)) != TQ_OK || empty) return st;
  RowsView qv;
  if ((st = check_rows(q, Hq, &qv)) != TQ_OK) return st;
  if (!out) return fail(TQ_ERR_INVALID_ARG, "null output");
  if (!aligned(out, 16)) return fail(TQ_ERR_ALIGNMENT, "the output must be 16-byte aligned");
  size_t need = 0;
  if (!(tree ? paged_tree_workspace(k, pv, Hq, &need) : paged_workspace(k, pv, Hq, &need)))
    return fail(TQ_ERR_UNSUPPORTED, "the batch passes 32-bit work counts");
  if (!ws || ws_bytes < need) {
    set_error("workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
    return TQ_ERR_WORKSPACE;
  }
  if (!aligned(ws, 256)) return fail(TQ_ERR_ALIGNMENT, "the workspace must be 256-byte aligned");
  if (scale == 0.f) scale = 1.0f / std::sqrt((float)D);
  const PagedOut o{out, out_dtype, diff};
  const uint8_t *kp = (const uint8_t *)kv->k_pages, *vp = (const uint8_t *)kv->v_pages;
  const cudaError_t e =
      tree ? launch_paged_tree(k, v, pv, parents, kp, vp, qv, Hq, rv, scale, o, ws, (cudaStream_t)stream, late)
           : launch_paged_attention(k, v, pv, kp, vp, qv, Hq, rv, scale, o, ws, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, who);
  return TQ_OK;
}

tq_status append(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv, const tq_paged_batch *batch,
                 const tq_rows *k, const tq_rows *v, const tq_rope *rope, tq_stream_t stream, const char *who,
                 bool tree = false, const int32_t *parents = nullptr) {
  PagedView pv;
  bool empty;
  tq_status st = check_paged(k_ctx, v_ctx, kv, batch, who, &pv, &empty);
  if (st != TQ_OK || (tree && (st = check_tree(batch, parents, empty)) != TQ_OK)) return st;
  RopeView rv;
  if ((st = check_rope(rope, &rv)) != TQ_OK || empty) return st;
  RowsView kr, vr;
  if ((st = check_rows(k, kv->Hkv, &kr)) != TQ_OK || (st = check_rows(v, kv->Hkv, &vr)) != TQ_OK) return st;
  if (kr.dtype != vr.dtype) return fail(TQ_ERR_INVALID_ARG, "k and v must have one dtype");
  const cudaError_t e = launch_paged_append(k_ctx, v_ctx, pv, (uint8_t *)kv->k_pages, (uint8_t *)kv->v_pages, kr, vr,
                                            rv, parents, (cudaStream_t)stream);
  return e == cudaSuccess ? TQ_OK : cuda_fail(e, who);
}

tq_status check_probs(const tq_probs *p, bool rows) {  // rows: some are read
  if (!p || (rows && !p->data)) return fail(TQ_ERR_INVALID_ARG, "null probabilities");
  if (!dtype_ok(p->dtype)) return fail(TQ_ERR_INVALID_ARG, "probabilities must be F32, BF16 or F16");
  if (p->vocab < 1) return fail(TQ_ERR_INVALID_ARG, "vocab must be >= 1");
  if (p->row_stride < p->vocab || p->row_stride > INT64_MAX / 8 / INT32_MAX) return fail(TQ_ERR_INVALID_ARG, "bad row stride of the probabilities");
  if (!aligned(p->data, p->dtype == TQ_DTYPE_F32 ? 4 : 2)) return fail(TQ_ERR_ALIGNMENT, "probabilities must be aligned to their elements");
  return TQ_OK;
}

// No exception crosses the ABI (host allocations of the launchers' caches).
template <typename F>
tq_status guarded(F f) {
  try {
    return f();
  } catch (...) {
    return fail(TQ_ERR_ALLOC, "host allocation failed");
  }
}

}  // namespace

extern "C" {

tq_status tq_make_rope_table(int rot_dim, double base, int64_t n_pos, float *cos_table, float *sin_table) {
  if (!cos_table || !sin_table) return fail(TQ_ERR_INVALID_ARG, "null output");
  if (rot_dim != 32 && rot_dim != 64 && rot_dim != 128) return fail(TQ_ERR_UNSUPPORTED, "rot_dim must be 32, 64 or 128");
  if (n_pos < 0 || !(base > 0.0) || !std::isfinite(base)) return fail(TQ_ERR_INVALID_ARG, "n_pos must be >= 0 and base positive");
  const int half = rot_dim / 2;
  for (int i = 0; i < half; ++i) {
    const double w = std::pow(base, -2.0 * i / rot_dim);
    for (int64_t p = 0; p < n_pos; ++p) {
      cos_table[p * half + i] = (float)std::cos((double)p * w);
      sin_table[p * half + i] = (float)std::sin((double)p * w);
    }
  }
  return TQ_OK;
}

tq_status tq_paged_append(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv,
                          const tq_paged_batch *batch, const tq_rows *k, const tq_rows *v,
                          const tq_rope *rope, tq_stream_t stream) {
  return guarded([&] { return append(k_ctx, v_ctx, kv, batch, k, v, rope, stream, "tq_paged_append"); });
}

tq_status tq_paged_gather(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv,
                          const tq_paged_batch *batch, int unrotate, void *k_out, void *v_out,
                          int out_dtype, tq_stream_t stream) {
  return guarded([&] {
    PagedView pv;
    bool empty;
    tq_status st = check_paged(k_ctx, v_ctx, kv, batch, "tq_paged_gather", &pv, &empty);
    if (st != TQ_OK) return st;
    if (!dtype_ok(out_dtype)) return fail(TQ_ERR_INVALID_ARG, "the output must be F32, BF16 or F16");
    if (empty) return TQ_OK;
    if (!k_out && !v_out) return fail(TQ_ERR_INVALID_ARG, "null outputs");
    if (!aligned(k_out, 16) || !aligned(v_out, 16)) return fail(TQ_ERR_ALIGNMENT, "outputs must be 16-byte aligned");
    const cudaError_t e = launch_paged_gather(k_ctx, v_ctx, pv, (const uint8_t *)kv->k_pages,
                                              (const uint8_t *)kv->v_pages, unrotate != 0, k_out, v_out, out_dtype,
                                              (cudaStream_t)stream);
    return e == cudaSuccess ? TQ_OK : cuda_fail(e, "tq_paged_gather");
  });
}

tq_status tq_paged_workspace_size(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv,
                                  const tq_paged_batch *batch, int Hq, size_t *bytes) {
  if (!bytes) return fail(TQ_ERR_INVALID_ARG, "null output");
  return guarded([&] {
    PagedView pv;
    bool empty;
    tq_status st = check_paged(k_ctx, v_ctx, kv, batch, "tq_paged_workspace_size", &pv, &empty);
    if (st != TQ_OK || (st = check_heads(kv, Hq)) != TQ_OK) return st;
    size_t n = 256;
    if (!empty && !paged_workspace(k_ctx, pv, Hq, &n)) return fail(TQ_ERR_UNSUPPORTED, "the batch passes 32-bit work counts");
    *bytes = n;
    return TQ_OK;
  });
}

tq_status tq_paged_attention(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv,
                             const tq_paged_batch *batch, const tq_rows *q, int Hq, const tq_rope *rope,
                             float scale, void *out, int out_dtype, void *workspace, size_t workspace_bytes,
                             tq_stream_t stream) {
  return guarded([&] {
    return attention(k_ctx, v_ctx, kv, batch, q, Hq, rope, DiffView{}, scale, out, out_dtype, workspace,
                     workspace_bytes, stream, "tq_paged_attention");
  });
}

tq_status tq_paged_diff_attention(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv,
                                  const tq_paged_batch *batch, const tq_rows *q, int Hq, const tq_rope *rope,
                                  const tq_diff *diff, float scale, void *out, int out_dtype,
                                  void *workspace, size_t workspace_bytes, tq_stream_t stream) {
  if (!diff || !diff->lambda_w) return fail(TQ_ERR_INVALID_ARG, "null differential weights");
  if (diff->lambda_stride != 0 && diff->lambda_stride < Hq / 2) return fail(TQ_ERR_INVALID_ARG, "lambda_stride must be 0 or >= Hq / 2");
  if (!(diff->eps >= 0.f) || !std::isfinite(diff->eps) || !std::isfinite(diff->out_scale))
    return fail(TQ_ERR_INVALID_ARG, "eps must be >= 0, eps and out_scale finite");
  if (!aligned(diff->lambda_w, 4) || !aligned(diff->gain, 16)) return fail(TQ_ERR_ALIGNMENT, "weights must be 4-byte, gain 16-byte aligned");
  return guarded([&] {
    const DiffView dv{diff->lambda_w, diff->lambda_stride, diff->gain, diff->eps, diff->out_scale};
    return attention(k_ctx, v_ctx, kv, batch, q, Hq, rope, dv, scale, out, out_dtype, workspace, workspace_bytes,
                     stream, "tq_paged_diff_attention");
  });
}

tq_status tq_paged_tree_append(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv,
                               const tq_paged_batch *batch, const int32_t *parents, const tq_rows *k,
                               const tq_rows *v, const tq_rope *rope, tq_stream_t stream) {
  return guarded([&] { return append(k_ctx, v_ctx, kv, batch, k, v, rope, stream, "tq_paged_tree_append", true, parents); });
}

tq_status tq_paged_tree_workspace_size(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv,
                                       const tq_paged_batch *batch, int Hq, size_t *bytes) {
  if (!bytes) return fail(TQ_ERR_INVALID_ARG, "null output");
  return guarded([&] {
    PagedView pv;
    bool empty;
    tq_status st = check_paged(k_ctx, v_ctx, kv, batch, "tq_paged_tree_workspace_size", &pv, &empty);
    if (st != TQ_OK || (st = check_heads(kv, Hq)) != TQ_OK) return st;
    if (batch->max_q > TREE_MAX) return fail(TQ_ERR_UNSUPPORTED, "at most 128 nodes per sequence");
    size_t n = 256;
    if (!empty && !paged_tree_workspace(k_ctx, pv, Hq, &n)) return fail(TQ_ERR_UNSUPPORTED, "the batch passes 32-bit work counts");
    *bytes = n;
    return TQ_OK;
  });
}

tq_status tq_paged_tree_attention(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv,
                                  const tq_paged_batch *batch, const int32_t *parents, const tq_rows *q, int Hq,
                                  const tq_rope *rope, float scale, void *out, int out_dtype, void *workspace,
                                  size_t workspace_bytes, tq_stream_t stream) {
  return guarded([&] {
    return attention(k_ctx, v_ctx, kv, batch, q, Hq, rope, DiffView{}, scale, out, out_dtype, workspace,
                     workspace_bytes, stream, "tq_paged_tree_attention", true, parents);
  });
}

tq_status tq_test_tree_columns(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv,
                               const tq_paged_batch *batch, int Hq, int32_t *columns) {
  if (!columns) return fail(TQ_ERR_INVALID_ARG, "null output");
  return guarded([&] {
    PagedView pv;
    bool empty;
    tq_status st = check_paged(k_ctx, v_ctx, kv, batch, "tq_test_tree_columns", &pv, &empty);
    if (st != TQ_OK || (st = check_heads(kv, Hq)) != TQ_OK) return st;
    *columns = empty ? 0 : paged_tree_columns(k_ctx, pv, Hq);
    return TQ_OK;
  });
}

tq_status tq_test_tree_wait_timeout(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv,
                                    const tq_paged_batch *batch, const int32_t *parents, const tq_rows *q, int Hq,
                                    void *out, int out_dtype, void *workspace, size_t workspace_bytes,
                                    tq_stream_t stream) {
  return guarded([&] {
    if (batch && batch->max_q < 2) return fail(TQ_ERR_UNSUPPORTED, "single nodes take the paged decode");
    return attention(k_ctx, v_ctx, kv, batch, q, Hq, nullptr, DiffView{}, 0.f, out, out_dtype, workspace,
                     workspace_bytes, stream, "tq_test_tree_wait_timeout", true, parents, true);
  });
}

tq_status tq_tree_verify(const tq_ctx *ctx, const tq_paged_batch *batch, const int32_t *parents,
                         const int32_t *tokens, const tq_probs *target, const tq_probs *draft,
                         const float *u_accept, const float *u_next, int32_t *path, int64_t path_stride,
                         int32_t *n_path, int32_t *next_token, tq_stream_t stream) {
  return guarded([&] {
    if (!ctx) return fail(TQ_ERR_INVALID_ARG, "null context");
    if (!batch) return fail(TQ_ERR_INVALID_ARG, "null batch");
    tq_status st = check_current_device(ctx->device, "tq_tree_verify");
    if (st != TQ_OK) return st;
    if (batch->B < 0 || batch->n_tokens < 0) return fail(TQ_ERR_INVALID_ARG, "B and n_tokens must be >= 0");
    if (batch->max_q < 1) return fail(TQ_ERR_INVALID_ARG, "max_q must be >= 1");
    if (batch->max_q > TREE_MAX) return fail(TQ_ERR_UNSUPPORTED, "at most 128 nodes per sequence");
    if (!batch->cu_q && (batch->n_tokens != batch->B || batch->max_q != 1))
      return fail(TQ_ERR_INVALID_ARG, "without cu_q every sequence has one row: n_tokens == B and max_q == 1");
    if (path_stride < batch->max_q || path_stride > INT64_MAX / 8 / INT32_MAX) return fail(TQ_ERR_INVALID_ARG, "path_stride below max_q");
    if (batch->B > INT32_MAX / 64) return fail(TQ_ERR_UNSUPPORTED, "too many sequences");
    const bool rows = batch->n_tokens > 0;  // (sequences without rows: nothing of them is read)
    if ((st = check_probs(target, rows)) != TQ_OK || (draft && (st = check_probs(draft, rows)) != TQ_OK)) return st;
    if (draft && (draft->dtype != target->dtype || draft->vocab != target->vocab))
      return fail(TQ_ERR_INVALID_ARG, "the draft's rows must have the target's dtype and vocab");
    if (batch->B == 0) return TQ_OK;
    if (!u_next || (rows && (!parents || !tokens || !u_accept))) return fail(TQ_ERR_INVALID_ARG, "null parents, tokens or random numbers");
    if (!path || !n_path || !next_token) return fail(TQ_ERR_INVALID_ARG, "null output");
    if (!aligned(parents, 4) || !aligned(tokens, 4) || !aligned(u_accept, 4) || !aligned(u_next, 4) || !aligned(path, 4) ||
        !aligned(n_path, 4) || !aligned(next_token, 4) || !aligned(batch->cu_q, 4))
      return fail(TQ_ERR_ALIGNMENT, "arrays must be 4-byte aligned");
    VerifyArgs a{};
    a.cu_q = batch->cu_q, a.B = batch->B, a.max_q = batch->max_q, a.n_tokens = batch->n_tokens;
    a.parents = parents, a.tokens = tokens;
    a.target = target->data, a.target_stride = target->row_stride, a.dtype = target->dtype, a.vocab = target->vocab;
    if (draft) a.draft = draft->data, a.draft_stride = draft->row_stride;
    a.u_accept = u_accept, a.u_next = u_next;
    a.path = path, a.path_stride = path_stride, a.n_path = n_path, a.next_token = next_token, a.status = ctx->d_status;
    const cudaError_t e = launch_tree_verify(a, ctx->num_sms, (cudaStream_t)stream);
    return e == cudaSuccess ? TQ_OK : cuda_fail(e, "tq_tree_verify");
  });
}

tq_status tq_paged_tree_keep(const tq_ctx *k_ctx, const tq_ctx *v_ctx, const tq_paged_kv *kv,
                             const tq_paged_batch *batch, const int32_t *path, int64_t path_stride,
                             const int32_t *n_path, int32_t *new_lens, tq_stream_t stream) {
  return guarded([&] {
    PagedView pv;
    bool empty;
    tq_status st = check_paged(k_ctx, v_ctx, kv, batch, "tq_paged_tree_keep", &pv, &empty);
    if (st != TQ_OK) return st;
    if (batch->max_q > TREE_MAX) return fail(TQ_ERR_UNSUPPORTED, "at most 128 nodes per sequence");
    if (path_stride < 1 || path_stride > INT64_MAX / 8 / INT32_MAX) return fail(TQ_ERR_INVALID_ARG, "path_stride must be >= 1");
    if (batch->B == 0) return TQ_OK;
    if (empty) return fail(TQ_ERR_INVALID_ARG, "a batch without rows has no path to keep");
    if (!path || !n_path || !new_lens) return fail(TQ_ERR_INVALID_ARG, "null path, counts or new lengths");
    if (!aligned(path, 4) || !aligned(n_path, 4) || !aligned(new_lens, 4)) return fail(TQ_ERR_ALIGNMENT, "path, counts and new lengths must be 4-byte aligned");
    const cudaError_t e = launch_paged_keep(pv, (uint8_t *)kv->k_pages, (uint8_t *)kv->v_pages, path, path_stride, n_path,
                                            new_lens, (cudaStream_t)stream);
    return e == cudaSuccess ? TQ_OK : cuda_fail(e, "tq_paged_tree_keep");
  });
}

}  // extern "C"
