// attn_abi.cu -- extern "C" entry points of the paged key/value cache and the
// batched attention over it: argument validation, workspace carving and
// kernel selection.  Declared in include/qmm.h.
#include "attn_entry.h"
#include "attn_batch.h"
#include "attn_internal.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

// Blocks of a power of two of rows, large enough strides, aligned pointers.
int check_cache(const char *who, const qmm_kv_cache *c) {
  if (!c) return refuse(QMM_ERR_INVALID_ARG, "%s: null cache", who);
  if (!dtype_ok(c->dtype))
    return refuse(QMM_ERR_INVALID_ARG, "%s: cache dtype must be QMM_F32 or QMM_BF16", who);
  const int rc = check_heads(who, c->n_kv, c->n_kv, c->head_dim);
  if (rc) return rc;
  if (c->block_size < 16 || c->block_size > 256 || (c->block_size & (c->block_size - 1)))
    return refuse(QMM_ERR_UNSUPPORTED, "%s: block_size must be 16, 32, 64, 128 or 256 (got %d)",
                  who, c->block_size);
  if (c->num_blocks < 0 || c->num_blocks > (int64_t(1) << 31) - 1)
    return refuse(QMM_ERR_SHAPE, "%s: num_blocks must be in [0, 2^31)", who);
  const int64_t block = static_cast<int64_t>(c->n_kv) * c->block_size * c->head_dim;
  if (c->block_stride < block)
    return refuse(QMM_ERR_SHAPE, "%s: block_stride is smaller than a block", who);
  if (c->block_stride > (int64_t(1) << 40))
    return refuse(QMM_ERR_SHAPE, "%s: block_stride is larger than 2^40", who);
  if (c->num_blocks > 0 && (!c->k || !c->v))
    return refuse(QMM_ERR_INVALID_ARG, "%s: null cache pointer", who);
  const int b = c->dtype == QMM_F32 ? 4 : 2;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->block_stride * b % 16)
    return refuse(QMM_ERR_ALIGN, "%s: cache pointers and block_stride must be multiples of 16 bytes",
                  who);
  return QMM_OK;
}

// Memory of an argument: rows of `len` bytes, `stride` bytes apart (one row for
// a vector).
struct Span {
  const char *name;
  const void *p;
  int64_t rows, stride, len;
};

Span vec_span(const char *name, const void *p, int64_t n, int size) {
  return {name, p, 1, n * size, n * size};
}

// Whether a vector and the rows of b share a byte.
bool overlap(const Span &a, const Span &b) {
  if (a.len <= 0 || b.len <= 0 || b.rows <= 0) return false;
  const int64_t lo = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.p) - reinterpret_cast<uintptr_t>(b.p));
  const int64_t hi = lo + a.len;
  // the first row of b that ends behind lo
  int64_t r = lo <= 0 ? 0 : lo / b.stride;
  if (r * b.stride + b.len <= lo) ++r;
  return r < b.rows && r * b.stride < hi;
}

// Which kernel runs a call, and its plan.
using Launch = cudaError_t (*)(const AttnBatch &, const AttnPlan &, const AttnSched &,
                               const AttnParts &, cudaStream_t);
Launch pick_plan(bool bf16, bool tc, bool paged, int64_t T, int n_head, int n_kv, int head_dim, int R,
                 AttnPlan *p) {
  if (tc) {
    *p = attn_tc_plan(paged, T, n_head, n_kv, R);
    return launch_attn_tc;
  }
  if (attn_rows_plan(paged, T, n_head, n_kv, head_dim, R, p)) return launch_attn_rows;
  if (attn_tile_plan(bf16, T, n_head, n_kv, head_dim, R, p)) return launch_attn_tile;
  *p = attn_simt_plan(bf16, T, n_head, n_kv, head_dim, R);
  return launch_attn_simt;
}

}  // namespace

size_t attn_batch_workspace_bytes(bool bf16, bool paged, int64_t T, int n_head, int n_kv, int head_dim, int R) {
  // whether a bf16 call takes the tensor cores also depends on its strides
  AttnPlan p;
  pick_plan(bf16, false, paged, T, n_head, n_kv, head_dim, R, &p);
  const size_t simt = parts_layout(p, head_dim).total;
  const size_t tc = bf16 && head_dim <= 128 ? parts_layout(attn_tc_plan(paged, T, n_head, n_kv, R), head_dim).total : 0;
  return simt > tc ? simt : tc;
}

cudaError_t launch_attn_batch(const AttnBatch &a, void *workspace, cudaStream_t s) {
  AttnPlan p;
  const Launch launch =
      pick_plan(a.bf16, attn_tc_takes(a), a.block_table != nullptr, a.T, a.n_head, a.n_kv, a.head_dim, a.R, &p);
  return run_attn_plan(a, p, workspace, s, [&](const AttnSched &sc, const AttnParts &parts) {
    return launch(a, p, sc, parts, s);
  });
}

}  // namespace qmm

using namespace qmm;

extern "C" {

int qmm_kv_plan(const int32_t *ctx_lens, const int32_t *new_lens, int32_t R, int32_t block_size,
                int32_t *block_table, int64_t table_stride, int32_t max_blocks,
                const int32_t *free_blocks, int64_t n_free, int64_t T, int32_t *cu_new,
                int32_t *kv_lens, int32_t *positions, int64_t *slots, int32_t *blocks_used,
                qmm_stream_t stream) {
  const char *who = "qmm_kv_plan";
  record_error("%s", "");
  if (R < 0 || T < 0 || T > (int64_t(1) << 31) - 1 || max_blocks < 0 || n_free < 0)
    return refuse(QMM_ERR_SHAPE, "%s: negative size, or T >= 2^31", who);
  if (R > kMaxPlanRequests)
    return refuse(QMM_ERR_UNSUPPORTED, "%s: more than %d requests (%d)", who, kMaxPlanRequests, R);
  if (block_size < 16 || block_size > 256 || (block_size & (block_size - 1)))
    return refuse(QMM_ERR_UNSUPPORTED, "%s: block_size must be 16, 32, 64, 128 or 256 (got %d)",
                  who, block_size);
  if (table_stride < max_blocks || table_stride > (int64_t(1) << 31))
    return refuse(QMM_ERR_SHAPE, "%s: table_stride must be in [max_blocks, 2^31]", who);
  if (!cu_new || !blocks_used || (R > 0 && (!ctx_lens || !new_lens || !kv_lens)) ||
      (R > 0 && max_blocks > 0 && !block_table) || (n_free > 0 && !free_blocks) ||
      (T > 0 && (!positions || !slots)))
    return refuse(QMM_ERR_INVALID_ARG, "%s: null pointer", who);
  const int rc = check_ints(who, {ctx_lens, new_lens, block_table, free_blocks, cu_new, kv_lens,
                                  positions, blocks_used}, slots);
  if (rc) return rc;
  // Every block of the launch reads the lengths and the free list from first to
  // last, so none of the outputs may lie on them (or on one another).
  const Span span[] = {vec_span("cu_new", cu_new, R + int64_t(1), 4),
                       vec_span("kv_lens", kv_lens, R, 4),
                       vec_span("positions", positions, T, 4),
                       vec_span("slots", slots, T, 8),
                       vec_span("blocks_used", blocks_used, 1, 4),
                       vec_span("ctx_lens", ctx_lens, R, 4),
                       vec_span("new_lens", new_lens, R, 4),
                       vec_span("free_blocks", free_blocks, n_free, 4)};
  const Span table{"block_table", block_table, R, table_stride * 4, int64_t(max_blocks) * 4};
  for (int i = 0; i < 8; ++i) {
    for (int j = i + 1; i < 5 && j < 8; ++j)
      if (overlap(span[i], span[j]))
        return refuse(QMM_ERR_INVALID_ARG, "%s: %s overlaps %s", who, span[i].name, span[j].name);
    if (overlap(span[i], table))
      return refuse(QMM_ERR_INVALID_ARG, "%s: %s overlaps %s", who, span[i].name, table.name);
  }
  const cudaError_t e = launch_kv_plan(
      ctx_lens, new_lens, R, log2i(block_size), block_table, table_stride, max_blocks, free_blocks,
      n_free, T, cu_new, kv_lens, positions, slots, blocks_used, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QMM_OK : cuda_refuse(e, who);
}

int qmm_rope_append(const void *qkv, int32_t x_dtype, int64_t T, int64_t row_stride, int32_t n_head,
                    int32_t n_kv, int32_t head_dim, const int32_t *positions, const int64_t *slots,
                    const float *rope_cos, const float *rope_sin, int64_t max_seq,
                    const qmm_kv_cache *cache, void *q, void *k, void *v, int32_t y_dtype,
                    qmm_stream_t stream) {
  const char *who = "qmm_rope_append";
  record_error("%s", "");
  int rc = check_heads(who, n_head, n_kv, head_dim);
  if (rc) return rc;
  if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype))
    return refuse(QMM_ERR_INVALID_ARG, "%s: dtypes must be QMM_F32 or QMM_BF16", who);
  if (T < 0 || max_seq < 0 || max_seq > (int64_t(1) << 31))
    return refuse(QMM_ERR_SHAPE, "%s: T must be >= 0 and max_seq in [0, 2^31]", who);
  if (cache) {
    rc = check_cache(who, cache);
    if (rc) return rc;
    if (cache->n_kv != n_kv || cache->head_dim != head_dim || cache->dtype != y_dtype)
      return refuse(QMM_ERR_SHAPE, "%s: the cache has other heads or another type than the outputs",
                    who);
  }
  if (T == 0) return QMM_OK;
  if (!qkv || !positions || !q || (cache && !slots) || (max_seq > 0 && (!rope_cos || !rope_sin)))
    return refuse(QMM_ERR_INVALID_ARG, "%s: null pointer", who);
  const int64_t row = (static_cast<int64_t>(n_head) + 2 * n_kv) * head_dim;
  if (row_stride < row || row_stride > (int64_t(1) << 40))
    return refuse(QMM_ERR_SHAPE, "%s: row_stride is smaller than a row, or larger than 2^40", who);
  if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(rope_cos, 16) || !aligned(rope_sin, 16) || row_stride % 4)
    return refuse(QMM_ERR_ALIGN,
                  "%s: tensors must be 16-byte aligned and rows a multiple of 4 elements apart", who);
  if ((rc = check_ints(who, {positions}, slots))) return rc;
  RopeAppend a{};
  a.qkv = qkv;
  a.x_bf16 = x_dtype == QMM_BF16;
  a.T = T;
  a.stride = row_stride;
  a.n_head = n_head;
  a.n_kv = n_kv;
  a.head_dim = head_dim;
  a.positions = positions;
  a.slots = slots;
  a.cos_t = rope_cos;
  a.sin_t = rope_sin;
  a.max_seq = max_seq;
  a.q = q;
  a.k = k;
  a.v = v;
  a.y_bf16 = y_dtype == QMM_BF16;
  if (cache) {
    a.cached = true;
    a.k_cache = cache->k;
    a.v_cache = cache->v;
    a.num_blocks = cache->num_blocks;
    a.block_stride = cache->block_stride;
    a.block_shift = log2i(cache->block_size);
  }
  const cudaError_t e = launch_rope_append(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QMM_OK : cuda_refuse(e, who);
}

size_t qmm_attn_prompt_workspace_bytes(int32_t dtype, int64_t T, int32_t n_head, int32_t n_kv,
                                       int32_t head_dim, int32_t n_seqs) {
  if (!dtype_ok(dtype) || check_heads("qmm_attn_prompt_workspace_bytes", n_head, n_kv, head_dim) ||
      T < 0 || n_seqs < 0)
    return 0;
  return attn_batch_workspace_bytes(dtype == QMM_BF16, false, T, n_head, n_kv, head_dim, n_seqs);
}

int qmm_attn_prompt(const void *q, const void *k, const void *v, int32_t dtype, int64_t T,
                    int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t n_head,
                    int32_t n_kv, int32_t head_dim, const int32_t *cu_seqlens, int32_t n_seqs,
                    float scale, void *y, int32_t y_dtype, void *workspace, size_t workspace_bytes,
                    qmm_stream_t stream) {
  const char *who = "qmm_attn_prompt";
  record_error("%s", "");
  const size_t need =
      qmm_attn_prompt_workspace_bytes(dtype, T, n_head, n_kv, head_dim, n_seqs);
  int rc = check_attn(who, q, T, q_stride, n_head, n_kv, head_dim, dtype, cu_seqlens, n_seqs, scale,
                      y, y_dtype, workspace, workspace_bytes, need);
  if (rc || T == 0) return rc;
  const int64_t row = static_cast<int64_t>(n_kv) * head_dim;
  if (!k || !v) return refuse(QMM_ERR_INVALID_ARG, "%s: null pointer", who);
  if (k_stride < row || v_stride < row || k_stride > (int64_t(1) << 40) ||
      v_stride > (int64_t(1) << 40))
    return refuse(QMM_ERR_SHAPE, "%s: k_stride or v_stride is smaller than a row, or larger than 2^40",
                  who);
  if (!aligned(k, 16) || !aligned(v, 16) || k_stride % 4 || v_stride % 4)
    return refuse(QMM_ERR_ALIGN, "%s: k and v must be 16-byte aligned, rows a multiple of 4 elements "
                  "apart", who);
  if ((rc = check_ints(who, {cu_seqlens}))) return rc;
  AttnBatch a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.bf16 = dtype == QMM_BF16;
  a.T = T;
  a.n_head = n_head;
  a.n_kv = n_kv;
  a.head_dim = head_dim;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cu = cu_seqlens;
  a.R = n_seqs;
  a.scale = default_scale(scale, head_dim);
  a.y = y;
  a.y_bf16 = y_dtype == QMM_BF16;
  const cudaError_t e = launch_attn_batch(a, workspace, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QMM_OK : cuda_refuse(e, who);
}

size_t qmm_attn_paged_workspace_bytes(const qmm_kv_cache *cache, int64_t T, int32_t n_head,
                                      int32_t R) {
  const char *who = "qmm_attn_paged_workspace_bytes";
  if (!cache || !dtype_ok(cache->dtype) || check_heads(who, n_head, cache->n_kv, cache->head_dim) ||
      T < 0 || R < 0)
    return 0;
  return attn_batch_workspace_bytes(cache->dtype == QMM_BF16, true, T, n_head, cache->n_kv,
                                    cache->head_dim, R);
}

int qmm_attn_paged(const void *q, int64_t T, int64_t q_stride, int32_t n_head,
                   const qmm_kv_cache *cache, const int32_t *block_table, int64_t table_stride,
                   int32_t max_blocks, const int32_t *cu_q, const int32_t *kv_lens, int32_t R,
                   float scale, void *y, int32_t y_dtype, void *workspace, size_t workspace_bytes,
                   qmm_stream_t stream) {
  const char *who = "qmm_attn_paged";
  record_error("%s", "");
  int rc = check_cache(who, cache);
  if (rc) return rc;
  const size_t need = qmm_attn_paged_workspace_bytes(cache, T, n_head, R);
  rc = check_attn(who, q, T, q_stride, n_head, cache->n_kv, cache->head_dim, cache->dtype, cu_q, R,
                  scale, y, y_dtype, workspace, workspace_bytes, need);
  if (rc) return rc;
  if (max_blocks < 0 || table_stride < max_blocks || table_stride > (int64_t(1) << 31))
    return refuse(QMM_ERR_SHAPE, "%s: table_stride must be in [max_blocks, 2^31]", who);
  if (T == 0) return QMM_OK;
  if (R > 0 && (!kv_lens || !block_table))
    return refuse(QMM_ERR_INVALID_ARG, "%s: null pointer", who);
  if ((rc = check_ints(who, {cu_q, kv_lens, block_table}))) return rc;
  AttnBatch a{};
  a.q = q;
  a.k = cache->k;
  a.v = cache->v;
  a.bf16 = cache->dtype == QMM_BF16;
  a.T = T;
  a.n_head = n_head;
  a.n_kv = cache->n_kv;
  a.head_dim = cache->head_dim;
  a.q_stride = q_stride;
  a.cu = cu_q;
  a.kvl = kv_lens;
  a.R = R;
  static const int32_t none = 0;
  a.block_table = block_table ? block_table : &none;  // R == 0: never read, marks the paged form
  a.table_stride = table_stride;
  a.max_blocks = max_blocks;
  a.block_size = cache->block_size;
  a.num_blocks = cache->num_blocks;
  a.block_stride = cache->block_stride;
  a.scale = default_scale(scale, cache->head_dim);
  a.y = y;
  a.y_bf16 = y_dtype == QMM_BF16;
  const cudaError_t e = launch_attn_batch(a, workspace, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QMM_OK : cuda_refuse(e, who);
}

}  // extern "C"
