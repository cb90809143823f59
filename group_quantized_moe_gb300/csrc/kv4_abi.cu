// kv4_abi.cu -- extern "C" entry points of the paged cache held in 4 bits:
// argument validation and kernel selection.  Declared in include/qmm.h.
#include "attn_entry.h"
#include "kv4.h"

namespace qmm {
namespace {

int check_form(const char *who, int n_kv, int head_dim, int group, int block_size) {
  const int rc = check_heads(who, n_kv, n_kv, head_dim);
  if (rc) return rc;
  if (head_dim % 8 != 0 || head_dim > 256)
    return refuse(QMM_ERR_UNSUPPORTED, "%s: head_dim must be a multiple of 8 in [8, 256] (got %d)", who, head_dim);
  if (group != 32 && group != 64)
    return refuse(QMM_ERR_UNSUPPORTED, "%s: group must be 32 or 64 (got %d)", who, group);
  if (block_size < 16 || block_size > 256 || (block_size & (block_size - 1)))
    return refuse(QMM_ERR_UNSUPPORTED, "%s: block_size must be 16, 32, 64, 128 or 256 (got %d)", who, block_size);
  return QMM_OK;
}

Kv4 form(int n_kv, int head_dim, int group, int block_size) {
  Kv4 c{};
  c.n_kv = n_kv;
  c.head_dim = head_dim;
  c.nc = kv4_chunks(head_dim);
  c.ng = kv4_groups(head_dim, group);
  c.cpg = group / 32;
  c.block_shift = log2i(block_size);
  return c;
}

int64_t block_bytes(const Kv4 &c) { return static_cast<int64_t>(c.n_kv) * kv4_head_bytes(c); }

// A cache the kernels can take, and what they are given of it.
int check_kv4(const char *who, const qmm_kv4_cache *c, Kv4 *out) {
  if (!c) return refuse(QMM_ERR_INVALID_ARG, "%s: null cache", who);
  const int rc = check_form(who, c->n_kv, c->head_dim, c->group, c->block_size);
  if (rc) return rc;
  if (c->num_blocks < 0 || c->num_blocks > (int64_t(1) << 31) - 1)
    return refuse(QMM_ERR_SHAPE, "%s: num_blocks must be in [0, 2^31)", who);
  *out = form(c->n_kv, c->head_dim, c->group, c->block_size);
  if (c->block_stride < block_bytes(*out))
    return refuse(QMM_ERR_SHAPE, "%s: block_stride is smaller than a block", who);
  if (c->block_stride > (int64_t(1) << 31))
    return refuse(QMM_ERR_SHAPE, "%s: block_stride is larger than 2^31", who);
  if (c->num_blocks > 0 && !c->data) return refuse(QMM_ERR_INVALID_ARG, "%s: null cache pointer", who);
  if (!aligned(c->data, 16) || c->block_stride % 16)
    return refuse(QMM_ERR_ALIGN, "%s: the cache and its block_stride must be multiples of 16 bytes", who);
  out->data = static_cast<uint8_t *>(c->data);
  out->num_blocks = c->num_blocks;
  out->block_stride = c->block_stride;
  return QMM_OK;
}

}  // namespace

namespace {

// Which form a call takes.  The form for few query rows reads a cache faster and
// begins sooner, the one for many costs hardly more with each row.  Rows per
// request and key/value head, few / many in us (32 heads of 128 over 8, groups
// of 64):
//   40 requests of 2000 keys    24: 99 / 116    32: 126 / 117   40: 155 / 120
//    8 requests of 16000 keys   24: 109 / 139   32: 138 / 139   40: 168 / 142
//  300 requests of 400 keys     16: 244 / 262   24: 354 / 268   32: 463 / 273
//    4 requests of 6000 keys    32: 45 / 47     40: 52 / 48     48: 59 / 49
// so kRows = 32.
// Where a call has chunks and may have single tokens beside them, each takes its
// own.  How long a request is stands on the device only, so both forms are launched
// and find their requests there, which costs 7 to 15 us where one has none.  One
// chunk and single tokens, 3000 keys each, few / many / both:
//   chunk of 64     20 requests  66 / 99 / 81     64 requests   99 / 257 / 131
//   chunk of 256     2 requests 126 / 59 / 73     20 requests  140 / 119 / 92
//                   64 requests 174 / 274 / 135
//   chunk of 1024    2 requests 390 / 92 / 106    64 requests  445 / 326 / 168
// so both from kMixed = 6 requests on (a single token costs the form for many about
// 3.5 us), and from kLong = 512 rows beyond a token a request; twice that where the
// average is for the form for few, as then the rows may be drafts of all requests
// (30 of up to 5 tokens, 28 heads over 4: 53 us, both 70).
struct Split {
  bool few, many;
  int tokens;  // of a request, up to which it goes to the form for few
};

Split split_rows(const Kv4 &c, int64_t T, int n_head, int R) {
  constexpr int kRows = 32, kLong = 512, kMixed = 6;
  const int64_t grp = n_head / c.n_kv;
  const bool many = T * grp > static_cast<int64_t>(kRows) * R;
  if (R >= kMixed && (T - R) * grp >= (many ? kLong : 2 * kLong)) return {true, true, static_cast<int>(kRows / grp)};
  return {!many, many, 0};
}

}  // namespace

size_t attn4_workspace_bytes(const Kv4 &c, bool q_bf16, int64_t T, int n_head, int R) {
  // whether a call takes the form for many rows also depends on its stride
  const size_t few = parts_layout(attn4_rows_plan(c, n_head), c.head_dim).total;
  if (!q_bf16 || c.head_dim > 128) return few;
  const Split f = split_rows(c, T, n_head, R);
  const size_t many = f.many ? parts_layout(attn_tc_plan(true, T, n_head, c.n_kv, R), c.head_dim).total : 0;
  return f.few ? few + many : many > few ? many : few;
}

cudaError_t launch_attn4(const AttnBatch &a, const Kv4 &c, void *workspace, cudaStream_t s) {
  const AttnPlan few = attn4_rows_plan(c, a.n_head);
  const auto run_few = [&](const AttnSched &sc, const AttnParts &parts) {
    return launch_attn4_rows(a, c, few, sc, parts, s);
  };
  const Split f = split_rows(c, a.T, a.n_head, a.R);
  if (!f.many || !attn4_tc_takes(a)) return run_attn_plan(a, few, workspace, s, run_few);
  const AttnPlan many = attn_tc_plan(true, a.T, a.n_head, a.n_kv, a.R);
  const auto run_many = [&](const AttnSched &sc, const AttnParts &parts) {
    return launch_attn4_tc(a, c, many, sc, parts, s);
  };
  if (!f.few) return run_attn_plan(a, many, workspace, s, run_many);
  const cudaError_t e = run_attn_plan(a, few, workspace, s, run_few, 0, f.tokens);
  if (e != cudaSuccess) return e;
  return run_attn_plan(a, many, static_cast<uint8_t *>(workspace) + parts_layout(few, c.head_dim).total, s, run_many,
                       f.tokens);
}

}  // namespace qmm

using namespace qmm;

extern "C" {

int64_t qmm_kv4_block_bytes(int32_t n_kv, int32_t head_dim, int32_t group, int32_t block_size) {
  record_error("%s", "");
  if (check_form("qmm_kv4_block_bytes", n_kv, head_dim, group, block_size)) return 0;
  return block_bytes(form(n_kv, head_dim, group, block_size));
}

int qmm_rope_append_kv4(const void *qkv, int32_t x_dtype, int64_t T, int64_t row_stride, int32_t n_head,
                        const int32_t *positions, const int64_t *slots, const float *rope_cos,
                        const float *rope_sin, int64_t max_seq, const qmm_kv4_cache *cache, void *q, void *k,
                        void *v, int32_t y_dtype, qmm_stream_t stream) {
  const char *who = "qmm_rope_append_kv4";
  record_error("%s", "");
  Kv4 c;
  int rc = check_kv4(who, cache, &c);
  if (rc) return rc;
  if ((rc = check_heads(who, n_head, c.n_kv, c.head_dim))) return rc;
  if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype))
    return refuse(QMM_ERR_INVALID_ARG, "%s: dtypes must be QMM_F32 or QMM_BF16", who);
  if (T < 0 || max_seq < 0 || max_seq > (int64_t(1) << 31))
    return refuse(QMM_ERR_SHAPE, "%s: T must be >= 0 and max_seq in [0, 2^31]", who);
  if (T == 0) return QMM_OK;
  if (!qkv || !positions || !slots || !q || (max_seq > 0 && (!rope_cos || !rope_sin)))
    return refuse(QMM_ERR_INVALID_ARG, "%s: null pointer", who);
  const int64_t row = (static_cast<int64_t>(n_head) + 2 * c.n_kv) * c.head_dim;
  if (row_stride < row || row_stride > (int64_t(1) << 40))
    return refuse(QMM_ERR_SHAPE, "%s: row_stride is smaller than a row, or larger than 2^40", who);
  if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(rope_cos, 16) || !aligned(rope_sin, 16) || row_stride % (x_dtype == QMM_F32 ? 4 : 8))
    return refuse(QMM_ERR_ALIGN, "%s: tensors must be 16-byte aligned and rows a multiple of 16 bytes apart", who);
  if ((rc = check_ints(who, {positions}, slots))) return rc;
  RopeAppend a{};
  a.qkv = qkv;
  a.x_bf16 = x_dtype == QMM_BF16;
  a.T = T;
  a.stride = row_stride;
  a.n_head = n_head;
  a.n_kv = c.n_kv;
  a.head_dim = c.head_dim;
  a.positions = positions;
  a.slots = slots;
  a.cos_t = rope_cos;
  a.sin_t = rope_sin;
  a.max_seq = max_seq;
  a.q = q;
  a.k = k;
  a.v = v;
  a.y_bf16 = y_dtype == QMM_BF16;
  const cudaError_t e = launch_rope_append_kv4(a, c, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QMM_OK : cuda_refuse(e, who);
}

int qmm_kv4_read(const qmm_kv4_cache *cache, const int64_t *slots, int64_t n, void *k, void *v, int32_t y_dtype,
                 qmm_stream_t stream) {
  const char *who = "qmm_kv4_read";
  record_error("%s", "");
  Kv4 c;
  int rc = check_kv4(who, cache, &c);
  if (rc) return rc;
  if (!dtype_ok(y_dtype)) return refuse(QMM_ERR_INVALID_ARG, "%s: dtypes must be QMM_F32 or QMM_BF16", who);
  if (n < 0) return refuse(QMM_ERR_SHAPE, "%s: n must be >= 0", who);
  if (n == 0) return QMM_OK;
  if (!slots || (!k && !v)) return refuse(QMM_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned(k, 16) || !aligned(v, 16))
    return refuse(QMM_ERR_ALIGN, "%s: outputs must be 16-byte aligned", who);
  if ((rc = check_ints(who, {}, slots))) return rc;
  const cudaError_t e = launch_kv4_read(c, slots, n, k, v, y_dtype == QMM_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QMM_OK : cuda_refuse(e, who);
}

size_t qmm_attn_paged_kv4_workspace_bytes(const qmm_kv4_cache *cache, int32_t q_dtype, int64_t T, int32_t n_head,
                                          int32_t R) {
  const char *who = "qmm_attn_paged_kv4_workspace_bytes";
  if (!cache || check_form(who, cache->n_kv, cache->head_dim, cache->group, cache->block_size) ||
      check_heads(who, n_head, cache->n_kv, cache->head_dim) || !dtype_ok(q_dtype) || T < 0 || R < 0)
    return 0;
  return attn4_workspace_bytes(form(cache->n_kv, cache->head_dim, cache->group, cache->block_size),
                               q_dtype == QMM_BF16, T, n_head, R);
}

int qmm_attn_paged_kv4(const void *q, int32_t q_dtype, int64_t T, int64_t q_stride, int32_t n_head,
                       const qmm_kv4_cache *cache, const int32_t *block_table, int64_t table_stride,
                       int32_t max_blocks, const int32_t *cu_q, const int32_t *kv_lens, int32_t R, float scale,
                       void *y, int32_t y_dtype, void *workspace, size_t workspace_bytes, qmm_stream_t stream) {
  const char *who = "qmm_attn_paged_kv4";
  record_error("%s", "");
  Kv4 c;
  int rc = check_kv4(who, cache, &c);
  if (rc) return rc;
  const size_t need = qmm_attn_paged_kv4_workspace_bytes(cache, q_dtype, T, n_head, R);
  rc = check_attn(who, q, T, q_stride, n_head, c.n_kv, c.head_dim, q_dtype, cu_q, R, scale, y, y_dtype, workspace,
                  workspace_bytes, need);
  if (rc) return rc;
  if (max_blocks < 0 || table_stride < max_blocks || table_stride > (int64_t(1) << 31))
    return refuse(QMM_ERR_SHAPE, "%s: table_stride must be in [max_blocks, 2^31]", who);
  if (T == 0) return QMM_OK;
  if (R > 0 && (!kv_lens || !block_table)) return refuse(QMM_ERR_INVALID_ARG, "%s: null pointer", who);
  if ((rc = check_ints(who, {cu_q, kv_lens, block_table}))) return rc;
  AttnBatch a{};
  a.q = q;
  a.bf16 = q_dtype == QMM_BF16;
  a.T = T;
  a.n_head = n_head;
  a.n_kv = c.n_kv;
  a.head_dim = c.head_dim;
  a.q_stride = q_stride;
  a.cu = cu_q;
  a.kvl = kv_lens;
  a.R = R;
  static const int32_t none = 0;
  a.block_table = block_table ? block_table : &none;  // R == 0: never read, marks the paged form
  a.table_stride = table_stride;
  a.max_blocks = max_blocks;
  a.block_size = cache->block_size;
  a.scale = default_scale(scale, c.head_dim);
  a.y = y;
  a.y_bf16 = y_dtype == QMM_BF16;
  const cudaError_t e = launch_attn4(a, c, workspace, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QMM_OK : cuda_refuse(e, who);
}

}  // extern "C"
