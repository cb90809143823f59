// attn_entry.h -- what the entry points of the paged caches and the batched
// attention share: argument checks, and how a planned call is cut up and run.
#pragma once

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/qmm.h"
#include "attn_internal.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

template <typename... A>
int refuse(int code, const char *fmt, A... args) {
  record_error(fmt, args...);
  return code;
}

inline int cuda_refuse(cudaError_t e, const char *where) {
  return refuse(QMM_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

inline bool dtype_ok(int32_t t) { return t == QMM_F32 || t == QMM_BF16; }

inline int check_heads(const char *who, int n_head, int n_kv, int head_dim) {
  if (n_head < 1 || n_kv < 1 || n_head % n_kv != 0)
    return refuse(QMM_ERR_SHAPE, "%s: n_head (%d) must be a positive multiple of n_kv (%d)", who,
                  n_head, n_kv);
  if (head_dim < 4 || head_dim > 512 || head_dim % 4 != 0)
    return refuse(QMM_ERR_UNSUPPORTED, "%s: head_dim must be a multiple of 4 in [4, 512] (got %d)",
                  who, head_dim);
  if (n_head > 1024)
    return refuse(QMM_ERR_UNSUPPORTED, "%s: more than 1024 query heads (%d)", who, n_head);
  return QMM_OK;
}

// Lengths, tables, positions and slots lie at multiples of their element.
inline int check_ints(const char *who, std::initializer_list<const void *> i32, const void *i64 = nullptr) {
  for (const void *p : i32)
    if (!aligned(p, 4)) return refuse(QMM_ERR_ALIGN, "%s: int32 arrays must be 4-byte aligned", who);
  if (!aligned(i64, 8)) return refuse(QMM_ERR_ALIGN, "%s: int64 arrays must be 8-byte aligned", who);
  return QMM_OK;
}

inline int log2i(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

constexpr int64_t kMaxKeys = (int64_t(1) << 29) - 1;  // of one request (costs of a unit fit 32 bits)

// What both attention calls check: T query rows, the lengths, scale, output,
// workspace.
inline int check_attn(const char *who, const void *q, int64_t T, int64_t q_stride, int n_head, int n_kv,
               int head_dim, int32_t dtype, const int32_t *cu, int32_t R, float scale, const void *y,
               int32_t y_dtype, const void *ws, size_t ws_bytes, size_t need) {
  int rc = check_heads(who, n_head, n_kv, head_dim);
  if (rc) return rc;
  if (!dtype_ok(dtype) || !dtype_ok(y_dtype))
    return refuse(QMM_ERR_INVALID_ARG, "%s: dtypes must be QMM_F32 or QMM_BF16", who);
  if (T < 0 || T > (int64_t(1) << 31) - 1 || R < 0)
    return refuse(QMM_ERR_SHAPE, "%s: T must be in [0, 2^31) and the request count >= 0", who);
  if (T > kMaxKeys) return refuse(QMM_ERR_UNSUPPORTED, "%s: 2^29 rows or more", who);
  if (!(scale >= 0.0f) || std::isinf(scale))
    return refuse(QMM_ERR_INVALID_ARG, "%s: scale must be finite and positive (0: 1 / sqrt(head_dim))",
                  who);
  const int b = dtype == QMM_F32 ? 4 : 2;
  if (T > 0) {
    if (!q || !y || (R > 0 && !cu)) return refuse(QMM_ERR_INVALID_ARG, "%s: null pointer", who);
    if (q_stride < static_cast<int64_t>(n_head) * head_dim || q_stride > (int64_t(1) << 40))
      return refuse(QMM_ERR_SHAPE, "%s: q_stride is smaller than a row, or larger than 2^40", who);
    if (!aligned(q, 16) || !aligned(y, 16) || q_stride * b % 8)
      return refuse(QMM_ERR_ALIGN,
                    "%s: q and y must be 16-byte aligned and rows a multiple of 8 bytes apart "
                    "(fp32: of 16)", who);
    if (dtype == QMM_F32 && q_stride % 4)
      return refuse(QMM_ERR_ALIGN, "%s: fp32 rows must be a multiple of 16 bytes apart", who);
    if (!ws || ws_bytes < need)
      return refuse(QMM_ERR_WORKSPACE, "%s: workspace needs %zu bytes", who, need);
    if (!aligned(ws, 256))
      return refuse(QMM_ERR_ALIGN, "%s: workspace must be 256-byte aligned", who);
  }
  return QMM_OK;
}

inline float default_scale(float scale, int head_dim) {
  return scale > 0.0f ? scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(head_dim)));
}

struct PartsLayout {
  size_t open, ml, o, total;
};

inline PartsLayout parts_layout(const AttnPlan &p, int head_dim) {
  PartsLayout l;
  l.open = 0;
  l.ml = up256(sizeof(AttnOpen) * p.workers);
  l.o = l.ml + up256(sizeof(float2) * 2 * p.workers * p.rows);
  l.total = l.o + up256(sizeof(float) * 2 * p.workers * p.rows * static_cast<size_t>(head_dim));
  return l;
}

// Runs a planned call: carves the workspace, cuts the call up, launches the
// kernel and, where units may be divided, the one that joins their parts.  For
// the requests of lo + 1 to hi tokens.
template <typename Launch>
cudaError_t run_attn_plan(const AttnBatch &a, const AttnPlan &p, void *workspace, cudaStream_t s,
                          Launch launch, int lo = 0, int hi = 0x7FFFFFFF) {
  const PartsLayout l = parts_layout(p, a.head_dim);
  uint8_t *base = static_cast<uint8_t *>(workspace);
  AttnParts parts{reinterpret_cast<AttnOpen *>(base + l.open),
                  reinterpret_cast<float2 *>(base + l.ml), reinterpret_cast<float *>(base + l.o),
                  p.rows};
  const int64_t cap = a.block_table  // at most kMaxKeys: T is checked to be
                          ? min64(static_cast<int64_t>(a.max_blocks) * a.block_size, kMaxKeys)
                          : a.T;
  const int64_t usual = a.block_table || a.R < 1 ? cap : a.T / a.R;
  const bool whole = cap <= kWholeKeys && usual <= p.whole;
  AttnSched sc{a.cu, a.kvl, a.R, a.n_kv * p.nsub, p.U, log2i(p.KT), p.fixed, p.min_run,
               ~uint64_t(0) / static_cast<uint64_t>(p.workers) + 1, whole, a.T,
               static_cast<int>(cap), lo, hi};
  const cudaError_t e = launch(sc, parts);
  if (e != cudaSuccess || whole) return e;
  return launch_attn_join(a, p, parts, s);
}

}  // namespace qmm
