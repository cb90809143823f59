// attn_batch.h -- host-side interface between the batched attention entry
// points (attn_abi.cu) and their kernels.  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace qmm {

// One call of the batched attention: q [T, n_head, head_dim] (rows q_stride
// elements apart), keys and values either packed like q (block_table ==
// nullptr; rows k_stride / v_stride apart) or in blocks of block_size rows
// [block][n_kv][block_size][head_dim], block_stride elements apart.
struct AttnBatch {
  const void *q, *k, *v;
  bool bf16;  // q, k and v (else fp32)
  int64_t T;
  int n_head, n_kv, head_dim;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *cu, *kvl;
  int R;
  const int32_t *block_table;
  int64_t table_stride;
  int max_blocks, block_size;
  int64_t num_blocks, block_stride;
  float scale;
  void *y;
  bool y_bf16;
};

// Bytes of workspace for a call with these sizes.
size_t attn_batch_workspace_bytes(bool bf16, bool paged, int64_t T, int n_head, int n_kv,
                                  int head_dim, int R);
cudaError_t launch_attn_batch(const AttnBatch &a, void *workspace, cudaStream_t s);

cudaError_t launch_kv_plan(const int32_t *ctx, const int32_t *add, int R, int block_shift,
                           int32_t *table, int64_t table_stride, int max_blocks,
                           const int32_t *free_blocks, int64_t n_free, int64_t T, int32_t *cu,
                           int32_t *kvl, int32_t *positions, int64_t *slots, int32_t *used,
                           cudaStream_t s);

// Rotary positions and the cache write (cached: there is a cache, of num_blocks
// blocks, which may be none).
struct RopeAppend {
  const void *qkv;
  bool x_bf16;
  int64_t T, stride;
  int n_head, n_kv, head_dim;
  const int32_t *positions;
  const int64_t *slots;
  const float *cos_t, *sin_t;
  int64_t max_seq;
  void *q, *k, *v;
  bool y_bf16;
  bool cached;
  void *k_cache, *v_cache;
  int block_shift;
  int64_t num_blocks, block_stride;
};
cudaError_t launch_rope_append(const RopeAppend &a, cudaStream_t s);

constexpr int kMaxPlanRequests = 16384;

}  // namespace qmm
