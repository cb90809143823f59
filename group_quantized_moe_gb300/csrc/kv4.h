// kv4.h -- a layer's paged cache held in 4 bits: its layout, and the host-side
// interface of the kernels that write, read and attend over it.  Not part of
// the public ABI.
//
// A block holds, for each key/value head, block_size rows in strips of 16.  A
// strip of a head is contiguous; with NC chunks of 32 dimensions (beyond four
// an even number) and G groups of 32 or 64 dimensions:
//   key codes     32-bit words [16 rows][4][NC]: nibble j of word (r, t, c) is
//                 dimension 32 c + 8 t + j of row r
//   value codes   words [2][8][4][NC]: the low half of word (h, g, t, c) belongs
//                 to row 8 h + 2 t, the high half to the row after it; nibble j
//                 of a half is dimension 32 c + 4 g + j
//   key params    words [16][G]: zero point (fp16, an integer up to 2048) in the
//                 low half, scale (bf16) in the high half
//   value params  the same
//   value = (code - zero point) scale
// These are the registers of one warp's 16 x 8 x 16 matrix products: lane
// 4 g + t reads NC consecutive words each for key rows g and g + 8, and for the
// value rows 2 t, 2 t + 1 and 2 t + 8, 2 t + 9, and a masked word is an operand
// register as it stands (attn4_rows.cu).  A row's bytes are its own, so that
// tokens are stored without a look at their neighbours.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "attn_batch.h"
#include "attn_internal.h"

namespace qmm {

struct Kv4 {
  uint8_t *data;
  int64_t num_blocks, block_stride;  // bytes between blocks
  int n_kv, head_dim;
  int nc, ng;       // chunks of a strip, groups of a row
  int cpg;          // chunks of a group: 1 or 2
  int block_shift;  // log2 of the rows of a block
};

// Chunks that a strip holds.
__host__ __device__ inline int kv4_chunks(int head_dim) {
  const int n = (head_dim + 31) / 32;
  return n <= 4 ? n : n + (n & 1);
}
__host__ __device__ inline int kv4_groups(int head_dim, int group) { return (head_dim + group - 1) / group; }
// Bytes of a strip; where its parts begin.
__host__ __device__ inline int kv4_strip(const Kv4 &c) { return 512 * c.nc + 128 * c.ng; }
__host__ __device__ inline int kv4_head_bytes(const Kv4 &c) { return kv4_strip(c) << (c.block_shift - 4); }

// The largest power of two by which query rows are scaled into fp16: scale log2(e)
// divided by it stays a normal number of fp32 (as zero it would make NaNs of masked scores).
inline int kv4_most_exponent(float sl2) {
  const int e = std::ilogb(sl2) + 126;
  return e < 100 ? e : 100;
}

// Rotary positions and the cache write (a.cached, a.k_cache, a.v_cache and the
// block fields of `a` are not used: c says where rows go).
cudaError_t launch_rope_append_kv4(const RopeAppend &a, const Kv4 &c, cudaStream_t s);

// Rows slots[i] of the cache as numbers: k, v [n, n_kv, head_dim] (either may be
// null); a slot below 0 or beyond the cache gives zeros.
cudaError_t launch_kv4_read(const Kv4 &c, const int64_t *slots, int64_t n, void *k, void *v, bool bf16,
                            cudaStream_t s);

// Attention over the cache: `a` as for the other caches, its k, v, num_blocks
// and block_stride not used.
size_t attn4_workspace_bytes(const Kv4 &c, bool q_bf16, int64_t T, int n_head, int R);
cudaError_t launch_attn4(const AttnBatch &a, const Kv4 &c, void *workspace, cudaStream_t s);

// The form for few rows.
AttnPlan attn4_rows_plan(const Kv4 &c, int n_head);
cudaError_t launch_attn4_rows(const AttnBatch &a, const Kv4 &c, const AttnPlan &p, const AttnSched &sc,
                              const AttnParts &parts, cudaStream_t s);
// The form for many (its plan is attn_tc_plan's): whether it takes a call.
bool attn4_tc_takes(const AttnBatch &a);
cudaError_t launch_attn4_tc(const AttnBatch &a, const Kv4 &c, const AttnPlan &p, const AttnSched &sc,
                            const AttnParts &parts, cudaStream_t s);

}  // namespace qmm
