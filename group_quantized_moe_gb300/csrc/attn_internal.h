// attn_internal.h -- what the batched attention kernels share.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_batch.h"
#include "attn_sched.cuh"

namespace qmm {

// Partial results of divided units: slot 2 w the unit that was open when
// worker w began, slot 2 w + 1 the one it left open; `rows` rows per slot.
struct AttnParts {
  AttnOpen *open;  // [workers]
  float2 *ml;      // [2 workers][rows] running maximum (log2 units) and sum
  float *o;        // [2 workers][rows][head_dim] sums relative to the maximum
  int rows;
};

constexpr int kWholeKeys = 512;
// How a call is cut up: rows (query rows of a unit), the query heads gsub of
// a group that one unit takes (nsub units cover the group), tokens U and keys
// KT of a tile, workers (fixed, min_run: see AttnSched).  Where requests have up
// to `whole` keys on average, and none can have more than kWholeKeys, dividing a unit
// gains less than the second launch costs, and units stay whole.
struct AttnPlan {
  int rows, gsub, nsub, U, KT, fixed, min_run, workers, whole;
};

AttnPlan attn_simt_plan(bool bf16, int64_t T, int n_head, int n_kv, int head_dim, int R);
cudaError_t launch_attn_simt(const AttnBatch &a, const AttnPlan &p, const AttnSched &sc,
                             const AttnParts &parts, cudaStream_t s);
// The form for few rows; false: not for this call.
bool attn_rows_plan(bool paged, int64_t T, int n_head, int n_kv, int head_dim, int R, AttnPlan *p);
cudaError_t launch_attn_rows(const AttnBatch &a, const AttnPlan &p, const AttnSched &sc,
                             const AttnParts &parts, cudaStream_t s);
// The form for many rows in fp32; false: not for this call.
bool attn_tile_plan(bool bf16, int64_t T, int n_head, int n_kv, int head_dim, int R, AttnPlan *p);
cudaError_t launch_attn_tile(const AttnBatch &a, const AttnPlan &p, const AttnSched &sc,
                             const AttnParts &parts, cudaStream_t s);
// The tensor-core form: whether it takes a call, its plan, its launch.
bool attn_tc_takes(const AttnBatch &a);
AttnPlan attn_tc_plan(bool paged, int64_t T, int n_head, int n_kv, int R);
cudaError_t launch_attn_tc(const AttnBatch &a, const AttnPlan &p, const AttnSched &sc,
                           const AttnParts &parts, cudaStream_t s);
cudaError_t launch_attn_join(const AttnBatch &a, const AttnPlan &p, const AttnParts &parts,
                             cudaStream_t s);

// The weight of a key that a row does not see, where some row of the tile sees
// it: a zero that the exponential never gives (its own, of a key far below the
// maximum, is +0).  A key with this weight is left out of the row's sums, since
// its value may be NaN; a NaN behind a weight of +0 is the row's to have.
__device__ __forceinline__ float unseen_weight() { return -0.0f; }
__device__ __forceinline__ bool is_unseen(float w) { return __float_as_uint(w) == 0x80000000u; }

// Four consecutive outputs, fp32 or rounded to bf16 (nearest even).
__device__ __forceinline__ void store_y4(void *y, int64_t i, float4 v, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(y) + i) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  } else {
    *reinterpret_cast<float4 *>(static_cast<float *>(y) + i) = v;
  }
}

// Output rows that belong to no request (padding before the first or behind
// the last) become zeros; worker w of n, with its first `threads` threads,
// takes its share.
__device__ __forceinline__ void zero_loose_rows(const AttnBatch &a, const AttnSched &s, int w, int n,
                                                int threads) {
  int64_t lo = s.R > 0 ? s.cu[0] : 0, hi = s.R > 0 ? s.cu[s.R] : 0;
  lo = lo < 0 ? 0 : (lo > a.T ? a.T : lo);
  hi = hi < lo ? lo : (hi > a.T ? a.T : hi);
  const int64_t per = static_cast<int64_t>(a.n_head) * a.head_dim / 4;
  const int64_t total = (lo + a.T - hi) * per;
#pragma unroll 1
  for (int64_t e = static_cast<int64_t>(w) * threads + threadIdx.x; e < total;
       e += static_cast<int64_t>(n) * threads) {
    const int64_t u = e < lo * per ? e : e - lo * per + hi * per;
    store_y4(a.y, 4 * u, make_float4(0.f, 0.f, 0.f, 0.f), a.y_bf16);
  }
}

}  // namespace qmm
