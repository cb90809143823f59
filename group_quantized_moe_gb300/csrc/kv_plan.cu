// kv_plan.cu -- block tables and slot maps of a paged key/value cache, from
// the requests' lengths.
//
// With S rows per block, request r holding c_r rows and adding n_r:
//   have_r = ceil(c_r / S), need_r = ceil((c_r + n_r) / S)
//   f_r    = sum_{i < r} (need_i - have_i)     (its place in the free list)
//   table[r, have_r + j] = free[f_r + j]       j < need_r - have_r
//   cu_r   = sum_{i < r} n_i
//   token t of the packed batch, in request r: position p = c_r + t - cu_r,
//   slot = table[r, p / S] * S + p % S
//
// The two prefix sums over the requests are all that the tokens depend on,
// and they are short (a few thousand lengths) next to a grid-wide barrier or
// a second launch, so every CTA forms both in its own shared memory and then
// takes its share of the tokens; one launch, no communication.  A token finds
// its request by bisecting the prefix sums in shared memory, and a block that
// this call hands out is read from the free list, never from the table rows
// that another CTA may be writing.
//
// Sums and positions are formed in 64 bits and stop at 2^31 - 1 where they are
// kept, so that lengths beyond all reason end in tokens without a slot and a
// flag, not in negative lengths.
//
// A few hundred kilobytes at most: bound by latency.  3.8 us for 256 single
// tokens, 6.8 us for 4096 requests (a launch that does nothing takes 2).
#include <cstdint>

#include "attn_batch.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kPlanThreads = 1024;

struct PlanArgs {
  const int32_t *ctx, *add;
  int R, shift;
  int32_t *table;
  int64_t table_stride;
  int max_blocks;
  const int32_t *free_blocks;
  int64_t n_free, T;
  int32_t *cu, *kvl, *positions;
  int64_t *slots;
  int32_t *used;
  uint32_t *status;
};

__device__ __forceinline__ int held(int64_t v) { return static_cast<int>(min64(v, 0x7FFFFFFF)); }

struct Sums {
  int64_t tokens, blocks;
};

// Inclusive sums over the lanes of a warp.
__device__ __forceinline__ Sums warp_sums(Sums v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, v.tokens, o);
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, v.blocks, o);
    if (lane >= o) {
      v.tokens += x;
      v.blocks += y;
    }
  }
  return v;
}

// Largest index r in [0, n) with v[r] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int last_at_most(const int32_t *v, int n, int x) {
  int a = 0, b = n;
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (v[mid] <= x) a = mid;
    else b = mid;
  }
  return a;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(PlanArgs a) {
  extern __shared__ int32_t sm[];
  int32_t *cu = sm, *blk = sm + a.R + 1;  // exclusive prefixes, [R + 1] each
  __shared__ Sums warp_tot[kPlanThreads / 32];
  __shared__ uint32_t flags;
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S1 = (1 << a.shift) - 1;
  if (tid == 0) flags = 0;
  const int per = (a.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  // a length below zero counts as zero; rows beyond the table's columns get
  // no block (their tokens have no slot)
  const int64_t cap = static_cast<int64_t>(a.max_blocks) << a.shift;
  auto lens = [&](int r, int &c, int &n, int &fresh) {
    c = max(a.ctx[r], 0);
    n = max(a.add[r], 0);
    const int64_t end = static_cast<int64_t>(c) + n;
    const int have = static_cast<int>(min64(c + static_cast<int64_t>(S1), cap) >> a.shift);
    const int need = static_cast<int>(min64(end + S1, cap) >> a.shift);
    fresh = max(need - have, 0);
    return end > cap;
  };
  Sums sum{0, 0};
  bool over = false;
  for (int r = r0; r < r1; ++r) {
    int c, n, fresh;
    over |= lens(r, c, n, fresh);
    sum.tokens += n;
    sum.blocks += fresh;
  }
  const Sums inc = warp_sums(sum, lane);
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const Sums own = warp_tot[lane], t = warp_sums(own, lane);
    if (lane == 31) {
      cu[a.R] = held(t.tokens);
      blk[a.R] = held(t.blocks);
    }
    warp_tot[lane] = Sums{t.tokens - own.tokens, t.blocks - own.blocks};
  }
  __syncthreads();
  int64_t at = warp_tot[warp].tokens + inc.tokens - sum.tokens;
  int64_t bt = warp_tot[warp].blocks + inc.blocks - sum.blocks;
  for (int r = r0; r < r1; ++r) {
    int c, n, fresh;
    lens(r, c, n, fresh);
    cu[r] = held(at);
    blk[r] = held(bt);
    at += n;
    bt += fresh;
  }
  if (over) atomicOr(&flags, kDevKvShort);
  __syncthreads();
  const int total = cu[a.R], fresh_total = blk[a.R];
  const int g = blockIdx.x * kPlanThreads + tid, gs = gridDim.x * kPlanThreads;
  for (int r = g; r <= a.R; r += gs) a.cu[r] = cu[r];
  for (int r = g; r < a.R; r += gs) a.kvl[r] = held(static_cast<int64_t>(max(a.ctx[r], 0)) + max(a.add[r], 0));
  if (g == 0) {
    *a.used = fresh_total;
    if (flags || fresh_total > a.n_free || total > a.T) atomicOr(a.status, kDevKvShort);
  }
  // the blocks handed out (beyond the free list: -1)
  for (int64_t f = g; f < fresh_total; f += gs) {
    const int r = last_at_most(blk, a.R, static_cast<int>(f));
    const int have = static_cast<int>(min64(static_cast<int64_t>(max(a.ctx[r], 0)) + S1, cap) >> a.shift);
    a.table[r * a.table_stride + have + (f - blk[r])] = f < a.n_free ? a.free_blocks[f] : -1;
  }
  // the tokens
  for (int64_t t = g; t < a.T; t += gs) {
    int32_t p = -1;
    int64_t slot = -1;
    if (t < total) {
      const int r = last_at_most(cu, a.R, static_cast<int>(t));
      const int c = max(a.ctx[r], 0);
      const int64_t pos = c + (t - cu[r]), b = pos >> a.shift;
      p = held(pos);
      if (b < a.max_blocks) {
        const int64_t have = (static_cast<int64_t>(c) + S1) >> a.shift;
        const int64_t f = blk[r] + b - have;
        const int id = b < have ? a.table[r * a.table_stride + b]
                                : (f >= 0 && f < a.n_free ? a.free_blocks[f] : -1);
        if (id >= 0) slot = (static_cast<int64_t>(id) << a.shift) + (pos & S1);
      }
    }
    a.positions[t] = p;
    a.slots[t] = slot;
  }
}

}  // namespace

cudaError_t launch_kv_plan(const int32_t *ctx, const int32_t *add, int R, int block_shift,
                           int32_t *table, int64_t table_stride, int max_blocks,
                           const int32_t *free_blocks, int64_t n_free, int64_t T, int32_t *cu,
                           int32_t *kvl, int32_t *positions, int64_t *slots, int32_t *used,
                           cudaStream_t s) {
  PlanArgs a{ctx, add, R, block_shift, table, table_stride, max_blocks, free_blocks, n_free, T,
             cu, kvl, positions, slots, used, device_status()};
  if (!a.status) return cudaErrorInvalidDevice;
  const int smem = 2 * (R + 1) * 4;
  cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kv_plan_kernel), smem);
  if (e != cudaSuccess) return e;
  // an idle step, without requests and tokens, still writes cu[0] and *used
  const int64_t work = T > R ? T : R;
  int64_t blocks = work > 0 ? (work + kPlanThreads - 1) / kPlanThreads : 1;
  if (blocks > sm_count()) blocks = sm_count();
  return launch_pdl(kv_plan_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kPlanThreads), smem,
                    s, a);
}

}  // namespace qmm
