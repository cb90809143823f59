// attn_sched.cuh -- how the batched attention kernels share their work out.
//
// A call has R requests; request r has n new tokens (query rows) and L cache
// rows, and token t of it sees the keys 0 .. L - n + t that the block table can
// hold (where L is beyond it, the later keys are left out and the rest of the
// mask stays where it is).  A unit of work is
// (request, block of U consecutive tokens, key/value head); its cost is the
// number of keys its last token sees, and `fixed` keys more for what a unit
// costs besides them (loading its queries, writing its results).  The units
// are laid end to end in the order (request, token block, head) and the cost
// W of the whole call is cut into equal runs of `step`, worker w's being
// [w step, (w + 1) step): every worker gets the same work whatever the lengths
// are, and a long context is split over as many workers as its share of the
// work asks for.  A tile of KT keys
// belongs to the run that holds its first key.  A unit that a cut divides
// leaves one partial result per worker, merged afterwards in worker order,
// so results are reproducible bit for bit.
//
// Costs are counted in keys, not in tiles, because the cost of a request's
// token blocks then grows by U from block to block and a prefix of them is
// a quadratic; with tiles it is a sum of rounded quotients, whose closed form
// (Euclid's steps) took a thread 12 us on a call of nine prompts.
//
// Everything here is computed on the device from the lengths (a call can be
// captured in a graph and replayed with other lengths in the same buffers).
#pragma once

#include <cstdint>

#include "qmm_device.cuh"

namespace qmm {

struct AttnSched {
  const int32_t *cu;   // [R + 1] prefix sum of the new tokens
  const int32_t *kvl;  // [R] cache rows, or nullptr: the new tokens themselves
  int R;
  int nvh;             // key/value heads (times the splits of a large query group)
  int U;               // tokens per unit
  int kt_shift;        // log2 of the keys per tile
  int fixed;           // cost of a unit besides its keys
  int min_run;         // a worker's run costs at least this much (KT or more, so
                       // that no run inside a unit is without a tile of it)
  uint64_t per_worker; // 2^64 / workers, rounded up
  bool whole;          // units are not divided: each goes to the run that holds its start
  int64_t T;           // query rows in the buffers
  int cap;             // keys the block table can hold (below 2^29)
};

struct AttnReq {
  int q0, n;  // first query row, new tokens
  int ctx;    // cache rows before them (L - n): token t sees ctx + t + 1 keys
};

// Request r, held inside the buffers whatever the lengths say.
__device__ __forceinline__ AttnReq sched_req(const AttnSched &s, int r) {
  AttnReq q;
  const int64_t a = s.cu[r], b = s.cu[r + 1];
  const int64_t lo = a < 0 ? 0 : (a > s.T ? s.T : a);
  const int64_t hi = b < lo ? lo : (b > s.T ? s.T : b);
  q.q0 = static_cast<int>(lo);
  q.n = static_cast<int>(hi - lo);
  // tokens of the request, those behind the buffers' end included: the rows
  // that there are keep their keys.  2^30 rows: more than any table holds, for
  // each of its tokens
  const int64_t tokens = (b < lo ? lo : b) - lo;
  int64_t L = s.kvl ? s.kvl[r] : tokens;
  if (L < 0) L = 0;
  if (L > (1 << 30)) L = 1 << 30;
  q.ctx = static_cast<int>(L - tokens);
  return q;
}

__device__ __forceinline__ int sched_blocks(const AttnSched &s, const AttnReq &q) {
  return (q.n + s.U - 1) / s.U;
}

// Keys that the last token of block i sees (0 or less: none), that token t
// sees, and whether the table is too short for the former.
__device__ __forceinline__ int sched_end(const AttnSched &s, const AttnReq &q, int i) {
  return min(q.ctx + min(q.n, (i + 1) * s.U), s.cap);
}

__device__ __forceinline__ int sched_seen(const AttnSched &s, const AttnReq &q, int t) {
  return min(q.ctx + t + 1, s.cap);
}

__device__ __forceinline__ bool sched_short(const AttnSched &s, const AttnReq &q, int i) {
  return q.ctx + min(q.n, (i + 1) * s.U) > s.cap;
}

__device__ __forceinline__ int sched_tiles(const AttnSched &s, const AttnReq &q, int i) {
  const int e = sched_end(s, q, i), kt = 1 << s.kt_shift;
  return e > kt ? (e + kt - 1) >> s.kt_shift : 1;
}

// Cost of one unit of block i, and of one head's units in the blocks before
// it (all of them full).  Rows that see no key (L < n) cost as if L = n; keys
// beyond the table count, so that a unit's tiles always fit its cost.
__device__ __forceinline__ int64_t sched_unit(const AttnSched &s, const AttnReq &q, int i) {
  return static_cast<int64_t>(max(q.ctx, 0)) + min(q.n, (i + 1) * s.U) + s.fixed;
}

__device__ __forceinline__ int64_t sched_before(const AttnSched &s, const AttnReq &q, int i) {
  const int64_t n = i;
  return n * (max(q.ctx, 0) + s.fixed) + n * (n + 1) / 2 * s.U;
}

__device__ __forceinline__ int64_t sched_cost(const AttnSched &s, const AttnReq &q) {
  const int m = sched_blocks(s, q);
  return m == 0 ? 0 : (sched_before(s, q, m - 1) + sched_unit(s, q, m - 1)) * s.nvh;
}

// One worker's run [first, last) of the call's cost, and the unit that holds
// its start: request r, token block i, head h, beginning at cost `unit`.
struct AttnRun {
  int64_t first, last, unit, step;
  int r, i, h;
};

// floor(a / b) for a >= 0, b > 0 and a quotient that fits an int (a worker, a
// head): the quotient in fp32, put right; far shorter than a 64-bit division.
__device__ __forceinline__ int small_quotient(int64_t a, int64_t b) {
  int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
#pragma unroll 1
  while (static_cast<int64_t>(q) * b > a) --q;
#pragma unroll 1
  while ((static_cast<int64_t>(q) + 1) * b <= a) ++q;
  return q;
}

// The run of worker w, by all NT threads of a block.  scratch: 8 (NT / 32 + 4)
// bytes of shared memory.  A worker without work gets first >= last.  (Written
// for few instructions: at the start of a call all of them are fetched from
// far, which costs more than executing them.)
template <int NT>
__device__ __forceinline__ AttnRun sched_run(const AttnSched &s, int w, int64_t *scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (s.R + NT - 1) / NT;
  const int r0 = min(s.R, tid * per), r1 = min(s.R, r0 + per);
  int64_t mine = 0;
#pragma unroll 1
  for (int r = r0; r < r1; ++r) mine += sched_cost(s, sched_req(s, r));
  int64_t inc = mine;  // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  int64_t lo = inc - mine, W = 0;  // lo: cost before this thread's requests
#pragma unroll
  for (int k = 0; k < NT / 32; ++k) {
    if (k == warp) lo += W;
    W += scratch[k];
  }
  AttnRun run;
  const int64_t even = static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(W), s.per_worker)) + 1;
  run.step = even > s.min_run ? even : s.min_run;
  run.first = w * run.step;
  run.last = min64(run.first + run.step, W);
  int64_t *found = scratch + NT / 32;
  if (run.first < run.last && run.first >= lo && run.first < lo + mine) {
    int r = r0;
    AttnReq q;
#pragma unroll 1
    for (;; ++r) {
      q = sched_req(s, r);
      const int64_t c = sched_cost(s, q);
      if (run.first < lo + c || r + 1 >= r1) break;
      lo += c;
    }
    // the block whose units hold the start: all heads of the blocks before
    // block a cost `before`
    int a = 0, b = sched_blocks(s, q);
    int64_t before = 0;
#pragma unroll 1
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      const int64_t c = sched_before(s, q, mid) * s.nvh;
      if (lo + c <= run.first) {
        a = mid;
        before = c;
      } else {
        b = mid;
      }
    }
    lo += before;
    const int64_t cost = sched_unit(s, q, a);
    const int h = small_quotient(run.first - lo, cost);
    found[0] = r;
    found[1] = a;
    found[2] = h;
    found[3] = lo + h * cost;
  }
  __syncthreads();
  const bool work = run.first < run.last;  // else nothing was found
  run.r = work ? static_cast<int>(found[0]) : 0;
  run.i = work ? static_cast<int>(found[1]) : 0;
  run.h = work ? static_cast<int>(found[2]) : 0;
  run.unit = work ? found[3] : run.last;
  return run;
}

// The tiles [tile, stop) of a unit of ntile tiles at cost x whose first keys
// the run holds; a cut inside the fixed cost leaves all tiles to the later run.
__device__ __forceinline__ int sched_cut(const AttnSched &s, int64_t at, int ntile) {
  if (at <= 0) return 0;
  const int64_t t = (at + (1 << s.kt_shift) - 1) >> s.kt_shift;
  return t < ntile ? static_cast<int>(t) : ntile;
}

__device__ __forceinline__ void sched_part(const AttnSched &s, const AttnRun &run, int64_t x,
                                           int ntile, int &tile, int &stop) {
  if (s.whole) {
    tile = x >= run.first ? 0 : ntile;
    stop = ntile;
    return;
  }
  tile = sched_cut(s, run.first - x - s.fixed, ntile);
  stop = sched_cut(s, run.last - x - s.fixed, ntile);
}

// The worker that has a unit's last tile.
__device__ __forceinline__ int sched_last(const AttnSched &s, const AttnRun &run, int64_t x,
                                          int ntile) {
  return small_quotient(x + s.fixed + (static_cast<int64_t>(ntile - 1) << s.kt_shift), run.step);
}

// What a worker leaves for the merge: the unit that is still open when its
// run ends and that it started (rows = 0: none).
struct AttnOpen {
  int q0, rows_tok;  // first token row of the unit, tokens
  int vh;            // (virtual) head
  int last;          // the worker whose run ends it
};

}  // namespace qmm
