// attn_sched.cuh -- how the batched attention kernels share their work out.
//
// A call has R requests; request r has n new tokens (query rows) and L cache
// rows, and token t of it sees the keys 0 .. L - n + t.  A unit of work is
// (request, block of U consecutive tokens, key/value head); its cost is the
// number of KT-key tiles its last token reaches (at least one, so that a
// token that sees no key still gets its row of zeros).  The units are laid
// end to end in the order (request, token block, head) and the W tiles of
// the whole call are cut into G equal runs, one per worker: every worker
// gets the same work whatever the lengths are, and a long context is split
// over as many workers as its share of the work asks for.  A unit that a cut
// divides leaves one partial result per worker, merged afterwards in worker
// order, so results are reproducible bit for bit.
//
// Everything here is computed on the device from the lengths (a call can be
// captured in a graph and replayed with other lengths in the same buffers).
#pragma once

#include <cstdint>

namespace qmm {

struct AttnSched {
  const int32_t *cu;   // [R + 1] prefix sum of the new tokens
  const int32_t *kvl;  // [R] cache rows, or nullptr: the new tokens themselves
  int R;
  int nvh;             // key/value heads (times the splits of a large query group)
  int U;               // tokens per unit
  int KT;              // keys per tile
  int min_tiles;       // a worker gets at least this many tiles
  int64_t T;           // query rows in the buffers
  int64_t cap;         // largest cache length the block table can hold
};

struct AttnReq {
  int q0, n;  // first query row, new tokens
  int L;      // cache rows
};

// Request r, held inside the buffers whatever the lengths say.
__device__ __forceinline__ AttnReq sched_req(const AttnSched &s, int r) {
  AttnReq q;
  const int64_t a = s.cu[r], b = s.cu[r + 1];
  const int64_t lo = a < 0 ? 0 : (a > s.T ? s.T : a);
  const int64_t hi = b < lo ? lo : (b > s.T ? s.T : b);
  q.q0 = static_cast<int>(lo);
  q.n = static_cast<int>(hi - lo);
  int64_t L = s.kvl ? s.kvl[r] : q.n;
  if (L < 0) L = 0;
  if (L > s.cap) L = s.cap;
  q.L = static_cast<int>(L);
  return q;
}

// sum_{i < n} floor((a i + b) / m) for n, a, b >= 0, m > 0: the whole parts of
// a / m and b / m are taken out, and what is left counts the lattice points
// under a line, which is the same sum with the axes exchanged (the steps of
// Euclid's algorithm on a and m).
__device__ inline int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t total = 0;
  while (n > 0) {
    total += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t y = a * n + b;
    n = y / m;
    b = y % m;
    const int64_t t = m;
    m = a;
    a = t;
    if (m == 0) break;
  }
  return total;
}

__device__ __forceinline__ int sched_blocks(const AttnSched &s, const AttnReq &q) {
  return (q.n + s.U - 1) / s.U;
}

// Keys that the last token of block i sees (0 or less: none).
__device__ __forceinline__ int sched_end(const AttnSched &s, const AttnReq &q, int i) {
  const int last = min(q.n, (i + 1) * s.U);
  return q.L - q.n + last;
}

__device__ __forceinline__ int sched_tiles(const AttnSched &s, const AttnReq &q, int i) {
  const int e = sched_end(s, q, i);
  return e > s.KT ? (e + s.KT - 1) / s.KT : 1;
}

// Tiles of one head in the token blocks before block i.
__device__ inline int64_t sched_before(const AttnSched &s, const AttnReq &q, int i) {
  // block j < i is full: its last token sees c + (j + 1) U keys, c = L - n
  const int64_t c = static_cast<int64_t>(q.L) - q.n;
  int64_t j0 = 0;  // blocks whose last token sees no key: one tile each
  if (c < 0) {
    j0 = -c / s.U;
    if (j0 > i) j0 = i;
  }
  return j0 + floor_sum(i - j0, s.KT, s.U, c + (j0 + 1) * s.U + s.KT - 1);
}

__device__ __forceinline__ int64_t sched_cost(const AttnSched &s, const AttnReq &q) {
  const int m = sched_blocks(s, q);
  if (m == 0) return 0;
  const int64_t before = m > 1 ? sched_before(s, q, m - 1) : 0;
  return (before + sched_tiles(s, q, m - 1)) * s.nvh;
}

// One worker's run: where it starts and how many tiles it has.  W and G
// describe the cut (worker w starts at tile floor(w W / G)).
struct AttnRun {
  int64_t W, first, last;  // tiles of the call; this worker's [first, last)
  int G;
  int r, i, h, tile;       // request, token block, head, tile where it starts
};

// The run of worker w of at most `workers`, by all NT threads of a block.
// scratch: 8 (NT / 32 + 8) bytes of shared memory.  A worker without work
// gets first == last.
template <int NT>
__device__ AttnRun sched_run(const AttnSched &s, int w, int workers, int64_t *scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (s.R + NT - 1) / NT;
  const int r0 = min(s.R, tid * per), r1 = min(s.R, r0 + per);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += sched_cost(s, sched_req(s, r));
  int64_t inc = mine;  // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  int64_t base = 0, W = 0;
#pragma unroll
  for (int k = 0; k < NT / 32; ++k) {
    const int64_t v = scratch[k];
    if (k < warp) base += v;
    W += v;
  }
  AttnRun run;
  run.W = W;
  const int64_t g = W / s.min_tiles;
  run.G = g < 1 ? 1 : (g < workers ? static_cast<int>(g) : workers);
  run.first = w < run.G ? w * W / run.G : W;
  run.last = w < run.G ? (w + 1) * W / run.G : W;
  int *found = reinterpret_cast<int *>(scratch + NT / 32);
  const int64_t lo = base + inc - mine;
  if (run.first < run.last && run.first >= lo && run.first < lo + mine) {
    int64_t o = run.first - lo;
    int r = r0;
    AttnReq q = sched_req(s, r);
    for (int64_t c = sched_cost(s, q); o >= c; c = sched_cost(s, q)) {
      o -= c;
      q = sched_req(s, ++r);
    }
    int a = 0, b = sched_blocks(s, q);  // the block holding tile o of the request
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (sched_before(s, q, mid) * s.nvh <= o) a = mid;
      else b = mid;
    }
    o -= sched_before(s, q, a) * s.nvh;
    const int t = sched_tiles(s, q, a);
    found[0] = r;
    found[1] = a;
    found[2] = static_cast<int>(o / t);
    found[3] = static_cast<int>(o % t);
  }
  __syncthreads();
  run.r = found[0];
  run.i = found[1];
  run.h = found[2];
  run.tile = found[3];
  return run;
}

// What a worker leaves for the merge: the unit that is still open when its
// run ends and that it started (rows = 0: none).
struct AttnOpen {
  int q0, rows_tok;  // first token row of the unit, tokens
  int vh;            // (virtual) head
  int last;          // the worker whose run ends it
};

// Worker that processes tile x of a call cut into G runs of W tiles.
__device__ __forceinline__ int sched_owner(int64_t x, int64_t W, int G) {
  int w = static_cast<int>(x * G / W);
  while (w + 1 < G && (w + 1) * W / G <= x) ++w;
  while (w > 0 && w * W / G > x) --w;
  return w;
}

}  // namespace qmm
