// attn_rows.cu -- batched attention for few query rows per key/value head
// (decoding) in fp32 arithmetic: fp32 caches, and head sizes the tensor cores
// do not take.
//
// The work is bound by reading the cache once, so the kernel keeps many wide
// loads in flight and spends few instructions on a key.  A team of LK lanes
// takes B consecutive keys at a time (one block's; the teams of a CTA cover a
// KT key tile), lane l holding columns 4 l + 4 LK c of the keys, values,
// queries and results in registers.  The RR x B partial dot products are
// reduced over the lanes by halving (every step sends the half of the values
// that the other lane keeps: RR B - 1 exchanges instead of log2(LK) RR B),
// which leaves the scores of one or a few (row, key) per lane; each lane keeps
// the running maximum and sum of its row, and the weights go back to all lanes
// by shuffles.  The warps run independently and meet at the end of a unit.
//
// One or two rows: a team is as many lanes as the row has pieces of four
// columns, which keeps the registers free for loads in flight.  Four rows and
// more: half as many lanes with two pieces each, which halves the exchanges of
// a key (16 heads over 4 of 64 columns, 128 requests: 5.8 TB/s instead of 4.2;
// 64 over 8 of 128: 5.5 instead of 4.8; 12 over 4 of 96: 5.2 instead of 4.8).
//
// Measured: 12 single tokens of 32 heads of 128 columns over 32 key/value
// heads' fp32 caches (623 MB) 98 us, 6.4 TB/s, 94% of a copy.  Eight rows a key are bound by
// instructions and their latency at two warps a scheduler (they issue 63% of the
// cycles; 47% of the instructions are the products): 82% of a copy.
//
// A request's rows beyond a unit's are further units that read its keys again,
// which over long caches still is cheaper up to four units (24 requests of 2048
// keys, 32 rows each: 282 us against attn_tile_kernel's 387; 256 columns, 16
// rows: 132 against attn_simt_kernel's 163); packed prompts, whose keys are few,
// go there at once (16 prompts of 32 tokens, 32 heads: 37 us against 74), unless
// all of their units are at most three to an SM: attn_tile_kernel's units of 128
// rows would leave SMs idle (a prompt of 37 tokens, 6 heads 8.2 us against 19; of
// 100 tokens, 32 heads, 400 units 22 against 32; 4 of 32 tokens, 512 units 22
// against 16).
#include <cstdint>

#include "attn_batch.h"
#include "attn_internal.h"
#include "attn_sched.cuh"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// NC: 4 LK-column groups of the head size; RR: query rows of a unit; LK: lanes
// that share a key (a "team").
template <int NC, int RR, int LK>
struct Rows {
  static constexpr int B = NC == 1 ? 8 : NC == 2 ? 4 : 2;  // keys of a team at a time
  static constexpr int teams = kThreads / LK;
  static constexpr int KT = teams * B;
  static constexpr int N = RR * B;                         // scores of a team at a time
  static constexpr int per_lane = N > LK ? N / LK : 1;     // ... of a lane
  static constexpr int dup = N < LK ? LK / N : 1;          // lanes with the same score
  // CTAs per SM: one where the registers of two would spill
  static constexpr int per_sm = NC * RR <= 4 ? 2 : 1;
  // With one CTA's eight warps an SM, the registers of a lane hold too few
  // loads: these copy their keys and values to shared memory, two tiles ahead.
  // Every lane copies what it reads itself, so no barrier is needed.
  static constexpr int stages = per_sm == 1 ? 3 : 0;
  static constexpr int out_bytes = teams * RR * NC * 4 * LK * 4;  // results of the teams
  static constexpr int pieces = B * NC * kThreads;  // four elements each: a stage's keys, or values
};

// Four elements, global -> shared, asynchronously.
template <bool BF16>
__device__ __forceinline__ void copy_x4(uint32_t dst, const void *base, int64_t i) {
  if constexpr (BF16)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst),
                 "l"(static_cast<const uint16_t *>(base) + i)
                 : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
                 "l"(static_cast<const float *>(base) + i)
                 : "memory");
}
template <bool BF16>
__device__ __forceinline__ float4 shared_x4(const uint8_t *p) {
  if constexpr (BF16) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
  } else {
    return *reinterpret_cast<const float4 *>(p);
  }
}

// v[i] summed over the team's lanes: lane l is left with values
// per_lane (l / dup) + j.
template <int N, int LK>
__device__ __forceinline__ void reduce_scatter(float (&v)[N], int lane) {
  int n = N;
#pragma unroll
  for (int o = LK / 2; o >= 1; o >>= 1) {
    if (n > 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i >= n / 2) break;
        const float send = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
        v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
      }
      n /= 2;
    } else {
      v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
    }
  }
}

template <bool BF16, int NC, int RR, int LK>
__global__ void __launch_bounds__(kThreads, Rows<NC, RR, LK>::per_sm)
    attn_rows_kernel(AttnBatch a, AttnSched sc, int gsub, int nsub, AttnParts parts,
                     uint32_t *status) {
  using C = Rows<NC, RR, LK>;
  constexpr int B = C::B, KT = C::KT, N = C::N, PL = C::per_lane, CW = NC * 4 * LK;
  __shared__ int64_t scratch[kWarps + 4];
  __shared__ float wm[C::teams][RR], wl[C::teams][RR];
  extern __shared__ __align__(16) float wo[];  // [team][row][CW], and the stages, then the stages
  constexpr int W = BF16 ? 8 : 16, HALF = C::pieces * W;
  uint8_t *const stages = reinterpret_cast<uint8_t *>(wo) + threadIdx.x * W;
  const int tid = threadIdx.x, team = tid / LK, lane = tid % LK;
  const int base_lane = (tid & 31) - lane;  // the team's first lane in its warp
  const int hd = a.head_dim, grp = a.n_head / a.n_kv;
  pdl_enter();
  const AttnRun run = sched_run<kThreads>(sc, blockIdx.x, scratch);
  if (tid == 0) parts.open[blockIdx.x].rows_tok = 0;
  const float sl2 = a.scale * 1.4426950408889634f;
  // this lane's scores: row srow, keys skey + j
  const int s0 = PL * (lane / C::dup), srow = s0 / B, skey = s0 % B;
  int64_t x = run.unit;
  int r = run.r, i = run.i, vh = run.h;
  AttnReq q;
  for (int64_t next = 0; x < run.last; x = next, vh = vh + 1 == sc.nvh ? 0 : vh + 1, i += vh == 0) {
    q = sched_req(sc, r);
    bool done = false;
    while (i >= sched_blocks(sc, q)) {
      if ((done = ++r >= sc.R)) break;  // lengths that changed during the call
      i = 0;
      q = sched_req(sc, r);
    }
    if (done) break;
    const int ntile = sched_tiles(sc, q, i);
    next = x + sched_unit(sc, q, i);
    int tile, stop;
    sched_part(sc, run, x, ntile, tile, stop);
    if (tile >= stop) continue;
    const int h = vh / nsub, sub = vh - h * nsub;
    const int g = min(gsub, grp - sub * gsub);
    const int t0 = i * sc.U, nt = min(sc.U, q.n - t0);
    const int rows = nt * g, head0 = h * grp + sub * gsub;
    const int end = sched_end(sc, q, i), all = sched_seen(sc, q, t0);
    const int vis = min(all + (srow < rows ? srow / g : 0), end);  // keys this lane's row sees
    if (tid == 0 && sched_short(sc, q, i)) atomicOr(status, kDevBadBlock);
    float4 qv[RR][NC], o[RR][NC];
#pragma unroll
    for (int p = 0; p < RR; ++p) {
      const int t = p / g, hq = p - t * g;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int d = 4 * lane + 4 * LK * c;
        const float4 v = p < rows && d < hd
                             ? load_x4<BF16>(a.q, static_cast<int64_t>(q.q0 + t0 + t) * a.q_stride +
                                                      static_cast<int64_t>(head0 + hq) * hd + d)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
        qv[p][c] = make_float4(v.x * sl2, v.y * sl2, v.z * sl2, v.w * sl2);  // scores in log2 units
        o[p][c] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    float m = -INFINITY, l = 0.0f;  // of this lane's row; l over this lane's keys
    const int32_t *table = a.block_table ? a.block_table + r * a.table_stride : nullptr;
    // block of the first key of this team's part of a tile (0 behind the end)
    auto block_of = [&](int kt) {
      const int k = kt * KT + team * B;
      return table && kt < stop && k < end ? table[k / a.block_size] : 0;
    };
    // keys of this team's part of a tile that lie in the cache, and their place
    int64_t kp = 0, vp = 0, ks = hd, vs = hd;  // first row, distance of rows
    auto locate = [&](int kt, int id) {
      const int k0 = kt * KT + team * B;
      const int nk = kt < stop ? max(0, min(B, end - k0)) : 0;
      if (table) {
        if (nk > 0 && (id < 0 || id >= a.num_blocks)) {
          if (lane == 0) atomicOr(status, kDevBadBlock);
          return 0;
        }
        kp = vp = id * a.block_stride +
                  static_cast<int64_t>(h * a.block_size + k0 % a.block_size) * hd;
      } else {
        ks = a.k_stride;
        vs = a.v_stride;
        kp = (static_cast<int64_t>(q.q0) + k0) * ks + static_cast<int64_t>(h) * hd;
        vp = (static_cast<int64_t>(q.q0) + k0) * vs + static_cast<int64_t>(h) * hd;
      }
      return nk;
    };
    int slot3 = 0;  // stage of the current tile
    auto fetch = [&](int kt, int id, int stage) {
      const int nk = locate(kt, id);
      uint8_t *const at = stages + stage * 2 * HALF;
#pragma unroll
      for (int k = 0; k < B; ++k)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int d = 4 * lane + 4 * LK * c;
          uint8_t *const kd = at + (k * NC + c) * kThreads * W, *const vd = kd + HALF;
          if (k < nk && d < hd) {
            copy_x4<BF16>(smem_addr(kd), a.k, kp + k * ks + d);
            copy_x4<BF16>(smem_addr(vd), a.v, vp + k * vs + d);
          } else if constexpr (BF16) {
            *reinterpret_cast<uint2 *>(kd) = *reinterpret_cast<uint2 *>(vd) = make_uint2(0, 0);
          } else {
            *reinterpret_cast<float4 *>(kd) = *reinterpret_cast<float4 *>(vd) =
                make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      asm volatile("cp.async.commit_group;" ::: "memory");
      return nk;
    };
    int id = block_of(tile), nk0 = 0, nk1 = 0;
    if constexpr (C::stages > 0) {
      const int id1 = block_of(tile + 1), id2 = block_of(tile + 2);
      nk0 = fetch(tile, id, 0);
      nk1 = fetch(tile + 1, id1, 1);
      id = id2;
    }
    for (int kt = tile; kt < stop; ++kt) {
      const int k0 = kt * KT + team * B;
      int nk;  // the team's keys; the warp's teams stay together
      const uint8_t *at = nullptr;
      if constexpr (C::stages > 0) {
        const int two = id, ahead = slot3 == 0 ? 2 : slot3 - 1;
        id = block_of(kt + 3);
        const int nk2 = fetch(kt + 2, two, ahead);
        asm volatile("cp.async.wait_group 2;" ::: "memory");
        at = stages + slot3 * 2 * HALF;
        slot3 = slot3 == 2 ? 0 : slot3 + 1;
        nk = nk0;
        nk0 = nk1;
        nk1 = nk2;
      } else {
        const int mine = id;
        id = block_of(kt + 1);
        nk = locate(kt, mine);
      }
      if (LK == 32 ? nk == 0 : !__any_sync(0xFFFFFFFFu, nk > 0)) continue;
      float4 kv[B][NC], vv[B][NC];
      if constexpr (C::stages > 0) {
#pragma unroll
        for (int k = 0; k < B; ++k)
#pragma unroll
          for (int c = 0; c < NC; ++c)
            kv[k][c] = shared_x4<BF16>(at + (k * NC + c) * kThreads * W);
      } else {
#pragma unroll
        for (int k = 0; k < B; ++k)
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int d = 4 * lane + 4 * LK * c;
            kv[k][c] = k < nk && d < hd ? load_x4<BF16>(a.k, kp + k * ks + d)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
        for (int k = 0; k < B; ++k)
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int d = 4 * lane + 4 * LK * c;
            vv[k][c] = k < nk && d < hd ? load_x4<BF16>(a.v, vp + k * vs + d)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
          }
      }
      float s[N];
#pragma unroll
      for (int p = 0; p < RR; ++p)
#pragma unroll
        for (int k = 0; k < B; ++k) {
          float acc = 0.0f;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            acc = fmaf(qv[p][c].x, kv[k][c].x, acc);
            acc = fmaf(qv[p][c].y, kv[k][c].y, acc);
            acc = fmaf(qv[p][c].z, kv[k][c].z, acc);
            acc = fmaf(qv[p][c].w, kv[k][c].w, acc);
          }
          s[p * B + k] = acc;
        }
      reduce_scatter<N, LK>(s, lane);
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < PL; ++j) {
        if (k0 + skey + j >= vis || skey + j >= nk) s[j] = -INFINITY;
        top = fmaxf(top, s[j]);
      }
#pragma unroll
      for (int w = C::dup; w < C::dup * (B / PL); w <<= 1)
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, w));
      const bool grow = top > m;
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float f = grow ? ex2(m - top) : 1.0f;  // m = -inf: 0
        if (grow) m = top;
        l *= f;
#pragma unroll
        for (int p = 0; p < RR; ++p) {
          const float fp = __shfl_sync(0xFFFFFFFFu, f, base_lane + p * B / PL * C::dup);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            o[p][c].x *= fp;
            o[p][c].y *= fp;
            o[p][c].z *= fp;
            o[p][c].w *= fp;
          }
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      // some row of some team misses some key: not even 0 * NaN may enter
      const bool guard = LK == 32 ? k0 + B > all : __any_sync(0xFFFFFFFFu, k0 + B > all || nk < B);
#pragma unroll
      for (int j = 0; j < PL; ++j) {
        s[j] = s[j] == -INFINITY ? unseen_weight() : ex2(s[j] - ref);
        l += s[j];
      }
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if constexpr (C::stages > 0) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
            vv[k][c] = shared_x4<BF16>(at + HALF + (k * NC + c) * kThreads * W);
        }
#pragma unroll
        for (int p = 0; p < RR; ++p) {
          const int v = p * B + k;
          const float w = __shfl_sync(0xFFFFFFFFu, s[v % PL], base_lane + v / PL * C::dup);
          if (guard && is_unseen(w)) continue;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            // pairs: 64 heads over 8 149 -> 145 us (the scores gain nothing from them)
            const f32x2 w2 = pack2(w, w);
            unpack2(fma2(w2, pack2(vv[k][c].x, vv[k][c].y), pack2(o[p][c].x, o[p][c].y)), o[p][c].x,
                    o[p][c].y);
            unpack2(fma2(w2, pack2(vv[k][c].z, vv[k][c].w), pack2(o[p][c].z, o[p][c].w)), o[p][c].z,
                    o[p][c].w);
          }
        }
      }
    }
    // the row's sum over its lanes, then the teams' parts together
#pragma unroll
    for (int w = C::dup; w < C::dup * (B / PL); w <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, w);
    if (C::stages > 0) __syncthreads();  // the stages' memory takes the results
    if (skey == 0 && lane % C::dup == 0) {
      wm[team][srow] = m;
      wl[team][srow] = l;
    }
#pragma unroll
    for (int p = 0; p < RR; ++p)
#pragma unroll
      for (int c = 0; c < NC; ++c)
        *reinterpret_cast<float4 *>(wo + (team * RR + p) * CW + 4 * LK * c + 4 * lane) = o[p][c];
    __syncthreads();
    const bool whole = tile == 0 && stop == ntile;
    const int slot = 2 * blockIdx.x + (tile == 0 ? 1 : 0);
    for (int e = tid; e < RR * CW / 4; e += kThreads) {
      const int p = e / (CW / 4), d = 4 * (e - p * (CW / 4));
      if (p >= rows || d >= hd) continue;
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int w = 0; w < C::teams; ++w) M = fmaxf(M, wm[w][p]);
      const float ref = M == -INFINITY ? 0.0f : M;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::teams; ++w) {
        // (zeros of a team that saw no key count nothing; a NaN makes the row NaN,
        // however small its team's factor is)
        const float f = ex2(wm[w][p] - ref);
        const float4 v = *reinterpret_cast<const float4 *>(wo + (w * RR + p) * CW + d);
        L = fmaf(f, wl[w][p], L);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      if (whole) {
        const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;
        const int t = p / g, hq = p - t * g;
        store_y4(a.y, (static_cast<int64_t>(q.q0 + t0 + t) * a.n_head + head0 + hq) * hd + d,
                 make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv), a.y_bf16);
      } else {
        const int64_t base = static_cast<int64_t>(slot) * parts.rows + p;
        if (d == 0) parts.ml[base] = make_float2(M, L);
        *reinterpret_cast<float4 *>(parts.o + base * hd + d) = acc;
      }
    }
    __syncthreads();
    if (tid == 0 && tile == 0 && !whole)
      parts.open[blockIdx.x] =
          AttnOpen{q.q0 + t0, nt, vh, sched_last(sc, run, x, ntile)};
  }
  zero_loose_rows(a, sc, blockIdx.x, gridDim.x, kThreads);
}

template <bool BF16, int NC, int RR, int LK = 32>
cudaError_t run_rows(const AttnBatch &a, const AttnPlan &p, const AttnSched &sc,
                     const AttnParts &parts, cudaStream_t s) {
  using C = Rows<NC, RR, LK>;
  auto kern = attn_rows_kernel<BF16, NC, RR, LK>;
  constexpr int staged = C::stages * 2 * C::pieces * (BF16 ? 8 : 16);
  constexpr int smem = staged > C::out_bytes ? staged : C::out_bytes;
  const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  uint32_t *status = device_status();
  if (!status) return cudaErrorInvalidDevice;
  return launch_pdl(kern, dim3(p.workers), dim3(kThreads), smem, s, a, sc, p.gsub, p.nsub, parts,
                    status);
}

template <bool BF16>
cudaError_t pick_rows(const AttnBatch &a, const AttnPlan &p, const AttnSched &sc,
                      const AttnParts &parts, cudaStream_t s) {
  if (a.head_dim <= 64) {
    if (p.rows == 1) return run_rows<BF16, 1, 1, 16>(a, p, sc, parts, s);
    if (p.rows == 2) return run_rows<BF16, 1, 2, 16>(a, p, sc, parts, s);
    if (p.rows == 4) return run_rows<BF16, 2, 4, 8>(a, p, sc, parts, s);
    return run_rows<BF16, 2, 8, 8>(a, p, sc, parts, s);
  }
  if (a.head_dim <= 128) {
    if (p.rows == 1) return run_rows<BF16, 1, 1>(a, p, sc, parts, s);
    if (p.rows == 2) return run_rows<BF16, 1, 2>(a, p, sc, parts, s);
    if (p.rows == 4) return run_rows<BF16, 2, 4, 16>(a, p, sc, parts, s);
    return run_rows<BF16, 2, 8, 16>(a, p, sc, parts, s);
  }
  if (a.head_dim <= 256) {
    if (p.rows <= 2) return run_rows<BF16, 2, 2>(a, p, sc, parts, s);
    return run_rows<BF16, 2, 4>(a, p, sc, parts, s);
  }
  return run_rows<BF16, 4, 2>(a, p, sc, parts, s);
}

}  // namespace

// Calls with few query rows per request and key/value head: at most 8, 4 or 2
// of them (what a thread's registers hold of queries and results at 128, 256
// and 512 columns).
bool attn_rows_plan(bool paged, int64_t T, int n_head, int n_kv, int head_dim, int R, AttnPlan *p) {
  const int most = head_dim <= 128 ? 8 : head_dim <= 256 ? 4 : 2;  // rows of a unit
  const int take = paged ? 4 * most : most;                        // rows of a request
  const int grp = n_head / n_kv;
  const int64_t total = T * n_head;
  const bool few = grp <= take && T * grp <= static_cast<int64_t>(take) * R;
  if (R < 1 || !(few || (!paged && total <= static_cast<int64_t>(3) * most * sm_count()))) return false;
  const int avg = static_cast<int>((T * grp + R - 1) / R);
  int rows = head_dim <= 128 ? 1 : 2;
  while (rows < most && (rows < avg || rows < grp)) rows *= 2;
  p->rows = rows;
  p->gsub = grp < rows ? grp : rows;
  p->nsub = (grp + p->gsub - 1) / p->gsub;
  p->U = rows / p->gsub;
  p->KT = head_dim <= 64 ? 128 : head_dim <= 128 ? 64 : head_dim <= 256 ? 32 : 16;
  p->fixed = 2 * p->KT;
  p->min_run = 2 * p->KT;
  p->whole = kWholeKeys;
  // CTAs an SM: two, or one that stages its loads
  p->workers = sm_count() * (rows * (head_dim <= 256 ? 2 : 4) <= 4 ? 2 : 1);
  return true;
}

cudaError_t launch_attn_rows(const AttnBatch &a, const AttnPlan &p, const AttnSched &sc,
                             const AttnParts &parts, cudaStream_t s) {
  return a.bf16 ? pick_rows<true>(a, p, sc, parts, s) : pick_rows<false>(a, p, sc, parts, s);
}

}  // namespace qmm
