// attn_tc.cu -- batched causal attention for bf16 on the 5th-generation tensor
// cores (tcgen05): packed prompts, chunks and single tokens over a paged cache.
//
//   S = Q K^T (fp32 in tensor memory), P = 2^(scale log2e (S - m)) rounded to
//   bf16, O += P V (fp32 in tensor memory), l += row sums of the unrounded P
// over 128-key tiles, with m the row maximum so far.  O and l are rescaled
// only when the maximum has grown by more than 2^8: until then P is at most
// 2^8, far inside bf16 and fp32, and the ratio O / l does not depend on m.
//
// Query rows: a tile holds 128 / gsub tokens times the gsub query heads that
// share a key/value head, so that a key or value tile is read once for all of
// them.  CTA = 12 warps, one per SM, persistent over its run of the call's
// tiles (attn_sched.cuh).  A unit has two query tiles (A, B):
//   pair    more tokens than one tile holds: warpgroup 0 owns A, warpgroup 1
//           owns B, and every key tile serves both;
//   single  one tile (decoding, short prompts): the warpgroups take the key
//           tiles in turn and their results meet in shared memory.
// Either way the tensor core works for one warpgroup while the other one
// computes its exponentials.
//   warps 0-3, 4-7  warpgroups: thread = query row.  S from tensor memory,
//             maximum, exponentials, P back over S's columns; the epilogue.
//   warp 8    TMA producer of key and value tiles, one box per (block, 64
//             columns), each lane its own boxes
//   warp 9    MMA issuer (one lane): P V of a tile, then Q K^T of the same
//             warpgroup's next tile, which may overwrite S and P because the
//             tensor core runs its work in order
//   warp 10   value tiles that hold keys some row does not see: rows beyond
//             the unit's last key become zeros (0 * NaN would reach the sums),
//             non-finite values are taken out and the unit marked, so that
//             its epilogue adds them to the rows that do see them
//   warp 11   walks the run and hands its units to the other roles through a
//             ring in shared memory; TMA producer of the query tiles
// Every wait is bounded; on a timeout the CTA raises QMM_DEV_WAIT_TIMEOUT,
// all roles leave their loops, wait (bounded) for what they have in flight,
// and the tensor memory is freed.
//
// P is rounded to bf16 because the tensor core's operands are: at most 2^-8 of a
// weight, and l sums the weights before it.  Against 64 bits a bf16 result is
// then off by 0.0020 to 0.0023 of its norm, 0.0016 to 0.0017 with fp32 weights.
//
// Measured: two prompts of 16384 tokens together (32 heads of 128) 690 to 750 us back to
// back, 1.55 to 1.69 PFLOP/s of the causal half, 81 to 88% of a library product (calls
// among others 765 to 780 us).  A tile
// pair takes 2950 cycles, 2150 of them tensor work: what is left is the hand-
// over S -> P -> next S of the two warpgroups.  64 single tokens over caches
// of 1.4 GB 230 us, 6.1 TB/s, 90% of a copy.  Short units cost 4.4 us each
// besides their tiles (37-token prompt 8.1 us).
#include <cstdint>

#include "attn_batch.h"
#include "attn_internal.h"
#include "attn_sched.cuh"
#include "qmm_device.cuh"
#include "qmm_internal.h"
#include "tc_device.cuh"

namespace qmm {
namespace {

constexpr int kThreads = 384;
constexpr int kKT = 128;              // keys per tile
constexpr int kWarpKv = 8, kWarpMma = 9, kWarpClean = 10, kWarpQ = 11;
constexpr uint32_t kChunk = 128 * 128;  // bytes of 128 rows x 64 bf16 columns
constexpr int kUnits = 4;             // units in the ring between warp 11 and the others
constexpr float kRescale = 8.0f;      // log2 of the growth of the maximum that is let pass

// NCH: 64-column chunks of the head size.  STAGED: results go out through
// shared memory, which leaves room for four key and value tiles; without it
// there are five, which decoding needs (it is bound by the loads in flight:
// 64 requests 236 us with five tiles, 252 us with four) and can afford (few
// rows to store).
template <int NCH, bool STAGED>
struct Tc {
  static constexpr uint32_t tile = NCH * kChunk;            // one Q, K or V tile
  static constexpr int stages = NCH == 1 ? (STAGED ? 8 : 10) : (STAGED ? 4 : 5);  // K, V in turn
  static constexpr uint32_t q_off = 0, kv_off = 2 * tile;
  static constexpr uint32_t out_off = kv_off + stages * tile;  // 4 KB a warp: 32 rows of 128 bytes
  static constexpr uint32_t bar_off = out_off + (STAGED ? 8 * 4096 : 0);
  // q_full[2], q_free[2], x_full, drain, s_full[2], p_full[2][2], o_full[2],
  // u_full[kUnits], u_free[kUnits], then full, freed, clean [stages]
  static constexpr int nbar = 14 + 2 * kUnits + 3 * stages;
  static constexpr uint32_t unit_off = (bar_off + nbar * 8 + 15) & ~15u;
  static constexpr uint32_t misc_off = unit_off + kUnits * 64;  // tmem, abort, bad, -, marked[16]
  static constexpr uint32_t bytes = misc_off + 80 + 2 * 128 * 4 + 1024;
  static constexpr uint32_t o_col = 256, o_step = NCH * 64;  // tensor memory columns of O
};

struct TcAttn {
  AttnBatch a;
  AttnSched sc;
  AttnParts parts;
  int gsub, nsub, tpt;  // query heads and tokens of a tile
  int box_rows;         // rows per key box
  int block_shift;      // log2 of the cache's block size
  float sl2;            // scale log2(e)
  uint32_t *status;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// True in one lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ bool nonfinite_bf16(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

// Not zero when one of eight bf16 values is not finite (its exponent, all ones,
// carries into the sign's place).
__device__ __forceinline__ uint32_t nonfinite_bits(uint4 t) {
  return (((t.x & 0x7FFF7FFFu) + 0x00800080u) | ((t.y & 0x7FFF7FFFu) + 0x00800080u) |
          ((t.z & 0x7FFF7FFFu) + 0x00800080u) | ((t.w & 0x7FFF7FFFu) + 0x00800080u)) & 0x80008000u;
}
__device__ __forceinline__ uint4 drop_nonfinite(uint4 t) {
  uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (nonfinite_bf16(w[k])) w[k] &= 0xFFFF0000u;
    if (nonfinite_bf16(w[k] >> 16)) w[k] &= 0xFFFFu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Value tiles are [key][column] in shared memory, columns contiguous: for the
// product P V the operand's N axis (columns) is the contiguous one.  128B
// swizzle: 64-column chunks kChunk apart, groups of eight keys 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_values(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) |
         (static_cast<uint64_t>(kChunk >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

// bf16 x bf16 -> fp32, M = 128; values: B with N contiguous.
__device__ __forceinline__ uint32_t idesc_bf16(int n, bool values) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (values ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

// One unit of this worker's run, as the roles see it.
struct __align__(16) Unit {
  int valid, pair, q_row, nt;      // 0: no unit any more; first query row, tokens
  int h, head0, g, r;              // key/value head, first query head, heads, request
  int tile, stop, ntile, ntile_a;  // this worker's tiles [tile, stop); tiles that query tile A reaches
  int all, end, k_row, pad;        // keys the first / last token sees; first key row (packed keys)
};

// The key tiles first, first + step, ... < last of warpgroup w.
__device__ __forceinline__ void wg_tiles(const Unit &u, int w, int &first, int &last, int &step) {
  first = u.pair ? u.tile : u.tile + w;
  last = u.pair && w == 0 ? min(u.stop, u.ntile_a) : u.stop;
  step = u.pair ? 1 : 2;
}

// Adds the non-finite values that warp 10 took out of the unit's value tiles
// to a row that sees their keys (p v of a non-finite v is v, whatever p > 0).
template <bool PAGED>
__device__ __noinline__ void add_marked(const TcAttn &p, const Unit &u, int vis, void *out, bool bf16) {
  const int hd = p.a.head_dim;
  const int last = min(min(vis, u.end), u.stop * kKT);
#pragma unroll 1
  for (int j = max(u.tile * kKT, max(u.all, 0)); j < last; ++j) {
    const uint16_t *src = static_cast<const uint16_t *>(p.a.v);
    if (PAGED) {
      const int32_t id = p.a.block_table[u.r * p.a.table_stride + j / p.a.block_size];
      if (id < 0 || id >= p.a.num_blocks) continue;
      src += id * p.a.block_stride +
             static_cast<int64_t>(u.h * p.a.block_size + (j & (p.a.block_size - 1))) * hd;
    } else {
      src += (static_cast<int64_t>(u.k_row) + j) * p.a.v_stride + static_cast<int64_t>(u.h) * hd;
    }
#pragma unroll 1
    for (int d = 0; d < hd; ++d) {
      if (!nonfinite_bf16(src[d])) continue;
      const float v = __uint_as_float(static_cast<uint32_t>(src[d]) << 16);
      if (bf16) {
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(out) + d;
        *y = __float2bfloat16_rn(__bfloat162float(*y) + v);
      } else {
        static_cast<float *>(out)[d] += v;
      }
    }
  }
}

template <int NCH, bool PAGED, bool STAGED>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TcAttn p) {
  using C = Tc<NCH, STAGED>;
  constexpr int NS = C::stages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (base - raw);
  const uint32_t bars = base + C::bar_off;
  const uint32_t x_full = bars, drain = bars + 8;
  auto q_full = [&](int w) { return bars + 16 + 8 * w; };
  auto q_free = [&](int w) { return bars + 32 + 8 * w; };
  auto s_full = [&](int w) { return bars + 48 + 8 * w; };
  auto p_full = [&](int w, int half) { return bars + 64 + 16 * w + 8 * half; };
  auto o_full = [&](int w) { return bars + 96 + 8 * w; };
  auto u_full = [&](uint32_t n) { return bars + 112 + 8 * (n % kUnits); };
  auto u_free = [&](uint32_t n) { return bars + 112 + 8 * (kUnits + n % kUnits); };
  constexpr int kStageBars = 112 + 16 * kUnits;
  auto full = [&](int s) { return bars + kStageBars + 8 * s; };
  auto freed = [&](int s) { return bars + kStageBars + 8 * (NS + s); };
  auto clean = [&](int s) { return bars + kStageBars + 8 * (2 * NS + s); };
  Unit *units = reinterpret_cast<Unit *>(gbase + C::unit_off);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + C::misc_off);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + C::misc_off + 4);
  volatile int *bad_seen = reinterpret_cast<volatile int *>(gbase + C::misc_off + 8);
  volatile int *marked = reinterpret_cast<volatile int *>(gbase + C::misc_off + 16);  // [16]
  float *xm = reinterpret_cast<float *>(gbase + C::misc_off + 80), *xl = xm + 128;
  __shared__ int64_t scratch[kThreads / 32 + 4];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(x_full, 4);
    mbar_init(drain, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(q_full(w), 1);
      mbar_init(q_free(w), 4);
      mbar_init(s_full(w), 1);
      mbar_init(p_full(w, 0), 4);
      mbar_init(p_full(w, 1), 4);
      mbar_init(o_full(w), 1);
    }
    for (int k = 0; k < kUnits; ++k) {
      mbar_init(u_full(k), 1);
      mbar_init(u_free(k), 11);  // warps 0-7, 8, 9, 10
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(freed(s), 2);  // the tensor core's and warp 10's
      mbar_init(clean(s), 1);
    }
    mbar_fence_init();
    *abort_flag = 0;
    *bad_seen = 0;
    for (int k = 0; k < 16; ++k) marked[k] = 0;
  }
  if (warp == kWarpMma) tmem_alloc(smem_addr(tmem_slot), 512);
  if (threadIdx.x == kWarpKv * 32) {
    prefetch_map(&tm_q);
    prefetch_map(&tm_k);
    prefetch_map(&tm_v);
  }
  pdl_enter();
  const AttnRun run = sched_run<kThreads>(p.sc, blockIdx.x, scratch);
  if (threadIdx.x == 0) p.parts.open[blockIdx.x].rows_tok = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int hd = p.a.head_dim;
  const int nch = NCH == 1 ? 1 : (hd + 63) / 64;  // chunks that hold columns
  // the whole warp waits for a barrier
  auto wait_warp = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, wait_ok(bar, parity, p.status, abort_flag)) != 0;
  };

  // 384 threads launched with 168 registers: 2 x 208 + 88 = 3 x 168
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kWarpQ) {
      // ------------------------------------------- units, and query tiles
      const int grp = p.a.n_head / p.a.n_kv;
      int64_t x = run.unit;
      int r = run.r, i = run.i, vh = run.h;
      AttnReq q{};
      bool fresh = true;
      // the next unit of the run with tiles of it, into ring slot n
      auto publish = [&](uint32_t n) {
        Unit u{};
        while (x < run.last) {
          if (fresh) q = sched_req(p.sc, r);
          fresh = false;
          if (i >= sched_blocks(p.sc, q)) {
            if (++r >= p.sc.R) break;  // lengths that changed during the call
            i = 0;
            fresh = true;
            continue;
          }
          u.ntile = sched_tiles(p.sc, q, i);
          sched_part(p.sc, run, x, u.ntile, u.tile, u.stop);
          if (u.tile < u.stop) {
            const int t0 = i * p.sc.U;
            u.valid = 1;
            u.nt = min(p.sc.U, q.n - t0);
            u.pair = u.nt > p.tpt;
            u.q_row = q.q0 + t0;
            u.h = p.nsub == 1 ? vh : vh / p.nsub;
            const int sub = vh - u.h * p.nsub;
            u.head0 = u.h * grp + sub * p.gsub;
            u.g = min(p.gsub, grp - sub * p.gsub);
            u.r = r;
            const int end_a = sched_seen(p.sc, q, t0 + min(u.nt, p.tpt) - 1);
            u.ntile_a = end_a > kKT ? (end_a + kKT - 1) / kKT : 1;
            u.all = sched_seen(p.sc, q, t0);
            u.end = sched_end(p.sc, q, i);
            if (lane == 0 && sched_short(p.sc, q, i)) atomicOr(p.status, kDevBadBlock);
            u.k_row = q.q0;
            if (lane == 0 && u.tile == 0 && u.stop < u.ntile)
              p.parts.open[blockIdx.x] =
                  AttnOpen{u.q_row, u.nt, vh, sched_last(p.sc, run, x, u.ntile)};
          }
          x += sched_unit(p.sc, q, i);
          if (++vh == p.sc.nvh) {
            vh = 0;
            ++i;
          }
          if (u.valid) break;
        }
        if (lane == 0) {
          units[n % kUnits] = u;
          mbar_arrive(u_full(n));
        }
        __syncwarp();
        return u.valid != 0;
      };
      uint32_t pub = 0, n = 0, loads[2] = {0, 0};  // units handed out, served; tiles loaded
      bool more = true, ok = true;
      while (ok) {
        // the first unit's queries go out before the next units are looked up
        for (; ok && more && pub < (n == 0 ? 1 : n + 3); ++pub) {
          ok = wait_warp(u_free(pub), ((pub / kUnits) & 1u) ^ 1u);
          if (ok) more = publish(pub);
        }
        if (!ok || (!more && n + 1 == pub)) break;
        const Unit &u = units[n % kUnits];
        // a tile is loaded as soon as its warpgroup has no more use for the last one
        for (int w = 0; w < (u.pair ? 2 : 1); ++w) {
          if (!(ok = wait_warp(q_free(w), (n & 1u) ^ 1u))) break;
          if (lane == 0)
            mbar_arrive_expect_tx(q_full(w), static_cast<uint32_t>(nch * p.tpt * p.gsub * 128));
          __syncwarp();
          if (lane < nch)
            tma_load_3d(base + C::q_off + w * C::tile + lane * kChunk, &tm_q, lane * 64, u.head0,
                        u.q_row + w * p.tpt, q_full(w));
          loads[w] += 1;
        }
        ++n;
      }
      for (int w = 0; w < 2; ++w)
        if (loads[w] > 0) mbar_wait_bounded(q_full(w), (loads[w] - 1) & 1u, p.status);
    } else if (warp == kWarpKv) {
      // ------------------------------------------------ key and value tiles
      uint32_t n = 0;  // tiles loaded so far; stage n % NS
      int s = 0;
      uint32_t phase = 1;
      bool ok = true;
      // box `lane` of a tile: block lane / nch, columns of chunk lane % nch
      const int c = lane % nch, row0 = lane / nch * p.box_rows;
      for (uint32_t un = 0; ok; ++un) {
        if (!wait_warp(u_full(un), (un / kUnits) & 1u)) break;
        const Unit u = units[un % kUnits];
        if (!u.valid) break;
        const int32_t *table = PAGED ? p.a.block_table + u.r * p.a.table_stride : nullptr;
        auto block_of = [&](int kt) {
          const int k0 = kt * kKT + row0;
          if (!PAGED || row0 >= kKT || k0 >= u.end) return 0;
          return table[k0 >> p.block_shift];
        };
        int id = block_of(u.tile);
        for (int kt = u.tile; kt < u.stop && ok; ++kt) {
          const int k0 = kt * kKT;
          const int keys = max(0, min(kKT, u.end - k0));
          const int rows = PAGED ? (keys + p.box_rows - 1) & ~(p.box_rows - 1) : kKT;
          const int mine = id;
          if (kt + 1 < u.stop) id = block_of(kt + 1);
          const bool issue = row0 < rows;
          const bool bad = PAGED && issue && (mine < 0 || mine >= p.a.num_blocks);
          if (bad) {
            *bad_seen = 1;
            atomicOr(p.status, kDevBadBlock);
          }
          __syncwarp();
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            ok = wait_warp(freed(s), phase);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(full(s), static_cast<uint32_t>(rows * 128 * nch));
            __syncwarp();
            if (issue) {
              const uint32_t dst = base + C::kv_off + s * C::tile + c * kChunk + row0 * 128;
              const CUtensorMap *tm = kv ? &tm_v : &tm_k;
              if (PAGED)  // a bad index: block num_blocks, outside the map, reads as zeros
                tma_load_4d(dst, tm, c * 64, (k0 + row0) & (p.a.block_size - 1), u.h,
                            bad ? static_cast<int>(p.a.num_blocks) : mine, full(s));
              else
                tma_load_3d(dst, tm, c * 64, u.h, u.k_row + k0, full(s));
            }
            ++n;
            if (++s == NS) {
              s = 0;
              phase ^= 1u;
            }
          }
        }
        if (lane == 0) mbar_arrive(u_free(un));
      }
      // copies still landing (after an abort; otherwise all have been consumed)
      for (uint32_t k = n > NS ? n - NS : 0; k < n; ++k)
        mbar_wait_bounded(full(k % NS), (k / NS) & 1u, p.status);
    } else if (warp == kWarpClean) {
      // ------------------------- value tiles with keys that some row misses
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (uint32_t un = 0; ok; ++un) {
        if (!wait_warp(u_full(un), (un / kUnits) & 1u)) break;
        const Unit &ur = units[un % kUnits];
        if (!ur.valid) break;
        const int tile = ur.tile, stop = ur.stop, all = ur.all, end = ur.end;
        for (int kt = tile; kt < stop && ok; ++kt) {
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            ok = wait_warp(full(s), phase);
            if (!ok) break;
            const int k0 = kt * kKT;
            if (kv && k0 + kKT > all) {
              // Keys from `lo` on are missed by some row, from `hi` on by all of
              // them (their rows may hold anything).  Eight lanes read a row of
              // a chunk, eight reads in flight.
              const int lo = max(0, all - k0), hi = end - k0;
              uint8_t *v = gbase + C::kv_off + s * C::tile + (lane & 7) * 16;
              bool found = false;
#pragma unroll 1
              for (int c = 0; c < nch; ++c, v += kChunk) {
#pragma unroll 1
                for (int r0 = (lo & ~3) + (lane >> 3); r0 < kKT; r0 += 32) {
                  uint32_t hit = 0;
#pragma unroll
                  for (int k = 0; k < 8; ++k) {
                    const int r = min(r0 + 4 * k, kKT - 1);
                    hit |= nonfinite_bits(*reinterpret_cast<const uint4 *>(v + r * 128));
                  }
                  if (hit) {
#pragma unroll 1
                    for (int r = r0; r < min(r0 + 32, kKT); r += 4) {
                      if (r < lo) continue;
                      uint4 *t = reinterpret_cast<uint4 *>(v + r * 128);
                      const uint4 x = *t;
                      if (!nonfinite_bits(x)) continue;
                      *t = drop_nonfinite(x);
                      if (r < hi) found = true;
                    }
                  }
                }
              }
              if (found) marked[un & 15u] = static_cast<int>(un + 1);
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (lane == 0) {
              mbar_arrive(clean(s));
              mbar_arrive(freed(s));
            }
            if (++s == NS) {
              s = 0;
              phase ^= 1u;
            }
          }
        }
        if (lane == 0) mbar_arrive(u_free(un));
      }
    } else if (elect_one()) {
      // ------------------------------------------------------------ MMA issue
      // Everything between two turns of the tensor core is latency of this one
      // thread, so a turn waits as little as it can: warp 10 passes the loads
      // in order, so that one look at the latest of them covers the others.
      const int ksteps = (hd + 15) / 16;
      const uint32_t id_s = idesc_bf16(kKT, false), id_o = idesc_bf16(ksteps * 16, true);
      const uint64_t kd0 = smem_desc_sw128(base + C::kv_off), vd0 = desc_values(base + C::kv_off);
      const uint64_t qd0 = smem_desc_sw128(base + C::q_off);
      uint32_t n0 = 0;                    // loads before the unit
      uint32_t ready = 0;                 // loads known to have passed warp 10
      uint32_t np = 0, np_other = 0;      // P tiles taken from this / the other warpgroup
      uint32_t pairs = 0;                 // units with two query tiles so far
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return wait_ok(bar, parity, p.status, abort_flag);
      };
      for (uint32_t un = 0; ok; ++un) {
        if (!wait(u_full(un), (un / kUnits) & 1u)) break;
        const Unit &u = units[un % kUnits];
        if (!u.valid) break;
        const int tile = u.tile, tiles = u.stop - tile;
        const bool pair = u.pair != 0;
        const int step = pair ? 1 : 2;
        // tile index from u.tile on: the next one and the end of this and the
        // other warpgroup; tile i's keys are load n0 + 2 i, its values the next
        int cur = 0, last = pair ? min(tiles, u.ntile_a - tile) : tiles;
        int cur_other = pair ? 0 : 1, last_other = tiles;
        // A turn of warpgroup w: P V of the tile whose scores it has had, then
        // Q K^T of its next tile.  The two take turns; cur, last, np, held
        // (scores out), first belong to w and change hands after every turn.
        // Warpgroup 1 is the last user of every tile of a pair.
        bool held = false, held_other = false, first = true, first_other = true;
        int w = 0;
        if (!(ok = wait(q_full(0), un & 1u))) break;
        for (; held || held_other || cur < last || cur_other < last_other; w ^= 1) {
          const bool more = cur < last, frees = !pair || w;
          const uint32_t nk = n0 + 2 * cur, nv = n0 + 2 * (cur - step) + 1;
          // single: those keys' stage may be that of values still in use, so
          // they are waited for after P V
          const uint32_t need = more && (pair || !held) ? nk : nv;
          if ((held || more) && static_cast<int>(need - ready) >= 0) {
            if (!(ok = wait(clean(need % NS), (need / NS) & 1u))) break;
            ready = need + 1;
          }
          if (held) {
            const int s = nv % NS;
            const uint64_t vd = vd0 + s * (C::tile >> 4);
            const uint32_t o = tmem + C::o_col + w * C::o_step;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (!(ok = wait(p_full(w, half), np & 1u))) break;
              tc_fence_after();
#pragma unroll
              for (int k = 4 * half; k < 4 * half + 4; ++k)
                tc_mma_ts(o, tmem + w * 128 + 8 * k, vd + k * (2048 >> 4), id_o, !first || k > 0);
            }
            if (!ok) break;
            ++np;
            if (frees) tc_commit(freed(s));
            if (pair && !more) tc_commit(o_full(w));
            first = false;
          }
          if (more) {
            if (static_cast<int>(nk - ready) >= 0) {
              if (!(ok = wait(clean(nk % NS), (nk / NS) & 1u))) break;
              ready = nk + 1;
            }
            if (pair && w && cur == 0 && !(ok = wait(q_full(1), pairs & 1u))) break;
            const int s = nk % NS;
            const uint64_t qd = qd0 + ((pair && w) ? C::tile >> 4 : 0u);
            const uint64_t kd = kd0 + s * (C::tile >> 4);
#pragma unroll
            for (int k = 0; k < NCH * 4; ++k) {
              constexpr int kC = kChunk >> 4;
              if (k < ksteps)
                tc_mma_ss(tmem + w * 128, qd + (k / 4) * kC + (k % 4) * 2,
                          kd + (k / 4) * kC + (k % 4) * 2, id_s, k > 0);
            }
            tc_commit(s_full(w));
            if (frees) tc_commit(freed(s));
          }
          held = more;
          cur += step;
          const int c = cur, l = last;
          const uint32_t m = np;
          const bool f = first, hl = held;
          cur = cur_other, last = last_other, np = np_other, first = first_other, held = held_other;
          cur_other = c, last_other = l, np_other = m, first_other = f, held_other = hl;
        }
        if (!ok) break;
        if (w == 1) {
          const uint32_t m = np;
          np = np_other;
          np_other = m;
        }
        // single: both results at once, when nothing reads the query tile any
        // more (its shared memory carries warpgroup 1's result to warpgroup 0)
        if (!pair) {
          tc_commit(o_full(0));
          if (tiles > 1) tc_commit(o_full(1));
        }
        mbar_arrive(u_free(un));
        pairs += pair ? 1u : 0u;
        n0 += 2 * tiles;
      }
      tc_commit(drain);
      mbar_wait_bounded(drain, 0u, p.status);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---------------------------------------------------------- warpgroups
    const int w = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 (warp % 4)
    const uint32_t ts = tmem + lanes + w * 128, to = tmem + lanes + C::o_col + w * C::o_step;
    const int ochunks = (hd + 31) / 32;
    // rows of a tile are (token, head) with gsub heads a token, of which g count
    const int tok = row / p.gsub, hq = row - tok * p.gsub;
    uint32_t nt = 0, no = 0, nx = 0;
    bool ok = true;
    for (uint32_t un = 0; ok; ++un) {
      if (!(ok = wait_warp(u_full(un), (un / kUnits) & 1u))) break;
      const Unit &u = units[un % kUnits];
      if (!u.valid) break;
      int first, last, step;
      wg_tiles(u, w, first, last, step);
      const bool pair = u.pair != 0;
      const int tw = pair ? w * p.tpt : 0;    // first token of this warpgroup's query tile
      const bool live = tok < min(p.tpt, u.nt - tw) && hq < u.g;
      const bool busy = __any_sync(0xFFFFFFFFu, live);
      const int all = min(u.all + tw, u.end);  // keys every row of the tile sees
      const int vis = min(all + tok, u.end);   // keys this row sees
      float m = -INFINITY, l = 0.0f;
#pragma unroll 1
      for (int kt = first; kt < last; kt += step, ++nt) {
        if (!(ok = wait_warp(s_full(w), nt & 1u))) break;
        tc_fence_after();
        // the last read of this query tile is done
        if (pair && kt + step >= last && lane == 0) mbar_arrive(q_free(w));
        if (busy) {
          const int k0 = kt * kKT;
          uint32_t gone = 0;  // 16-key pieces in blocks outside the cache
          if (PAGED && *bad_seen) {
            const int j = k0 + lane * 16;
            bool bad = false;
            if (lane < 8 && j < u.end) {
              const int32_t id = p.a.block_table[u.r * p.a.table_stride + (j >> p.block_shift)];
              bad = id < 0 || id >= p.a.num_blocks;
            }
            gone = __ballot_sync(0xFFFFFFFFu, bad);
          }
          if (k0 + kKT > all || gone) {
            const int lim = vis - k0;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const int left = lim - 32 * c;
              uint32_t keep = left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1u;
              if (gone >> (2 * c) & 1u) keep &= 0xFFFF0000u;
              if (gone >> (2 * c + 1) & 1u) keep &= 0x0000FFFFu;
              uint32_t s[32];
              tmem_ld32(ts + 32 * c, s);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(keep >> j & 1u)) s[j] = 0xFF800000u;
              tmem_st32(ts + 32 * c, s);
            }
            tmem_wait_st();
          }
          uint32_t s[128];
          tmem_ld128(ts, s);
          float mx[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmaxf(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]));
#pragma unroll
          for (int j = 8; j < 128; j += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = max3(mx[k], __uint_as_float(s[j + 2 * k]), __uint_as_float(s[j + 2 * k + 1]));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const bool grow = (top - m) * p.sl2 > kRescale;  // -inf - -inf: NaN, no
          if (__any_sync(0xFFFFFFFFu, grow)) {
            const float mn = grow ? top : m;
            const float f = mn == m ? 1.0f : ex2((m - mn) * p.sl2);
            l *= f;
            m = mn;
            if (kt != first) {
#pragma unroll 1
              for (int c = 0; c < ochunks; ++c) {
                uint32_t o[32];
                tmem_ld32(to + 32 * c, o);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_st32(to + 32 * c, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.0f : m * p.sl2;
          const f32x2 a2 = pack2(p.sl2, p.sl2), b2 = pack2(-ref, -ref);
          f32x2 sum[2] = {0ull, 0ull};
          // P overwrites the first columns of S, and goes out in two halves:
          // the tensor core starts on the first while the second is computed
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int c = 2 * half; c < 2 * half + 2; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const int k = 32 * c + 2 * j;
                float x0, x1;
                unpack2(fma2(pack2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), a2, b2), x0, x1);
                x0 = ex2(x0);
                x1 = ex2(x1);
                sum[j & 1] = add2(sum[j & 1], pack2(x0, x1));
                pk[j] = bf16x2(x0, x1);
              }
              tmem_st16(ts + 16 * c, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(w, half));
          }
          float s0, s1;
          unpack2(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane < 2) mbar_arrive(p_full(w, lane));
        }
      }
      if (!ok) break;
      const bool have = first < last;
      if (have) {
        if (!(ok = wait_warp(o_full(w), no++ & 1u))) break;
        tc_fence_after();
      } else if (pair) {
        // no tile for warpgroup 0 here: its query tile is free, but not before
        // it is in (so that the arrival counts for this unit)
        if (!(ok = wait_warp(q_full(0), un & 1u))) break;
        if (lane == 0) mbar_arrive(q_free(0));
      }
      // single: warpgroup 1's result to warpgroup 0 through the query tiles' memory
      const bool join = !pair && u.stop - u.tile > 1;
      float *xo = reinterpret_cast<float *>(gbase + C::q_off);
      auto xat = [&](int c4) { return xo + row * (NCH * 64) + ((c4 ^ (row & 7)) << 2); };
      float f0 = 1.0f, f1 = 0.0f;
      if (!pair && w == 1) {
        if (join) {
          if (busy) {
#pragma unroll 1
            for (int c = 0; c < ochunks; ++c) {
              uint32_t o[32];
              tmem_ld32(to + 32 * c, o);
              if (live)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  *reinterpret_cast<uint4 *>(xat(8 * c + j)) =
                      make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
            if (live) {
              xm[row] = m;
              xl[row] = l;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(x_full);
        }
      } else {
        if (join) {
          if (!(ok = wait_warp(x_full, nx++ & 1u))) break;
          if (live) {
            const float m1 = xm[row], mn = fmaxf(m, m1);
            const float r = mn == -INFINITY ? 0.0f : mn;
            f0 = ex2((m - r) * p.sl2);
            f1 = ex2((m1 - r) * p.sl2);
            l = l * f0 + xl[row] * f1;
            m = mn;
          }
        }
        if (busy) {
          const bool whole = u.tile == 0 && u.stop == u.ntile;
          const float inv = whole ? (l > 0.0f || l != l ? 1.0f / l : 0.0f) : 1.0f;
          // row `line` of the partial result's slot, or of the output from the
          // unit's first row on
          const int line = whole ? (tw + tok) * p.a.n_head + hq : (tw + tok) * u.g + hq;
          const int64_t slot = (2 * blockIdx.x + (u.tile == 0 ? 1 : 0)) *
                               static_cast<int64_t>(p.parts.rows);
          const bool bf16 = whole && p.a.y_bf16;
          const int esize = bf16 ? 2 : 4, bytes = hd * esize;  // of an element, of a row
          uint8_t *out0 =
              whole ? static_cast<uint8_t *>(p.a.y) +
                          (static_cast<int64_t>(u.q_row) * p.a.n_head + u.head0) * bytes
                    : reinterpret_cast<uint8_t *>(p.parts.o + slot * hd);
          uint8_t *out = out0 + static_cast<int64_t>(line) * bytes;
          if (!whole && live)
            p.parts.ml[slot + line] = make_float2(m == -INFINITY ? m : m * p.sl2, l);
          const float k0 = f0 * inv, k1 = f1 * inv;
          // STAGED: a thread holds a row, and rows lie far apart: stored from
          // here, one instruction would touch 32 lines.  128 bytes of each row
          // go through shared memory (16-byte units swizzled by the row), and
          // eight lanes store one row's.
          uint8_t *stage = gbase + C::out_off + warp * 4096;
#pragma unroll 1
          for (int c = 0; c < ochunks; ++c) {
            float v[32];
            {
              uint32_t o[32];
              tmem_ld32(to + 32 * c, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = have ? __uint_as_float(o[j]) * k0 : 0.0f;
            }
            if (join) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float4 t = *reinterpret_cast<const float4 *>(xat(8 * c + j));
                v[4 * j] = fmaf(t.x, k1, v[4 * j]);
                v[4 * j + 1] = fmaf(t.y, k1, v[4 * j + 1]);
                v[4 * j + 2] = fmaf(t.z, k1, v[4 * j + 2]);
                v[4 * j + 3] = fmaf(t.w, k1, v[4 * j + 3]);
              }
            }
            // 16-byte unit j of this piece of the row
            auto put = [&](int j, uint4 t) {
              if constexpr (STAGED)
                *reinterpret_cast<uint4 *>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = t;
              else if (live && c * 32 * esize + 16 * j < bytes)
                *reinterpret_cast<uint4 *>(out + c * 32 * esize + 16 * j) = t;
            };
            if (bf16) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                put(STAGED ? 4 * (c & 1) + j : j,
                    make_uint4(bf16x2(v[8 * j], v[8 * j + 1]), bf16x2(v[8 * j + 2], v[8 * j + 3]),
                               bf16x2(v[8 * j + 4], v[8 * j + 5]), bf16x2(v[8 * j + 6], v[8 * j + 7])));
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                put(j, make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                  __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
            }
            if constexpr (STAGED) {
              if (bf16 && !(c & 1) && c + 1 < ochunks) continue;  // 128 bytes not full yet
              const int b0 = c * 32 * esize & ~127, j = lane & 7;
              const bool in = b0 + 16 * j < bytes;
              uint8_t *col = out0 + b0 + 16 * j;
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int r = 4 * k + (lane >> 3);
                const uint4 t = *reinterpret_cast<const uint4 *>(stage + r * 128 + ((j ^ (r & 7)) << 4));
                const int at = __shfl_sync(0xFFFFFFFFu, live ? line : -1, r);
                if (at >= 0 && in) *reinterpret_cast<uint4 *>(col + static_cast<int64_t>(at) * bytes) = t;
              }
              __syncwarp();
            }
          }
          if (live && marked[un & 15u] == static_cast<int>(un + 1))
            add_marked<PAGED>(p, u, vis, out, bf16);
        }
        if (!pair) fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        // single: warpgroup 0 is the last to use the query tiles' memory
        if (!pair && w == 0) {
          mbar_arrive(q_free(0));
          mbar_arrive(q_free(1));
        }
        mbar_arrive(u_free(un));
      }
    }
    zero_loose_rows(p.a, p.sc, blockIdx.x, gridDim.x, 256);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

// bf16 [rows][heads][head_dim] as a 3-D map, box [64 columns, heads, rows].
bool map_rows(CUtensorMap *m, const void *p, int64_t rows, int64_t stride, int heads, int hd,
              int box_heads, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(hd) * 2, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 [block][n_kv][block_size][head_dim] as a 4-D map, box [64 columns,
// box_rows, 1, 1].
bool map_blocks(CUtensorMap *m, const void *p, const AttnBatch &a, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t hd = a.head_dim;
  cuuint64_t dims[4] = {hd, static_cast<cuuint64_t>(a.block_size), static_cast<cuuint64_t>(a.n_kv),
                        static_cast<cuuint64_t>(a.num_blocks)};
  cuuint64_t strides[3] = {hd * 2, hd * 2 * a.block_size, static_cast<cuuint64_t>(a.block_stride) * 2};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NCH, bool PAGED, bool STAGED>
cudaError_t run_tc(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const TcAttn &p,
                   int workers, cudaStream_t s) {
  auto kern = attn_tc_kernel<NCH, PAGED, STAGED>;
  constexpr uint32_t smem = Tc<NCH, STAGED>::bytes;
  static_assert(smem <= 227 * 1024, "shared memory");
  const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(workers), dim3(kThreads), smem, s, q, k, v, p);
}

}  // namespace

// Head sizes a multiple of 8 up to 128 (TMA rows of whole 16-byte units;
// tensor memory holds two 128-column results), rows and blocks 16 bytes apart.
bool attn_tc_takes(const AttnBatch &a) {
  if (!a.bf16 || a.head_dim % 8 != 0 || a.head_dim > 128 || a.q_stride % 8 != 0) return false;
  const int64_t most = int64_t(1) << 38;  // strides below 2^40 bytes
  if (a.q_stride > most) return false;
  if (a.block_table) return a.num_blocks > 0 && a.block_stride % 8 == 0 && a.block_stride < most;
  return a.k_stride % 8 == 0 && a.v_stride % 8 == 0 && a.k_stride < most && a.v_stride < most;
}

// Requests of up to a query tile on average: the form for decoding.
static bool tc_few(bool paged, int64_t T, int gsub, int R) {
  return paged && T * gsub <= static_cast<int64_t>(128) * R;
}

AttnPlan attn_tc_plan(bool paged, int64_t T, int n_head, int n_kv, int R) {
  const int grp = n_head / n_kv;
  AttnPlan p;
  p.rows = 256;
  p.gsub = grp < 128 ? grp : 128;
  p.nsub = (grp + p.gsub - 1) / p.gsub;
  p.U = 2 * (128 / p.gsub);
  p.KT = kKT;
  const bool few = tc_few(paged, T, p.gsub, R);
  // a unit costs about three tiles besides its own (4.4 us of 1.4 us each);
  // one with a single query tile less, as do its tiles
  p.fixed = few ? 5 * kKT / 2 : 3 * kKT;
  p.min_run = 2 * kKT;
  p.whole = kWholeKeys;  // a prompt of 37 tokens 8.1 us, 10.7 with a launch to join
  p.workers = sm_count();
  return p;
}

cudaError_t launch_attn_tc(const AttnBatch &a, const AttnPlan &pl, const AttnSched &sc,
                           const AttnParts &parts, cudaStream_t s) {
  TcAttn p{};
  p.a = a;
  p.sc = sc;
  p.parts = parts;
  p.gsub = pl.gsub;
  p.nsub = pl.nsub;
  p.tpt = pl.U / 2;
  p.box_rows = a.block_table ? (a.block_size < kKT ? a.block_size : kKT) : kKT;
  while (a.block_table && (1 << p.block_shift) < a.block_size) ++p.block_shift;
  p.sl2 = a.scale * 1.4426950408889634f;
  p.status = device_status();
  if (!p.status) return cudaErrorInvalidDevice;
  CUtensorMap q, k, v;
  bool ok = map_rows(&q, a.q, a.T, a.q_stride, a.n_head, a.head_dim, p.gsub, p.tpt);
  if (a.block_table)
    ok = ok && map_blocks(&k, a.k, a, p.box_rows) && map_blocks(&v, a.v, a, p.box_rows);
  else
    ok = ok && map_rows(&k, a.k, a.T, a.k_stride, a.n_kv, a.head_dim, 1, kKT) &&
         map_rows(&v, a.v, a.T, a.v_stride, a.n_kv, a.head_dim, 1, kKT);
  if (!ok) return cudaErrorInvalidValue;
  const bool few = tc_few(a.block_table != nullptr, a.T, p.gsub, a.R);
  if (!a.block_table)
    return a.head_dim <= 64 ? run_tc<1, false, true>(q, k, v, p, pl.workers, s)
                            : run_tc<2, false, true>(q, k, v, p, pl.workers, s);
  if (a.head_dim <= 64)
    return few ? run_tc<1, true, false>(q, k, v, p, pl.workers, s)
               : run_tc<1, true, true>(q, k, v, p, pl.workers, s);
  return few ? run_tc<2, true, false>(q, k, v, p, pl.workers, s)
             : run_tc<2, true, true>(q, k, v, p, pl.workers, s);
}

}  // namespace qmm
