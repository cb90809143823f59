// attn4_rows.cu -- batched attention over a paged cache held in 4 bits (layout:
// kv4.h) for few query rows: decoding, drafted tokens, fp32 queries.
//
// A key or value element is (code - zp) s with one zp and s per row and group.
// Both products run on the tensor cores (mma.sync, 16 x 8 x 16, fp16 operands,
// fp32 sums) on the codes themselves:
//   S[key, q] = sum_g s_g (sum_d code q' - zp_g sum_d q'),   q' = q 2^E
//   O[dim, q] = sum_key (p s_g) code,   Z[g, q] = sum_key (p s_g) zp_g
//   y = (O - Z) / l
// A masked word of the cache is an operand register: a code in the low four
// bits of an fp16 is the number code 2^-24, and one four bits higher 16 times
// that, so that eight codes cost five instructions and no conversion.  What is
// odd about the factors is put right once: queries of odd places are divided by
// 16 where they are made, odd rows of O when a unit ends.  (The tensor cores line
// products up by the operands' exponents, without the leading zeros of a
// subnormal, so sums with codes in the lowest bits are cut off at about 2^-19 of
// the sum of their magnitudes: far below the weights' rounding, but not for fp32
// queries, which take the codes as whole numbers.)  Keys and dimensions go to
// the operands' rows (16), query rows to their columns (8): few query rows waste
// little, and the scores of one product are, transposed by movmatrix, the
// weights' operand of the next.
//
// Roundings: q' is fp16 with E such that the row's largest |q'| lies in
// [2^14, 2^15): bf16 queries are exact down to 2^-25 of the largest; fp32 ones
// are split into two fp16.  The weights p s_g c are rounded to fp16 (2^-11;
// fp32 queries: split in two as well), c a power of two per query row and group
// that keeps them below 2^15 and moves when the maximum moves or the scale of a
// value is so large that a product could leave the range: each group's own, as the
// others' scales may lie any number of powers of two away.  Z takes them before the
// rounding, which then costs 15 steps of a scale at most, not |zp| of them.  The
// tensor cores' sums of weights run over 32 keys and are added up in fp32.
//
// Measured, 32 heads of 128 over 8, groups of 64, bf16: one token of 64 requests of
// 5400 keys (400 MB of cache) 105 us, 3.8 TB/s, 55 % of a copy; with direct loads
// instead of bulk copies ahead of each warp 226, with conversions in place of masked
// words 111.  DRAM reads are the cache's bytes.  Nothing is full: DRAM 49 %, issue
// slots 45 %, the integer pipe 47 %.  What bounds it is the chain within a warp
// (products, maximum, exponentials, products; 322 instructions to a strip of 2.3 KB):
// of three warps to a scheduler one can issue in 51 % of the cycles.  Fifteen warps of
// 128 registers spill.  Half of each product's columns are empty with four heads to a
// key/value head.  fp32 queries, with two parts to each, 42 us for 12 requests, 32
// heads over 32 (49 MB).  Each further eight query rows of a head cost a pass over the
// codes: 40 requests of 2000 keys 38 us with 4 rows, 74 with 16, 126 with 32.
#include <cuda_fp16.h>

#include <cstdint>

#include "attn_batch.h"
#include "attn_internal.h"
#include "attn_sched.cuh"
#include "kv4.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"
#include "tc_device.cuh"

namespace qmm {
namespace {

constexpr int kKT = 32;           // keys of a step: two strips
constexpr int kUnits = 32;           // units in the ring between the loading warp and the others
constexpr int kAlone = 12;           // tiles of a unit that one warp takes alone (750 requests of
                                    // 200 keys 87 us; 181 where eleven warps share seven tiles)
constexpr float kRescale = 8.0f;  // log2 of the growth of the maximum that is let pass
constexpr float kTop = 32768.0f;  // of a weight
constexpr float kMost = 0x1p120f;  // of a power of two that it is multiplied by, and that to begin with

struct Attn4 {
  AttnBatch a;
  Kv4 c;
  AttnSched sc;
  AttnParts parts;
  int gsub, nsub;
  float sl2;   // scale log2(e)
  int most_e;  // of the power of two that a query row is scaled by
  uint32_t *status;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d += a b (first: d = a b), a [16 x 16], b [16 x 8] fp16, d fp32.
__device__ __forceinline__ void mma(bool first, float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(first ? 0.0f : d[0]), "f"(first ? 0.0f : d[1]),
        "f"(first ? 0.0f : d[2]), "f"(first ? 0.0f : d[3]));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float low_half(uint32_t v) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(v)));
}

// Maximum over the eight lanes that hold one column of the scores.
__device__ __forceinline__ float column_max(float v) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ float column_sum(float v) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Whether the phase with the given parity is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Keeps a rarely taken block behind a branch (not predicated, which would cost
// its instructions every time).
__device__ __forceinline__ void branch() { asm volatile("" ::: "memory"); }

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// N words of shared memory, 16 bytes at a time where they lie so.
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t *p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * c);
      w[c] = v.x, w[c + 1] = v.y, w[c + 2] = v.z, w[c + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const uint2 v = *reinterpret_cast<const uint2 *>(p + 4 * c);
      w[c] = v.x, w[c + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) w[c] = *reinterpret_cast<const uint32_t *>(p + 4 * c);
  }
}

// The four operand registers of a word of codes: its nibbles (0, 4), (1, 5),
// (2, 6), (3, 7), each as code 2^-24 (odd ones 16 times that), or with fp32
// queries as code - 8: sums of codes that are never negative grow, and what the tensor cores cut off them is
// then no longer small against a result in which most of them cancel (1.7e-6 of
// its norm for 300 tokens of 2500 keys; centred 2.6e-7).
template <bool F32>
__device__ __forceinline__ void operands(uint32_t w, uint32_t (&a)[4]) {
  if constexpr (F32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t v = (w >> (4 * k) & 0x000F000Fu) | 0x64006400u;  // 1024 + code
      const __half2 c = __hsub2(*reinterpret_cast<const __half2 *>(&v), __half2half2(__ushort_as_half(0x6408)));
      a[k] = *reinterpret_cast<const uint32_t *>(&c);
    }
    return;
  }
  const uint32_t x = w >> 8;
  a[0] = w & 0x000F000Fu;
  a[1] = w & 0x00F000F0u;
  a[2] = x & 0x000F000Fu;
  a[3] = x & 0x00F000F0u;
}

// NC: chunks of 32 dimensions; CPG: chunks of a group; F32: the queries' type
// (else bf16).  A unit has up to eight query rows: one tile of columns.  (Two tiles
// share the codes' unpacking but leave a thread registers for seven warps instead
// of eleven: 32 drafted tokens a head 82 us either way.)
template <int NC, int CPG, bool F32>
struct Form {
  static constexpr int G = (NC + CPG - 1) / CPG, R = 8, P = F32 ? 2 : 1, HD = 32 * NC;
  // an operand of code c is (c - centre) / unit, at odd places odd times that
  static constexpr float unit = F32 ? 1.0f : 0x1p24f, centre = F32 ? 8.0f : 0.0f, odd = F32 ? 1.0f : 16.0f;
  // warps that multiply, and one that loads: three to a scheduler leave a thread
  // 168 registers, two 255
  static constexpr int warps = NC <= 4 && !(F32 && NC == 4 && CPG == 1) ? 11 : 7, threads = 32 * (warps + 1);
  static constexpr int stage = 2 * (512 * NC + 128 * G);  // a tile of the cache
  static constexpr bool qreg = !F32 && NC <= 4;    // queries in registers, else in shared memory
  static constexpr int q_warp = qreg ? 0 : P * NC * 512, q_bytes = warps * q_warp;
  static constexpr int OS = HD + 4;  // floats between rows of results (four lanes store one each)
  static constexpr int o_bytes = warps * R * OS * 4, ml_bytes = warps * R * 8;
  static constexpr int fixed = q_bytes + o_bytes + ml_bytes + kUnits * 64 + 2048;
  static constexpr int room = (225 * 1024 - fixed) / (stage * warps);
  static constexpr int depth = room < 4 ? room : 4;  // tiles in flight a warp
  static constexpr int stages = depth * warps;
  static constexpr int o_off = stages * stage, ml_off = o_off + o_bytes, q_off = ml_off + ml_bytes;
  static constexpr int unit_off = (q_off + q_bytes + 15) & ~15, bar_off = unit_off + kUnits * 64;
  // full [stages], u_full, joined, wrote [kUnits], the abort flag
  static constexpr int flag_off = bar_off + 8 * (stages + 3 * kUnits);
  static constexpr int bytes = flag_off + 16;
  static_assert(depth >= 1 && bytes <= 227 * 1024, "shared memory");
};

// One unit of this worker's run, as the warps see it.
struct __align__(16) Unit4 {
  int valid, q_row, rows, g;    // 0: no unit any more; first query row, rows, heads
  int h, head0, r, pad;         // key/value head, first query head, request
  int tile, stop, whole, slot;  // this worker's tiles [tile, stop); all of them: not divided; its slot if not
  int all, end, alone, n0;      // keys the first / last token sees; one warp has all tiles; turn of its first
};

// A query row's elements as operands: lane 4 col + t holds dimensions
// 32 c + 8 t + j of row `col`, in pairs (0, 4), (1, 5), (2, 6), (3, 7).
// ke: unit / 2^E scale log2 e, sum: by group, both of that row.
template <int NC, int CPG, bool F32>
__device__ __forceinline__ void make_queries(const Attn4 &p, const Unit4 &u, uint32_t (&op)[F32 ? 2 : 1][NC][4],
                                             float (&sum)[Form<NC, CPG, F32>::G], float &ke) {
  using C = Form<NC, CPG, F32>;
  const int lane = threadIdx.x & 31, row = lane >> 2, t4 = lane & 3, hd = p.a.head_dim;
  const int t = row / u.g;
  const int64_t i = static_cast<int64_t>(u.q_row + t) * p.a.q_stride + static_cast<int64_t>(u.head0 + row - t * u.g) * hd;
  float x[NC][8], top = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int d = 32 * c + 8 * t4;
    const bool in = row < u.rows && d < hd;
    if constexpr (F32) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 v = in ? __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p.a.q) + i + d) + k)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        x[c][4 * k] = v.x, x[c][4 * k + 1] = v.y, x[c][4 * k + 2] = v.z, x[c][4 * k + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // (rows are multiples of 8 bytes apart)
        const uint2 v = in ? __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.a.q) + i + d) + k)
                           : make_uint2(0, 0);
        x[c][4 * k] = __uint_as_float(v.x << 16), x[c][4 * k + 1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[c][4 * k + 2] = __uint_as_float(v.y << 16), x[c][4 * k + 3] = __uint_as_float(v.y & 0xFFFF0000u);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[c][j]));
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  int E = 14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
  E = top > 0.0f ? max(-100, min(E, p.most_e)) : 0;
  const float up = pow2i(E);
  ke = p.sl2 * C::unit * pow2i(-E);
#pragma unroll
  for (int k = 0; k < C::G; ++k) sum[k] = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[c][j] *= up;
      sum[c / CPG] += x[c][j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float part = j & 1 ? 1.0f / C::odd : 1.0f;
      op[0][c][j] = half2_of(x[c][j] * part, x[c][j + 4] * part);
      if constexpr (F32)
        op[C::P - 1][c][j] = half2_of(x[c][j] - low_half(op[0][c][j]), x[c][j + 4] - low_half(op[0][c][j] >> 16));
    }
  }
#pragma unroll
  for (int k = 0; k < C::G; ++k) {
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) sum[k] += __shfl_xor_sync(0xFFFFFFFFu, sum[k], o);
    sum[k] *= 1.0f / C::unit;
  }
}

// Four elements of row `row` of a unit: of the output, or of its partial result.
__device__ __forceinline__ void store_row4(const Attn4 &p, const Unit4 &u, int row, int d, float4 v) {
  const int hd = p.a.head_dim, t = row / u.g;
  if (u.whole)
    store_y4(p.a.y, (static_cast<int64_t>(u.q_row + t) * p.a.n_head + u.head0 + row - t * u.g) * hd + d, v, p.a.y_bf16);
  else
    *reinterpret_cast<float4 *>(p.parts.o + (static_cast<int64_t>(u.slot) * p.parts.rows + row) * hd + d) = v;
}

template <int NC, int CPG, bool F32>
__global__ void __launch_bounds__(Form<NC, CPG, F32>::threads, 1)
    attn4_rows_kernel(const __grid_constant__ Attn4 p) {
  using C = Form<NC, CPG, F32>;
  constexpr int G = C::G, NW = C::warps, NS = C::stages, D = C::depth, P = C::P;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scratch[NW + 1 + 4];
  const uint32_t base = smem_addr(smem), bars = base + C::bar_off;
  auto full = [&](int s) { return bars + 8 * s; };
  auto u_full = [&](uint32_t n) { return bars + 8 * (NS + n % kUnits); };
  auto joined = [&](uint32_t n) { return bars + 8 * (NS + kUnits + n % kUnits); };
  auto wrote = [&](uint32_t n) { return bars + 8 * (NS + 2 * kUnits + n % kUnits); };
  volatile int *const abort_flag = reinterpret_cast<volatile int *>(smem + C::flag_off);
  Unit4 *const units = reinterpret_cast<Unit4 *>(smem + C::unit_off);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(full(s), 1);
    for (int k = 0; k < kUnits; ++k) {
      mbar_init(u_full(k), 1);
      mbar_init(joined(k), 1);
      mbar_init(wrote(k), NW);
    }
    mbar_fence_init();
    *abort_flag = 0;
  }
  pdl_enter();
  const AttnRun run = sched_run<C::threads>(p.sc, blockIdx.x, scratch);
  if (tid == 0) p.parts.open[blockIdx.x].rows_tok = 0;
  __syncthreads();
  const int hd = p.a.head_dim, strip = 512 * NC + 128 * (NC <= 4 ? G : p.c.ng);
  auto wait_warp = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, wait_ok(bar, parity, p.status, abort_flag)) != 0;
  };

  if (warp == NW) {
    // -------------------- units of the run, and the warps' results of them joined
    const int grp = p.a.n_head / p.a.n_kv;
    int64_t x = run.unit;
    int r = run.r, i = run.i, vh = run.h;
    AttnReq q{};
    bool fresh = true;
    uint32_t n = 0;  // the warps' turns so far
    // Short units of a long run go to one warp each: nothing to join, and others
    // run beside it.
    const bool many = run.last - run.first >= 2 * NW * kAlone * kKT;
    // the next unit of the run with tiles of it
    auto next_unit = [&]() {
      Unit4 u{};
      while (x < run.last) {
        if (fresh) q = sched_req(p.sc, r);
        fresh = false;
        if (i >= sched_blocks(p.sc, q)) {
          if (++r >= p.sc.R) break;  // lengths that changed during the call
          i = 0;
          fresh = true;
          continue;
        }
        const int ntile = sched_tiles(p.sc, q, i);
        sched_part(p.sc, run, x, ntile, u.tile, u.stop);
        if (u.tile < u.stop) {
          u.valid = 1;
          u.h = vh / p.nsub;
          const int sub = vh - u.h * p.nsub, t0 = i * p.sc.U, nt = min(p.sc.U, q.n - t0);
          u.g = min(p.gsub, grp - sub * p.gsub);
          u.q_row = q.q0 + t0;
          u.rows = nt * u.g;
          u.head0 = u.h * grp + sub * p.gsub;
          u.r = r;
          u.whole = u.tile == 0 && u.stop == ntile;
          u.slot = 2 * blockIdx.x + (u.tile == 0 ? 1 : 0);
          u.all = sched_seen(p.sc, q, t0);
          u.end = sched_end(p.sc, q, i);
          u.n0 = static_cast<int>(n);
          u.alone = many && u.stop - u.tile <= kAlone;
          if (lane == 0 && sched_short(p.sc, q, i)) atomicOr(p.status, kDevBadBlock);
          if (lane == 0 && u.tile == 0 && !u.whole)
            p.parts.open[blockIdx.x] = AttnOpen{u.q_row, nt, vh, sched_last(p.sc, run, x, ntile)};
        }
        x += sched_unit(p.sc, q, i);
        if (++vh == p.sc.nvh) {
          vh = 0;
          ++i;
        }
        if (u.valid) break;
      }
      return u;
    };
    uint32_t made = 0, done = 0;  // units handed out, joined
    bool more = true;
    while (true) {
      while (more && made - done < kUnits) {
        const Unit4 u = next_unit();
        if (lane == 0) {
          units[made % kUnits] = u;
          mbar_arrive(u_full(made));
        }
        __syncwarp();
        n += u.alone ? 1 : u.stop - u.tile;
        more = u.valid != 0;
        if (more) ++made;
      }
      if (done == made || !wait_warp(wrote(done), (done / kUnits) & 1u)) break;
      // the warps' results of a unit: part k is warp (n0 + k) % NW's
      const Unit4 u = units[done % kUnits];
      const int parts = u.alone ? 1 : min(NW, u.stop - u.tile), first = static_cast<uint32_t>(u.n0) % NW;
      if (parts > 1) {
        const float2 *const ml = reinterpret_cast<const float2 *>(smem + C::ml_off);
        auto part = [&](int k) { return first + k < NW ? first + k : first + k - NW; };
        // lane = row: its maximum and sum
        float M = -INFINITY, L = 0.0f;
        const int mine = min(lane, C::R - 1);
#pragma unroll 4
        for (int k = 0; k < parts; ++k) M = fmaxf(M, ml[part(k) * C::R + mine].x);
        const float ref = M == -INFINITY ? 0.0f : M;
        // (zeros of a warp that saw no key count nothing; a NaN makes the row NaN,
        // however small its warp's factor is)
#pragma unroll 4
        for (int k = 0; k < parts; ++k) {
          const float2 v = ml[part(k) * C::R + mine];
          L = fmaf(ex2(v.x - ref), v.y, L);
        }
        const float inv = u.whole ? (L > 0.0f || L != L ? 1.0f / L : 0.0f) : 1.0f;
        if (!u.whole && lane < u.rows)
          p.parts.ml[static_cast<int64_t>(u.slot) * p.parts.rows + lane] = make_float2(M, L);
        const int from = part(min(lane, parts - 1));
#pragma unroll 2
        for (int row = 0; row < u.rows; ++row) {
          // lane = part: its factor
          const float f = ex2(ml[from * C::R + row].x - __shfl_sync(0xFFFFFFFFu, ref, row)) *
                          __shfl_sync(0xFFFFFFFFu, inv, row);
#pragma unroll
          for (int c0 = 0; c0 < 8 * NC; c0 += 32) {
            const int d = 4 * (c0 + lane);
            const float *const o = reinterpret_cast<const float *>(smem + C::o_off) + row * C::OS + min(d, C::HD - 4);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int k = 0; k < parts; ++k) {
              const float4 v = *reinterpret_cast<const float4 *>(o + part(k) * C::R * C::OS);
              const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
              acc.x = fmaf(fk, v.x, acc.x);
              acc.y = fmaf(fk, v.y, acc.y);
              acc.z = fmaf(fk, v.z, acc.z);
              acc.w = fmaf(fk, v.w, acc.w);
            }
            if (d < hd) store_row4(p, u, row, d, acc);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(joined(done));
      ++done;
    }
  } else {
    // ---------------------------------------------------------------- products
    // Tile n of the worker is warp n % NW's, which also fetches it, up to D tiles
    // ahead and across units, into a stage of its own.
    const int bshift = p.c.block_shift, bmask = (1 << bshift) - 1;
    const int64_t head_bytes = kv4_head_bytes(p.c);
    int ahead = 0, f_stage = 0;    // tiles fetched and not used; stage of the next one
    int stage = 0;                 // of the next one to be used, and its barrier's parity
    uint32_t parity = 0;
    uint32_t here = 0;             // two bits a stage: its strips that are in the cache
    // the unit that is being fetched, this warp's tiles left of it and their
    // distance; sixteen of them at a time: lane 2 i + u has the place of strip u of
    // tile i, and the block of that strip of the next sixteen
    uint32_t f_un = 0xFFFFFFFFu, f_have = 0;
    int f_key = 0, f_end = 0, f_left = 0, f_step = NW, f_batch = 0;
    const int32_t *f_table = nullptr;
    const uint8_t *f_head = nullptr, *f_src = nullptr;
    int32_t f_id = 0;
    bool f_more = true, ok = true;
    auto look = [&](int key) {
      const int k = key + (lane >> 1) * f_step * kKT + 16 * (lane & 1);
      return k < f_end ? f_table[k >> bshift] : 0;
    };
    // places of the sixteen tiles from f_key on, whose blocks have been looked up
    auto place = [&]() {
      const int k = f_key + (lane >> 1) * f_step * kKT + 16 * (lane & 1);
      const bool in = k < f_end, there = in && f_id >= 0 && f_id < p.c.num_blocks;
      if (in && !there) atomicOr(p.status, kDevBadBlock);
      f_have = __ballot_sync(0xFFFFFFFFu, there);
      f_src = f_head + f_id * p.c.block_stride + ((k & bmask) >> 4) * strip;
      f_batch = 0;
      f_id = look(f_key + 16 * f_step * kKT);
    };
    // fetches this warp's next tile, if there is one before unit `limit`
    auto fetch = [&](uint32_t limit) {
      while (f_left <= 0) {
        // (a unit that is not there yet is left for later: this may run ahead)
        if (!f_more || f_un + 1 >= limit ||
            !__all_sync(0xFFFFFFFFu, mbar_test(u_full(f_un + 1), ((f_un + 1) / kUnits) & 1u)))
          return;
        ++f_un;
        const Unit4 &u = units[f_un % kUnits];
        if (!(f_more = u.valid != 0)) return;
        const int rank = (warp + NW - static_cast<uint32_t>(u.n0) % NW) % NW;
        f_step = u.alone ? 1 : NW;
        f_left = u.alone ? (rank == 0 ? u.stop - u.tile : 0) : (u.stop - u.tile - rank + NW - 1) / NW;
        if (f_left <= 0) continue;
        f_key = (u.tile + rank) * kKT;
        f_end = min(u.end, u.stop * kKT);
        f_head = p.c.data + u.h * head_bytes;
        f_table = p.a.block_table + u.r * p.a.table_stride;
        f_id = look(f_key);
        place();
      }
      const uint32_t have = f_have >> (2 * f_batch) & 3u;
      here = (here & ~(3u << (2 * f_stage))) | have << (2 * f_stage);
      if ((lane >> 1) == f_batch) {
        const int s = warp * D + f_stage, u = lane & 1;
        if (u == 0) mbar_arrive_expect_tx(full(s), __popc(have) * strip);
        // strips of one block follow one another
        const int bytes = (bshift > 4 ? (u ? 0 : __popc(have)) : have >> u & 1) * strip;
        if (bytes) bulk_g2s(base + s * C::stage + u * strip, f_src, bytes, full(s));
      }
      __syncwarp();
      ++ahead;
      f_stage = f_stage + 1 == D ? 0 : f_stage + 1;
      --f_left;
      f_key += f_step * kKT;
      if (++f_batch == 16) place();
    };
    uint32_t last_un = 0;  // the unit whose results this warp has in shared memory, plus one
    for (uint32_t un = 0;; ++un) {
      if (!ok || !wait_warp(u_full(un), (un / kUnits) & 1u)) break;
      const Unit4 &us = units[un % kUnits];
      if (!us.valid) break;
      // as far ahead as the ring of units goes (this unit is there: its first tile is not missed)
#pragma unroll 1
      for (int k = 0; k < D && ahead < D; ++k) fetch(un + kUnits);
      // the warps from n0 % NW on have its tiles; the others go on to the next unit
      const int rank = (warp + NW - static_cast<uint32_t>(us.n0) % NW) % NW;
      const int parts = us.alone ? 1 : min(NW, us.stop - us.tile), step = us.alone ? 1 : NW;
      if (rank >= parts) {
        if (lane == 0) mbar_arrive(wrote(un));
        continue;
      }
      const Unit4 u = us;
      // this thread's columns: query rows 2 t4 and the next
      uint32_t qop[P][C::qreg ? NC : 1][4];
      float o[2 * NC][4], z[G][2], qs[G][2], m[2], l[2], cw[G][2], ke[2];
      int vis[2];
      uint8_t *const qmem = smem + C::q_off + warp * C::q_warp;
        float sum[G], k;
        if constexpr (C::qreg) {
          make_queries<NC, CPG, F32>(p, u, qop, sum, k);
        } else {
          uint32_t op[P][NC][4];
          make_queries<NC, CPG, F32>(p, u, op, sum, k);
#pragma unroll
          for (int part = 0; part < P; ++part)
#pragma unroll
            for (int c = 0; c < NC; ++c)
              *reinterpret_cast<uint4 *>(qmem + ((part * NC + c) * 32 + lane) * 16) =
                  make_uint4(op[part][c][0], op[part][c][1], op[part][c][2], op[part][c][3]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int from = 4 * (2 * t4 + e);
          ke[e] = __shfl_sync(0xFFFFFFFFu, k, from);
#pragma unroll
          for (int j = 0; j < G; ++j) qs[j][e] = __shfl_sync(0xFFFFFFFFu, sum[j], from);
        }
#pragma unroll
        for (int k = 0; k < 2 * NC; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][e] = 0.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 2 * t4 + e;
          m[e] = -INFINITY;
          l[e] = 0.0f;
          vis[e] = row < u.rows ? min(u.all + row / u.g, u.end) : 0;
#pragma unroll
          for (int k = 0; k < G; ++k) {
            z[k][e] = 0.0f;
            cw[k][e] = kMost;
          }
        }
#pragma unroll 1
      for (int kt = u.tile + rank; kt < u.stop; kt += step) {
        const int s = warp * D + stage;
        if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(full(s), parity)) && !(ok = wait_warp(full(s), parity))) break;
        const int k0 = kt * kKT;
        const uint8_t *const at = smem + s * C::stage;
        const uint32_t have = here >> (2 * stage) & 3u;
        // some row misses some key of the tile
        const bool guard = k0 + kKT > u.all || have != 3u;
        float sc[2][4];
        uint32_t vp[2][2][G];  // value parameters of rows g8 and g8 + 8 of the strips
#pragma unroll
        for (int w2 = 0; w2 < 2; ++w2) {
          const uint8_t *const src = at + w2 * strip;
          uint32_t kw[2][NC], kp[2][G];
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            load_words<NC>(kw[w], src + (32 * w + lane) * 4 * NC);
            if constexpr (NC <= 4) {
              load_words<G>(kp[w], src + 512 * NC + (8 * w + g8) * 4 * G);
              load_words<G>(vp[w2][w], src + 512 * NC + 64 * G + (8 * w + g8) * 4 * G);
            } else {
#pragma unroll
              for (int k = 0; k < G; ++k) {
                const int kk = min(k, p.c.ng - 1);  // (a chunk of padding has no group: its codes are zeros)
                kp[w][k] = reinterpret_cast<const uint32_t *>(src + 512 * NC)[(8 * w + g8) * p.c.ng + kk];
                vp[w2][w][k] = reinterpret_cast<const uint32_t *>(src + 512 * NC)[(16 + 8 * w + g8) * p.c.ng + kk];
              }
            }
          }
          if (guard) {
            branch();
            // rows behind the last key may hold anything
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const bool in = (have >> w2 & 1u) && k0 + 16 * w2 + 8 * w + g8 < u.end;
#pragma unroll
              for (int k = 0; k < G; ++k)
                if (!in) kp[w][k] = vp[w2][w][k] = 0u;
            }
          }
#pragma unroll
          for (int k = 0; k < G; ++k) {
            float acc[4];
#pragma unroll
            for (int c = k * CPG; c < (k + 1) * CPG && c < NC; ++c) {
              uint32_t lo[4], hi[4];
              operands<F32>(kw[0][c], lo);
              operands<F32>(kw[1][c], hi);
#pragma unroll
                for (int part = 0; part < P; ++part) {
                  uint32_t b[4];
                  if constexpr (C::qreg) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) b[j] = qop[part][c][j];
                  } else {
                    load_words<4>(b, qmem + ((part * NC + c) * 32 + lane) * 16);
                  }
                  mma(c == k * CPG && part == 0, acc, lo[0], hi[0], lo[1], hi[1], b[0], b[1]);
                  mma(false, acc, lo[2], hi[2], lo[3], hi[3], b[2], b[3]);
                }
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              float zp = low_half(kp[w][k]);
              if constexpr (F32) zp -= C::centre;
              const float ks = __uint_as_float(kp[w][k] & 0xFFFF0000u);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float t = fmaf(-zp, qs[k][e], acc[2 * w + e]);
                  float &y = sc[w2][2 * w + e];
                  y = k == 0 ? ks * t : fmaf(ks, t, y);
                }
            }
          }
        }
        // weights
        // The scale of some value is so large that a weight could leave fp16's range.
        bool large = false;
#pragma unroll
        for (int k = 0; k < G; ++k) {
          const float most = fmaxf(fmaxf(__uint_as_float(vp[0][0][k]), __uint_as_float(vp[0][1][k])),
                                   fmaxf(__uint_as_float(vp[1][0][k]), __uint_as_float(vp[1][1][k])));
          large |= most * fmaxf(cw[k][0], cw[k][1]) > kTop / 256.0f;
        }
        uint32_t b[2][G][2][P];
          uint32_t gone = 0;  // keys that the rows do not see
          if (guard) {
            branch();
#pragma unroll
            for (int w2 = 0; w2 < 2; ++w2)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = k0 + 16 * w2 + 8 * (e >> 1) + g8;
                if (key >= vis[e & 1] || !(have >> w2 & 1u)) {
                  sc[w2][e] = -INFINITY;
                  gone |= 1u << (4 * w2 + e);
                }
              }
          }
          float top[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            top[e] = fmaxf(fmaxf(sc[0][e], sc[0][2 + e]), fmaxf(sc[1][e], sc[1][2 + e])) * ke[e];
          // or a row's maximum moves on by more than kRescale
          const bool move =
              __any_sync(0xFFFFFFFFu, top[0] > m[0] + kRescale || top[1] > m[1] + kRescale || large);
          float f[2] = {1.0f, 1.0f};
          if (move) {
            branch();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float t = column_max(top[e]);
              if (t > m[e] + kRescale) {
                f[e] = ex2(m[e] - t);
                m[e] = t;
                l[e] *= f[e];
              }
            }
          }
          float w[2][4];
#pragma unroll
          for (int w2 = 0; w2 < 2; ++w2)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float mm = m[e & 1] == -INFINITY ? 0.0f : m[e & 1];
              w[w2][e] = ex2(fmaf(sc[w2][e], ke[e & 1], -mm));
              l[e & 1] += w[w2][e];
            }
          if (move) {
            branch();
            // c of each group anew: the largest product to [2^4, 2^5), of this tile or, at
            // least 2^4 / c, of those before
#pragma unroll
            for (int k = 0; k < G; ++k) {
              float most[2] = {0.0f, 0.0f};
#pragma unroll
              for (int w2 = 0; w2 < 2; ++w2)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (!(gone >> (4 * w2 + e) & 1u))  // (2^-10: scales up to 2^125)
                    most[e & 1] = fmaxf(most[e & 1], w[w2][e] * 0x1p-10f * __uint_as_float(vp[w2][e >> 1][k] & 0xFFFF0000u));
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int old = static_cast<int>(__float_as_uint(cw[k][e]) >> 23);  // biased exponents
                const float before = f[e] * __uint_as_float(static_cast<uint32_t>(248 - old) << 23);
                const float t = fmaxf(column_max(most[e]), before);
                const int now = max(5, min(248 - static_cast<int>(__float_as_uint(t) >> 23), 247));
                cw[k][e] = __uint_as_float(static_cast<uint32_t>(now) << 23);
                const int turn = now - old;
                const float f0 = f[e] * pow2i(turn / 2), f1 = pow2i(turn - turn / 2);
                z[k][e] = z[k][e] * f0 * f1;
#pragma unroll
                for (int c = 2 * CPG * k; c < 2 * CPG * (k + 1) && c < 2 * NC; ++c) {
                  o[c][e] = o[c][e] * f0 * f1;
                  o[c][2 + e] = o[c][2 + e] * f0 * f1;
                }
              }
            }
          }
          constexpr int KB = G < 4 ? G : 4;  // groups at a time (registers)
#pragma unroll
          for (int kb = 0; kb < G; kb += KB) {
            float ws[2][KB][4];
#pragma unroll
            for (int k = kb; k < kb + KB && k < G; ++k) {
              const f32x2 c2 = pack2(cw[k][0], cw[k][1]);
#pragma unroll
              for (int w2 = 0; w2 < 2; ++w2)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const float s = __uint_as_float(vp[w2][half][k] & 0xFFFF0000u);
                  unpack2(mul2(mul2(pack2(w[w2][2 * half], w[w2][2 * half + 1]), c2), pack2(s, s)),
                          ws[w2][k - kb][2 * half], ws[w2][k - kb][2 * half + 1]);
                }
            }
            if (guard) {
              branch();
              // not even 0 * NaN of a key that is not seen
#pragma unroll
              for (int w2 = 0; w2 < 2; ++w2)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (gone >> (4 * w2 + e) & 1u)
#pragma unroll
                    for (int k = 0; k < KB; ++k) ws[w2][k][e] = 0.0f;
            }
#pragma unroll
            for (int w2 = 0; w2 < 2; ++w2)
#pragma unroll
              for (int k = kb; k < kb + KB && k < G; ++k)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const float w0 = ws[w2][k - kb][2 * half], w1 = ws[w2][k - kb][2 * half + 1];
                  float zp = low_half(vp[w2][half][k]);
                  if constexpr (F32) zp -= C::centre;
                  z[k][0] = fmaf(w0, zp, z[k][0]);
                  z[k][1] = fmaf(w1, zp, z[k][1]);
                  const uint32_t hi = half2_of(w0, w1);
                  b[w2][k][half][0] = transpose8(hi);
                  if constexpr (F32)
                    b[w2][k][half][P - 1] = transpose8(half2_of(w0 - low_half(hi), w1 - low_half(hi >> 16)));
                }
          }
        uint32_t vw[2][2][NC];
#pragma unroll
        for (int w2 = 0; w2 < 2; ++w2)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            load_words<NC>(vw[w2][half], at + w2 * strip + 256 * NC + (32 * half + lane) * 4 * NC);
        __syncwarp();
        --ahead;
        if (++stage == D) {
          stage = 0;
          parity ^= 1u;
        }
        fetch(un + kUnits);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float acc[2][4];
#pragma unroll
          for (int w2 = 0; w2 < 2; ++w2) {
            uint32_t lo[4], hi[4];
            operands<F32>(vw[w2][0][c], lo);
            operands<F32>(vw[w2][1][c], hi);
#pragma unroll
              for (int part = 0; part < P; ++part) {
                const uint32_t b0 = b[w2][c / CPG][0][part], b1 = b[w2][c / CPG][1][part];
                mma(w2 == 0 && part == 0, acc[0], lo[0], lo[1], hi[0], hi[1], b0, b1);
                mma(w2 == 0 && part == 0, acc[1], lo[2], lo[3], hi[2], hi[3], b0, b1);
              }
          }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 4; e += 2)
                unpack2(add2(pack2(o[2 * c + k][e], o[2 * c + k][e + 1]), pack2(acc[k][e], acc[k][e + 1])),
                        o[2 * c + k][e], o[2 * c + k][e + 1]);
        }
      }
      if (!ok) break;

      // This warp's result to shared memory, once its last one there has been joined
      // to the others' (sure, if the ring of units has gone round since); one that is
      // the whole unit's goes out from here.
      const bool only = parts == 1;
      if (!only) {
        if (last_un > 0 && un + 1 - last_un < kUnits &&
            !(ok = wait_warp(joined(last_un - 1), ((last_un - 1) / kUnits) & 1u)))
          break;
        last_un = un + 1;
      }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 2 * t4 + e;
          const float sum = column_sum(l[e]);
          const float inv = only && u.whole ? (sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f) : 1.0f;
          if (g8 == 0) {
            if (!only)
              reinterpret_cast<float2 *>(smem + C::ml_off)[warp * C::R + row] = make_float2(m[e], sum);
            else if (!u.whole && row < u.rows)
              p.parts.ml[static_cast<int64_t>(u.slot) * p.parts.rows + row] = make_float2(m[e], sum);
          }
          float *const out = reinterpret_cast<float *>(smem + C::o_off) + (warp * C::R + row) * C::OS;
#pragma unroll
          for (int k = 0; k < G; ++k) z[k][e] = column_sum(z[k][e]);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float zz = z[c / CPG][e];
            const float down = __uint_as_float((254u << 23) - __float_as_uint(cw[c / CPG][e]));  // 1 / c
            auto put = [&](float v, float zz, float odd) { return fmaf(v, C::unit / odd, -zz) * down * inv; };
            // dimensions 4 g8 .. + 3 of the chunk: rows g8 and g8 + 8 of two products
            const float4 v = make_float4(put(o[2 * c][e], zz, 1.0f), put(o[2 * c][2 + e], zz, C::odd),
                                         put(o[2 * c + 1][e], zz, 1.0f), put(o[2 * c + 1][2 + e], zz, C::odd));
            const int d = 32 * c + 4 * g8;
            if (!only)
              *reinterpret_cast<float4 *>(out + d) = v;
            else if (row < u.rows && d < hd)
              store_row4(p, u, row, d, v);
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(wrote(un));
    }
    // copies still landing (after an abort; otherwise all have been used)
    for (; ahead > 0; --ahead) {
      mbar_wait_bounded(full(warp * D + stage), parity, p.status);
      if (++stage == D) {
        stage = 0;
        parity ^= 1u;
      }
    }
    zero_loose_rows(p.a, p.sc, blockIdx.x, gridDim.x, 32 * NW);
  }
}

template <int NC, int CPG, bool F32>
cudaError_t run_form(const Attn4 &p, int workers, cudaStream_t s) {
  auto kern = attn4_rows_kernel<NC, CPG, F32>;
  constexpr int smem = Form<NC, CPG, F32>::bytes;
  const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(workers), dim3(Form<NC, CPG, F32>::threads), smem, s, p);
}

template <int NC, int CPG>
cudaError_t run_type(const Attn4 &p, int workers, cudaStream_t s) {
  return p.a.bf16 ? run_form<NC, CPG, false>(p, workers, s) : run_form<NC, CPG, true>(p, workers, s);
}

template <int NC>
cudaError_t run_nc(const Attn4 &p, int workers, cudaStream_t s) {
  if constexpr (NC > 1)
    if (p.c.cpg == 2) return run_type<NC, 2>(p, workers, s);
  return run_type<NC, 1>(p, workers, s);
}

}  // namespace

AttnPlan attn4_rows_plan(const Kv4 &c, int n_head) {
  const int grp = n_head / c.n_kv;
  AttnPlan p;
  p.rows = 8;
  p.gsub = grp < p.rows ? grp : p.rows;
  p.nsub = (grp + p.gsub - 1) / p.gsub;
  p.U = p.rows / p.gsub;
  p.KT = kKT;
  // A unit costs 2 to 4 us besides its keys, of which a CTA does 170 a us (64 requests
  // of 100 to 16384 keys: 108 us; 132 with 128 keys, where workers of short ones lag).
  p.fixed = 640;
  p.min_run = 4 * kKT;
  p.whole = kWholeKeys;
  p.workers = sm_count();
  return p;
}

cudaError_t launch_attn4_rows(const AttnBatch &a, const Kv4 &c, const AttnPlan &pl, const AttnSched &sc,
                              const AttnParts &parts, cudaStream_t s) {
  const float sl2 = a.scale * 1.4426950408889634f;
  Attn4 p{a, c, sc, parts, pl.gsub, pl.nsub, sl2, kv4_most_exponent(sl2), device_status()};
  if (!p.status) return cudaErrorInvalidDevice;
  switch (c.nc) {
    case 1: return run_nc<1>(p, pl.workers, s);
    case 2: return run_nc<2>(p, pl.workers, s);
    case 3: return run_nc<3>(p, pl.workers, s);
    case 4: return run_nc<4>(p, pl.workers, s);
    case 6: return run_nc<6>(p, pl.workers, s);
    default: return run_nc<8>(p, pl.workers, s);
  }
}

}  // namespace qmm
