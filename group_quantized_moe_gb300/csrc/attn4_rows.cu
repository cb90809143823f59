// attn4_rows.cu -- batched attention over a paged cache held in 4 bits (layout:
// kv4.h) for few query rows: decoding, drafted tokens, fp32 queries.
//
// A key or value element is (code - zp) s with one zp and s per row and group.
// Both products run on the tensor cores (mma.sync, 16 x 8 x 16, fp16 operands,
// fp32 sums) on the codes themselves:
//   S[key, q] = sum_g s_g (sum_d code q' - zp_g sum_d q'),   q' = q 2^E
//   O[dim, q] = sum_key (p s_g) code,   Z[g, q] = sum_key (p s_g) zp_g
//   y = (O - Z) / l
// A masked word of the cache is an operand register: a code in bits 4 to 7 of
// an fp16 is the number code 2^-20, so that eight codes cost seven instructions
// (three shifts, four masks) and no conversion.  (In bits 0 to 3 two of the
// shifts could go, but the tensor cores line products up by the operands'
// exponents, without the leading zeros of a subnormal: sums are then cut off at
// 2^-19 of them, with the codes four bits higher at 2^-27.)  Keys and
// dimensions go to the operands' rows (16), query rows to their columns (8):
// few query rows waste little, and the scores of one product are, transposed by
// movmatrix, the weights' operand of the next.
//
// Roundings: q' is fp16 with E such that the row's largest |q'| lies in
// [2^14, 2^15): bf16 queries are exact down to 2^-29 of the largest; fp32 ones
// are split into two fp16.  The weights p s_g c are rounded to fp16 (2^-11;
// fp32 queries: split in two as well), c a power of two per query row that
// keeps them below 2^15 and moves when the maximum moves or a product would
// leave the range.  The tensor cores cut their sums off instead of rounding,
// so they run over 32 keys only and are added up in fp32.
#include <cuda_fp16.h>

#include <cstdint>

#include "attn_batch.h"
#include "attn_internal.h"
#include "attn_sched.cuh"
#include "kv4.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kKT = 32;           // keys of a step: two strips
constexpr float kRescale = 8.0f;  // log2 of the growth of the maximum that is let pass
constexpr float kTop = 32768.0f;  // of a weight

struct Attn4 {
  AttnBatch a;
  Kv4 c;
  AttnSched sc;
  AttnParts parts;
  int gsub, nsub;
  float sl2;  // scale log2(e)
  uint32_t *status;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d += a b, a [16 x 16], b [16 x 8] fp16, d fp32.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint32_t *p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p + c));
      w[c] = v.x, w[c + 1] = v.y, w[c + 2] = v.z, w[c + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p + c));
      w[c] = v.x, w[c + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) w[c] = __ldg(p + c);
  }
}

// NC: chunks of 32 dimensions; CPG: chunks of a group; NQ: tiles of eight query
// rows; F32: the queries' type (else bf16).
template <int NC, int CPG, int NQ, bool F32>
struct Form {
  static constexpr int G = (NC + CPG - 1) / CPG, R = 8 * NQ, P = F32 ? 2 : 1, HD = 32 * NC;
  // an operand of code c is (c - centre) / unit
  static constexpr float unit = F32 ? 1.0f : 0x1p20f, centre = F32 ? 8.0f : 0.0f;
  // queries as operands [P][NQ][NC][32 lanes] of 16 bytes, their group sums
  // [R][G] in an operand's unit, unit / 2^E times the scale [R], then the warps' results
  static constexpr int q_bytes = P * NQ * NC * 512;
  static constexpr int sum_off = q_bytes, ke_off = sum_off + R * G * 4;
  static constexpr int ml_off = (ke_off + R * 4 + 15) & ~15;
  static constexpr int o_off = ml_off + kWarps * R * 8;
  static constexpr int bytes = o_off + kWarps * R * HD * 4;
};

// The four operand registers of a word of codes: its nibbles (0, 4), (1, 5),
// (2, 6), (3, 7), each as code 2^-20, or with fp32 queries as code - 8: sums of
// codes that are never negative grow, and what the tensor cores cut off them is
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
  a[0] = (w << 4) & 0x00F000F0u;
  a[1] = w & 0x00F000F0u;
  a[2] = (x << 4) & 0x00F000F0u;
  a[3] = x & 0x00F000F0u;
}

// A unit's query rows as operands.  Thread t of a column's eight holds
// dimensions 32 c + 8 t + j of chunk c: pairs (0, 4), (1, 5), (2, 6), (3, 7).
template <int NC, int CPG, int NQ, bool F32>
__device__ __forceinline__ void stage_queries(const Attn4 &p, uint8_t *smem, int row0, int head0, int g, int rows) {
  using C = Form<NC, CPG, NQ, F32>;
  const int lane = threadIdx.x & 31, hd = p.a.head_dim;
  for (int row = threadIdx.x >> 5; row < C::R; row += kWarps) {
    const int t = row / g, h = head0 + row - t * g;
    float x[NC], top = 0.0f;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = 32 * c + lane;
      x[c] = 0.0f;
      if (row < rows && d < hd) {
        const int64_t i = static_cast<int64_t>(row0 + t) * p.a.q_stride + static_cast<int64_t>(h) * hd + d;
        x[c] = F32 ? __ldg(static_cast<const float *>(p.a.q) + i)
                   : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t *>(p.a.q) + i)) << 16);
      }
      top = fmaxf(top, fabsf(x[c]));
    }
#pragma unroll
    for (int o = 1; o <= 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    int E = 14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
    E = top > 0.0f ? max(-100, min(E, 100)) : 0;
    const float up = pow2i(E);
    const int n = row >> 3, col = row & 7, t4 = (lane >> 3) & 3, j = lane & 7;
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float v = x[c] * up;
      float s = v;
#pragma unroll
      for (int o = 1; o <= 16; o <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      sum = c % CPG == 0 ? s : sum + s;
      if ((c % CPG == CPG - 1 || c == NC - 1) && lane == 0)
        reinterpret_cast<float *>(smem + C::sum_off)[row * C::G + c / CPG] = sum * (1.0f / C::unit);
      // nibble j: pair j & 3, place j >> 2 of it
      const __half hi = __float2half_rn(v);
      const int at = ((n * NC + c) * 32 + col * 4 + t4) * 16 + (j & 3) * 4 + (j >> 2) * 2;
      *reinterpret_cast<__half *>(smem + at) = hi;
      if constexpr (F32)
        *reinterpret_cast<__half *>(smem + NQ * NC * 512 + at) = __float2half_rn(v - __half2float(hi));
    }
    if (lane == 0) reinterpret_cast<float *>(smem + C::ke_off)[row] = p.sl2 * C::unit * pow2i(-E);
  }
}

template <int NC, int CPG, int NQ, bool F32>
__global__ void __launch_bounds__(kThreads) attn4_rows_kernel(const __grid_constant__ Attn4 p) {
  using C = Form<NC, CPG, NQ, F32>;
  constexpr int G = C::G;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t scratch[kWarps + 4];
  pdl_enter();
  const AttnRun run = sched_run<kThreads>(p.sc, blockIdx.x, scratch);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
  const int hd = p.a.head_dim, grp = p.a.n_head / p.a.n_kv;
  const int strip = kv4_strip(p.c), head_bytes = kv4_head_bytes(p.c), bshift = p.c.block_shift;
  if (tid == 0) p.parts.open[blockIdx.x].rows_tok = 0;
  int64_t x = run.unit;
  int r = run.r, i = run.i, vh = run.h;
  AttnReq q{};
  bool fresh = true;
  while (x < run.last) {
    if (fresh) q = sched_req(p.sc, r);
    fresh = false;
    if (i >= sched_blocks(p.sc, q)) {
      if (++r >= p.sc.R) break;  // lengths that changed during the call
      i = 0;
      fresh = true;
      continue;
    }
    const int ntile = sched_tiles(p.sc, q, i), block = i, v = vh;
    const int64_t x0 = x;
    int tile, stop;
    sched_part(p.sc, run, x, ntile, tile, stop);
    x += sched_unit(p.sc, q, i);
    if (++vh == p.sc.nvh) {
      vh = 0;
      ++i;
    }
    if (tile >= stop) continue;
    const int h = v / p.nsub, sub = v - h * p.nsub, g = min(p.gsub, grp - sub * p.gsub);
    const int t0 = block * p.sc.U, nt = min(p.sc.U, q.n - t0), rows = nt * g, head0 = h * grp + sub * p.gsub;
    const int all = sched_seen(p.sc, q, t0), end = sched_end(p.sc, q, block);
    if (tid == 0 && sched_short(p.sc, q, block)) atomicOr(p.status, kDevBadBlock);
    stage_queries<NC, CPG, NQ, F32>(p, smem, q.q0 + t0, head0, g, rows);
    __syncthreads();

    // this thread's columns of tile n: query rows 8 n + 2 t4 and the next
    float o[NQ][2 * NC][4], z[NQ][G][2], qs[NQ][G][2], m[NQ][2], l[NQ][2], cw[NQ][2], top_w[NQ][2], ke[NQ][2];
    int vis[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int k = 0; k < 2 * NC; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][k][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * n + 2 * t4 + e;
        m[n][e] = -INFINITY;
        l[n][e] = top_w[n][e] = 0.0f;
        cw[n][e] = 1.0f;
        ke[n][e] = reinterpret_cast<const float *>(smem + C::ke_off)[row];
        vis[n][e] = row < rows ? min(all + row / g, end) : 0;
#pragma unroll
        for (int k = 0; k < G; ++k) {
          z[n][k][e] = 0.0f;
          qs[n][k][e] = reinterpret_cast<const float *>(smem + C::sum_off)[row * G + k];
        }
      }
    }
    const int32_t *table = p.a.block_table + r * p.a.table_stride;
    for (int kt = tile + warp; kt < stop; kt += kWarps) {
      const int k0 = kt * kKT;
      // strip u of the step: its place, and its first key that is not there
      const uint8_t *src[2];
      int lim[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = k0 + 16 * u;
        src[u] = p.c.data;
        lim[u] = k;
        if (k >= end) continue;
        const int32_t id = table[k >> bshift];
        if (id < 0 || id >= p.c.num_blocks) {
          if (lane == 0) atomicOr(p.status, kDevBadBlock);
          continue;
        }
        src[u] += id * p.c.block_stride + static_cast<int64_t>(h) * head_bytes +
                  ((k & ((1 << bshift) - 1)) >> 4) * strip;
        lim[u] = min(end, k + 16);
      }
      float s[NQ][2][4];
      uint32_t kp[2][2][G], vp[2][2][G];  // parameters of rows g8 and g8 + 8 of the strips
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool there = lim[u] > k0 + 16 * u;
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][u][e] = 0.0f;
        uint32_t kw[2][NC];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t *const par = reinterpret_cast<const uint32_t *>(src[u] + 512 * NC) + (8 * w + g8) * p.c.ng;
          // rows behind the last key may hold anything
          const bool in = k0 + 16 * u + 8 * w + g8 < lim[u];
#pragma unroll
          for (int k = 0; k < G; ++k) {
            kp[u][w][k] = in && k < p.c.ng ? __ldg(par + k) : 0u;
            vp[u][w][k] = in && k < p.c.ng ? __ldg(par + 16 * p.c.ng + k) : 0u;
          }
          if (there) {
            load_words<NC>(kw[w], reinterpret_cast<const uint32_t *>(src[u]) + (32 * w + lane) * NC);
          } else {
#pragma unroll
            for (int c = 0; c < NC; ++c) kw[w][c] = 0u;
          }
        }
#pragma unroll
        for (int k = 0; k < G; ++k) {
          float acc[NQ][4];
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
#pragma unroll
          for (int c = k * CPG; c < (k + 1) * CPG && c < NC; ++c) {
            uint32_t lo[4], hi[4];
            operands<F32>(kw[0][c], lo);
            operands<F32>(kw[1][c], hi);
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int part = 0; part < C::P; ++part) {
                const uint4 b = *reinterpret_cast<const uint4 *>(smem + (((part * NQ + n) * NC + c) * 32 + lane) * 16);
                mma(acc[n], lo[0], hi[0], lo[1], hi[1], b.x, b.y);
                mma(acc[n], lo[2], hi[2], lo[3], hi[3], b.z, b.w);
              }
          }
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float zp = low_half(kp[u][w][k]) - C::centre, sc = __uint_as_float(kp[u][w][k] & 0xFFFF0000u);
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                s[n][u][2 * w + e] = fmaf(sc, fmaf(-zp, qs[n][k][e], acc[n][2 * w + e]), s[n][u][2 * w + e]);
          }
        }
      }
      // weights
      uint32_t b[NQ][2][G][2][C::P];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float top[2] = {-INFINITY, -INFINITY};
        uint32_t gone = 0;  // keys that the rows do not see
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = k0 + 16 * u + 8 * (e >> 1) + g8;
            float y = s[n][u][e] * ke[n][e & 1];
            if (key >= min(vis[n][e & 1], lim[u])) {
              y = -INFINITY;
              gone |= 1u << (4 * u + e);
            }
            s[n][u][e] = y;
            top[e & 1] = fmaxf(top[e & 1], y);
          }
        float f[2] = {1.0f, 1.0f};
        bool move = false;
        if (__any_sync(0xFFFFFFFFu, top[0] > m[n][0] + kRescale || top[1] > m[n][1] + kRescale)) {
          move = true;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float t = column_max(top[e]);
            if (t > m[n][e] + kRescale) {
              f[e] = ex2(m[n][e] - t);
              m[n][e] = t;
              l[n][e] *= f[e];
              top_w[n][e] *= f[e];
            }
          }
        }
        float w[2][G][4], most[2] = {0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float ref = m[n][e & 1] == -INFINITY ? 0.0f : m[n][e & 1];
            const float pr = ex2(s[n][u][e] - ref);
            l[n][e & 1] += pr;
            const float pc = pr * cw[n][e & 1];
#pragma unroll
            for (int k = 0; k < G; ++k) {
              float t = pc * __uint_as_float(vp[u][e >> 1][k] & 0xFFFF0000u);
              if (gone >> (4 * u + e) & 1u) t = 0.0f;
              w[u][k][e] = t;
              most[e & 1] = fmaxf(most[e & 1], t);
            }
          }
        if (__any_sync(0xFFFFFFFFu, move || most[0] > kTop || most[1] > kTop)) {
          // c anew: the largest weight so far to [2^7, 2^8)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float t = fmaxf(column_max(most[e]), top_w[n][e]);
            float turn = 1.0f;
            if (t > 0.0f) {
              const int old = static_cast<int>(__float_as_uint(cw[n][e]) >> 23);  // biased exponents
              const int E = old + 7 - (static_cast<int>(__float_as_uint(t) >> 23) - 127);
              const float cn = __uint_as_float(static_cast<uint32_t>(max(2, min(min(E, old + 100), 252))) << 23);
              turn = cn / cw[n][e];
              cw[n][e] = cn;
            }
            top_w[n][e] = t * turn;
            f[e] *= turn;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int k = 0; k < G; ++k)
#pragma unroll
                for (int j = e; j < 4; j += 2) w[u][k][j] *= turn;
#pragma unroll
            for (int k = 0; k < G; ++k) z[n][k][e] *= f[e];
#pragma unroll
            for (int k = 0; k < 2 * NC; ++k) {
              o[n][k][e] *= f[e];
              o[n][k][2 + e] *= f[e];
            }
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int k = 0; k < G; ++k)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const float w0 = w[u][k][2 * half], w1 = w[u][k][2 * half + 1];
              const float zp = low_half(vp[u][half][k]) - C::centre;
              z[n][k][0] = fmaf(w0, zp, z[n][k][0]);
              z[n][k][1] = fmaf(w1, zp, z[n][k][1]);
              const uint32_t hi = half2_of(w0, w1);
              b[n][u][k][half][0] = transpose8(hi);
              if constexpr (F32)
                b[n][u][k][half][C::P - 1] = transpose8(half2_of(w0 - low_half(hi), w1 - low_half(hi >> 16)));
            }
      }
      uint32_t vw[2][2][NC];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (lim[u] > k0 + 16 * u) {
            load_words<NC>(vw[u][half], reinterpret_cast<const uint32_t *>(src[u] + 256 * NC) + (32 * half + lane) * NC);
          } else {
#pragma unroll
            for (int c = 0; c < NC; ++c) vw[u][half][c] = 0u;
          }
        }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float acc[NQ][2][4];
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[n][e >> 2][e & 3] = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t lo[4], hi[4];
          operands<F32>(vw[u][0][c], lo);
          operands<F32>(vw[u][1][c], hi);
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int part = 0; part < C::P; ++part) {
              const uint32_t b0 = b[n][u][c / CPG][0][part], b1 = b[n][u][c / CPG][1][part];
              mma(acc[n][0], lo[0], lo[1], hi[0], hi[1], b0, b1);
              mma(acc[n][1], lo[2], lo[3], hi[2], hi[3], b0, b1);
            }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 8; ++e) o[n][2 * c + (e >> 2)][e & 3] += acc[n][e >> 2][e & 3];
      }
    }

    // the warps' results meet in shared memory
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * n + 2 * t4 + e;
        const float sum = column_sum(l[n][e]), inv = 1.0f / cw[n][e];
        if (g8 == 0) reinterpret_cast<float2 *>(smem + C::ml_off)[warp * C::R + row] = make_float2(m[n][e], sum);
        float *const out = reinterpret_cast<float *>(smem + C::o_off) + (warp * C::R + row) * C::HD;
#pragma unroll
        for (int k = 0; k < G; ++k) z[n][k][e] = column_sum(z[n][k][e]);
        auto put = [&](float v, float zz) { return fmaf(v, C::unit, -zz) * inv; };
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float zz = z[n][c / CPG][e];
          // dimensions 4 g8 .. + 3 of the chunk: rows g8 and g8 + 8 of two products
          *reinterpret_cast<float4 *>(out + 32 * c + 4 * g8) =
              make_float4(put(o[n][2 * c][e], zz), put(o[n][2 * c][2 + e], zz),
                          put(o[n][2 * c + 1][e], zz), put(o[n][2 * c + 1][2 + e], zz));
        }
      }
    __syncthreads();
    const bool whole = tile == 0 && stop == ntile;
    const int slot = 2 * blockIdx.x + (tile == 0 ? 1 : 0);
    for (int e = tid; e < rows * (C::HD / 4); e += kThreads) {
      const int row = e / (C::HD / 4), d = 4 * (e - row * (C::HD / 4));
      if (d >= hd) continue;
      const float2 *const ml = reinterpret_cast<const float2 *>(smem + C::ml_off) + row;
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * C::R].x);
      const float ref = M == -INFINITY ? 0.0f : M;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        // (zeros of a warp that saw no key count nothing; a NaN makes the row NaN,
        // however small its warp's factor is)
        const float f = ex2(ml[w * C::R].x - ref);
        const float4 t = *reinterpret_cast<const float4 *>(smem + C::o_off + ((w * C::R + row) * C::HD + d) * 4);
        L = fmaf(f, ml[w * C::R].y, L);
        acc.x = fmaf(f, t.x, acc.x);
        acc.y = fmaf(f, t.y, acc.y);
        acc.z = fmaf(f, t.z, acc.z);
        acc.w = fmaf(f, t.w, acc.w);
      }
      if (whole) {
        const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;
        const int t = row / g, hq = row - t * g;
        store_y4(p.a.y, (static_cast<int64_t>(q.q0 + t0 + t) * p.a.n_head + head0 + hq) * hd + d,
                 make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv), p.a.y_bf16);
      } else {
        const int64_t base = static_cast<int64_t>(slot) * p.parts.rows + row;
        if (d == 0) p.parts.ml[base] = make_float2(M, L);
        *reinterpret_cast<float4 *>(p.parts.o + base * hd + d) = acc;
      }
    }
    __syncthreads();
    if (tid == 0 && tile == 0 && !whole)
      p.parts.open[blockIdx.x] = AttnOpen{q.q0 + t0, nt, v, sched_last(p.sc, run, x0, ntile)};
  }
  zero_loose_rows(p.a, p.sc, blockIdx.x, gridDim.x, kThreads);
}

template <int NC, int CPG, int NQ, bool F32>
cudaError_t run_form(const Attn4 &p, int workers, cudaStream_t s) {
  auto kern = attn4_rows_kernel<NC, CPG, NQ, F32>;
  constexpr int smem = Form<NC, CPG, NQ, F32>::bytes;
  static_assert(smem <= 227 * 1024, "shared memory");
  const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(workers), dim3(kThreads), smem, s, p);
}

template <int NC, int CPG, int NQ>
cudaError_t run_type(const Attn4 &p, int workers, cudaStream_t s) {
  return p.a.bf16 ? run_form<NC, CPG, NQ, false>(p, workers, s) : run_form<NC, CPG, NQ, true>(p, workers, s);
}

template <int NC>
cudaError_t run_nc(const Attn4 &p, int rows, int workers, cudaStream_t s) {
  if constexpr (NC > 1) {
    if (p.c.cpg == 2) {
      if constexpr (NC <= 4)
        if (rows > 8) return run_type<NC, 2, 2>(p, workers, s);
      return run_type<NC, 2, 1>(p, workers, s);
    }
  }
  if constexpr (NC <= 4)
    if (rows > 8) return run_type<NC, 1, 2>(p, workers, s);
  return run_type<NC, 1, 1>(p, workers, s);
}

}  // namespace

AttnPlan attn4_rows_plan(const Kv4 &c, int64_t T, int n_head, int R) {
  const int grp = n_head / c.n_kv;
  // rows that a request has for a key/value head, on average
  const int64_t usual = R > 0 ? (T + R - 1) / R * grp : grp;
  AttnPlan p;
  p.rows = usual > 8 && c.nc <= 4 ? 16 : 8;
  p.gsub = grp < p.rows ? grp : p.rows;
  p.nsub = (grp + p.gsub - 1) / p.gsub;
  p.U = p.rows / p.gsub;
  p.KT = kKT;
  p.fixed = 4 * kKT;
  p.min_run = kWarps * kKT;
  p.whole = kWholeKeys;
  p.workers = sm_count();
  return p;
}

cudaError_t launch_attn4_rows(const AttnBatch &a, const Kv4 &c, const AttnPlan &pl, const AttnSched &sc,
                              const AttnParts &parts, cudaStream_t s) {
  Attn4 p{a, c, sc, parts, pl.gsub, pl.nsub, a.scale * 1.4426950408889634f, device_status()};
  if (!p.status) return cudaErrorInvalidDevice;
  switch (c.nc) {
    case 1: return run_nc<1>(p, pl.rows, pl.workers, s);
    case 2: return run_nc<2>(p, pl.rows, pl.workers, s);
    case 3: return run_nc<3>(p, pl.rows, pl.workers, s);
    case 4: return run_nc<4>(p, pl.rows, pl.workers, s);
    case 6: return run_nc<6>(p, pl.rows, pl.workers, s);
    default: return run_nc<8>(p, pl.rows, pl.workers, s);
  }
}

}  // namespace qmm
