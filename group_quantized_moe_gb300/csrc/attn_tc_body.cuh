// attn_tc_body.cuh -- the body of the tensor-core attention kernels: attn_tc.cu
// (bf16 keys and values, packed or paged) and attn4_tc.cu (a paged cache held in
// 4 bits).  What they compute and how their warps share it stands there.
#pragma once

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

constexpr int kKT = 128;              // keys per tile
constexpr int kWarpKv = 8, kWarpMma = 9, kWarpClean = 10, kWarpQ = 11;
constexpr int kWarpCodes = 12;        // 4-bit cache: four warps for keys (to fp16), four for values (to bf16)
constexpr int kRaw = 3;               // half tiles of codes in flight
constexpr uint32_t kChunk = 128 * 128;  // bytes of 128 rows x 64 bf16 columns
constexpr int kUnits = 4;             // units in the ring between warp 11 and the others
constexpr float kRescale = 8.0f;      // log2 of the growth of the maximum that is let pass

// NCH: 64-column chunks of the head size.  STAGED: results go out through
// shared memory, which leaves room for four key and value tiles; without it
// there are five, which decoding needs (it is bound by the loads in flight:
// 64 requests 236 us with five tiles, 252 us with four) and can afford (few
// rows to store).
template <int NCH, bool STAGED, bool Q4>
struct Tc {
  static constexpr int threads = Q4 ? 640 : 384;
  static constexpr uint32_t tile = NCH * kChunk;            // one Q, K or V tile
  static constexpr int stages = NCH == 1 ? (STAGED || Q4 ? 8 : 10) : (STAGED || Q4 ? 4 : 5);  // K, V in turn
  static constexpr uint32_t q_off = 0, kv_off = 2 * tile;
  // codes of 64 keys: four strips of up to two chunks a column chunk, groups of 32
  static constexpr uint32_t raw_off = kv_off + stages * tile, raw = Q4 ? 4 * 2 * NCH * (512 + 128) : 0;
  static constexpr uint32_t out_off = raw_off + kRaw * raw;    // 4 KB a warp: 32 rows of 128 bytes
  static constexpr uint32_t bar_off = out_off + (STAGED ? 8 * 4096 : 0);
  // q_full[2], q_free[2], x_full, drain, s_full[2], p_full[2][2], o_full[2],
  // u_full[kUnits], u_free[kUnits], then full, freed, clean [stages], and raw_full,
  // raw_free [kRaw], q_ready [kUnits + 1]
  static constexpr int nbar = 14 + 2 * kUnits + 3 * stages + 2 * kRaw + kUnits + 1;
  static constexpr uint32_t unit_off = (bar_off + nbar * 8 + 15) & ~15u;
  static constexpr uint32_t misc_off = unit_off + kUnits * 64;  // tmem, abort, bad, -, marked[16], strips[kRaw + 1]
  // 4-bit keys: by tile, whether a warp scaled rows of it [4], what their scores are to be
  // multiplied by [128].  A ring twice as deep as that of the key tiles: the commit behind
  // Q K^T that frees a key tile says nothing of the warpgroups, which read marks and
  // factors after it.  Tile t + key_slots is made once Q K^T of tile t + key_slots / 2 is
  // done, which is issued after the weights of tile t have been handed over.
  static constexpr int key_slots = Q4 ? stages : 0;
  static constexpr uint32_t key_off = misc_off + 96 + 2 * 128 * 4;
  static constexpr uint32_t bytes = key_off + key_slots * 528 + 1024;
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
  int most_e;           // (4-bit keys) of the power of two that a query row is scaled by
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
// The same, but numbers beyond bf16's largest become that one, not infinities.
__device__ __forceinline__ uint32_t bf16x2_finite(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
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

// bf16 x bf16 (f16: fp16 x fp16) -> fp32, M = 128; values: B with N contiguous.
__device__ __forceinline__ uint32_t idesc_bf16(int n, bool values, bool f16 = false) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (values ? 1u << 16 : 0u) |
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

// The same for a 4-bit cache, where a value is not finite if its group's scale is
// not: all of the group.
__device__ __noinline__ void add_marked4(const TcAttn &p, const Kv4 &c, const Unit &u, int vis, void *out, bool bf16) {
  const int hd = p.a.head_dim, strip = kv4_strip(c);
  const int last = min(min(vis, u.end), u.stop * kKT);
#pragma unroll 1
  for (int j = max(u.tile * kKT, max(u.all, 0)); j < last; ++j) {
    const int32_t id = p.a.block_table[u.r * p.a.table_stride + (j >> c.block_shift)];
    if (id < 0 || id >= c.num_blocks) continue;
    const int row = j & ((1 << c.block_shift) - 1);
    const uint32_t *par = reinterpret_cast<const uint32_t *>(
        c.data + id * c.block_stride + static_cast<int64_t>(u.h) * kv4_head_bytes(c) + (row >> 4) * strip +
        512 * c.nc + 64 * c.ng + (row & 15) * 4 * c.ng);
#pragma unroll 1
    for (int d = 0; d < hd; ++d) {
      const float s = __uint_as_float(par[d / (32 * c.cpg)] & 0xFFFF0000u);
      if (fabsf(s) <= 3.0e38f) continue;
      if (bf16)
        static_cast<__nv_bfloat16 *>(out)[d] = __float2bfloat16_rn(s);
      else
        static_cast<float *>(out)[d] = s;
    }
  }
}

// (code - zp) s of eight codes in bf16, each rounded once.  Codes and zero points
// of up to 120 are whole numbers that bf16 has (0x4300 + code is 128 + code), and
// so are their differences; WIDE ones go through fp32, as do scales of 2^121 or more:
// their values may be beyond bf16's largest, and an infinity would make a NaN of the
// weight 0 of a row that does not see it.  Dimensions j and j + 4 become neighbours, as
// a mask leaves them: where results leave tensor memory, dim_at finds dimension j of 32.
__device__ __forceinline__ bool wide_values(uint32_t par) {
  // (of an fp16's bits: its magnitude is above 120's, or it is not a number)
  return (par & 0x7FFFu) > 0x5780u || par >= 0x7C000000u;
}
template <bool Q4>
__device__ __forceinline__ constexpr int dim_at(int j) {
  return Q4 ? (j & ~7) + (j % 8 < 4 ? 2 * (j % 8) : 2 * (j % 8) - 7) : j;
}
template <bool WIDE>
struct Dequant {
  __nv_bfloat162 zp, s;  // 128 + zp, s
  float zf, sf;
  __device__ __forceinline__ void set(uint32_t par) {
    zf = __half2float(__ushort_as_half(static_cast<unsigned short>(par)));
    sf = __uint_as_float(par & 0xFFFF0000u);
    zp = __float2bfloat162_rn(128.0f + zf);
    const uint32_t b = __byte_perm(par, 0u, 0x3232u);
    s = *reinterpret_cast<const __nv_bfloat162 *>(&b);
  }
  __device__ __forceinline__ uint4 of(uint32_t w) const {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (WIDE) {
        r[i] = bf16x2_finite((static_cast<float>(w >> (4 * i) & 15u) - zf) * sf,
                             (static_cast<float>(w >> (4 * i + 16) & 15u) - zf) * sf);
      } else {
        const uint32_t t = (w >> (4 * i) & 0x000F000Fu) | 0x43004300u;
        const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&t), zp), s);
        r[i] = *reinterpret_cast<const uint32_t *>(&v);
      }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
};

// Eight dimensions of every chunk of a row (unit: which eight), from their words
// and the groups' parameters (0 gives zeros), to row `key` of a tile.
template <bool WIDE, int NC, int CPG>
__device__ __forceinline__ void put_row(uint8_t *tile, int key, int unit, const uint32_t (&w)[NC],
                                        const uint32_t (&par)[(NC + CPG - 1) / CPG]) {
  uint8_t *const row = tile + key * 128;
  Dequant<WIDE> q;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (c % CPG == 0) q.set(par[c / CPG]);
    *reinterpret_cast<uint4 *>(row + (c >> 1) * kChunk + ((((c & 1) * 4 + unit) ^ (key & 7)) << 4)) = q.of(w[c]);
  }
}

// A key row's like it in fp16, which holds (code - zp) s to 2^-11 of it where bf16
// holds 2^-8 (with bf16 keys a chunk's result is off by 0.0028 of its norm, with
// fp16 ones 0.0020): scores magnify what is lost.  s: scales that have been
// brought into fp16's range.  Dimensions j and j + 4 of eight become neighbours, as
// a mask leaves them, in keys and queries alike (scale_query): 13 instructions an
// eight codes, 19 in their order.
__device__ __forceinline__ bool wide_zp16(uint32_t par) { return (par & 0x7FFFu) > 0x63D0u; }  // above 1000
template <bool WIDE, int NC, int CPG>
__device__ __forceinline__ void put_key(uint8_t *tile, int key, int unit, const uint32_t (&w)[NC],
                                        const uint32_t (&par)[(NC + CPG - 1) / CPG], float scale) {
  uint8_t *const row = tile + key * 128;
  const __half2 sixteenth = __float2half2_rn(0.0625f);
  __half2 z2, z16, s2;
  float zf = 0.0f, sf = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (c % CPG == 0) {
      zf = __half2float(__ushort_as_half(static_cast<unsigned short>(par[c / CPG])));
      sf = __uint_as_float(par[c / CPG] & 0xFFFF0000u) * scale;
      z2 = __float2half2_rn(1024.0f + zf);
      z16 = __float2half2_rn(-64.0f - zf);
      s2 = __float2half2_rn(sf);
    }
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (WIDE) {
        const __half2 v = __floats2half2_rn((static_cast<float>(w[c] >> (4 * i) & 15u) - zf) * sf,
                                            (static_cast<float>(w[c] >> (4 * i + 16) & 15u) - zf) * sf);
        r[i] = *reinterpret_cast<const uint32_t *>(&v);
      } else {  // 0x6400 + code: 1024 + code, four bits higher 1024 + 16 code; both less zp exact
        const uint32_t at = i < 2 ? w[c] : w[c] >> 8;
        const uint32_t t = (at & (i % 2 ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
        const __half2 n = *reinterpret_cast<const __half2 *>(&t);
        const __half2 v = __hmul2(i % 2 ? __hfma2(n, sixteenth, z16) : __hsub2(n, z2), s2);
        r[i] = *reinterpret_cast<const uint32_t *>(&v);
      }
    }
    *reinterpret_cast<uint4 *>(row + (c >> 1) * kChunk + ((((c & 1) * 4 + unit) ^ (key & 7)) << 4)) =
        make_uint4(r[0], r[1], r[2], r[3]);
  }
}

__device__ __forceinline__ float pow2_of(int e) { return __int_as_float((e + 127) << 23); }

// Parameters of a group of zeros (or of values up to 2^-96, which count as zeros), and
// those of key rows that are not there: the smallest scale, 2^-100, and no zero point.
constexpr uint32_t kZeros = 0x0D800000u;
// Whether a group of keys goes into fp16 as it is: a scale in [2^-14, 2^5), which fp16
// has exactly (rounded below that, all of the group's values would be off alike, by up
// to 2^-6), and a zero point of up to 1000.
__device__ __forceinline__ bool plain_keys(uint32_t par) {
  return (par - 0x38800000u < 0x42000000u - 0x38800000u || par == kZeros) && !wide_zp16(par);
}
// The power of two that a row with other groups is divided by: none where its scales
// and values lie in fp16's range all the same, else what brings its bound
// (|zp| + 16) s >= |code - zp| s to [2^13, 2^14).
template <int G>
__device__ __forceinline__ int key_exponent(const uint32_t (&par)[G]) {
  float top = 0.0f;
  bool low = false;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    top = fmaxf(top, __uint_as_float(par[g] & 0xFFFF0000u) *
                         (fabsf(__half2float(__ushort_as_half(static_cast<unsigned short>(par[g])))) + 16.0f));
    low |= par[g] < 0x38800000u && par[g] != kZeros;
  }
  return low || top >= 0x1p15f ? static_cast<int>(__float_as_uint(top) >> 23) - 127 - 13 : 0;
}

// A query row of a tile from bf16 to fp16, times 2^E with its largest element in
// [2^14, 2^15), dimensions in put_key's order; returns E.  (An element of 2^114 or
// more becomes infinite.)
__device__ __forceinline__ int scale_query(uint8_t *tile, int row, int nch, int most) {
  auto at = [&](int c, int j) { return reinterpret_cast<uint4 *>(tile + c * kChunk + row * 128 + ((j ^ (row & 7)) << 4)); };
  uint32_t top = 0;
#pragma unroll 1
  for (int c = 0; c < nch; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint4 v = *at(c, j);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, max(x[i] & 0x7FFFu, x[i] >> 16 & 0x7FFFu));
    }
  // of bf16 bits; not finite: as it is
  const int E = top == 0 || top >= 0x7F80u ? 0 : max(-100, min(14 - (static_cast<int>(top >> 7) - 127), most));
  const float up = pow2_of(E);
#pragma unroll 1
  for (int c = 0; c < nch; ++c)
#pragma unroll 4
    for (int j = 0; j < 8; ++j) {
      const uint4 v = *at(c, j);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
      auto number = [&](int i) { return __uint_as_float(i & 1 ? x[i >> 1] & 0xFFFF0000u : x[i >> 1] << 16) * up; };
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(number(i), number(i + 4));
        r[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
      *at(c, j) = make_uint4(r[0], r[1], r[2], r[3]);
    }
  return E;
}

// N words of shared memory.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], const uint32_t *p) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) w[c] = p[c];
  }
}

// Q4: keys and values from the 4-bit cache c4, of NC4 chunks of 32 dimensions, CPG4
// to a group (tm_k, tm_v not used); 0: bf16.
template <int NCH, bool PAGED, bool STAGED, int NC4, int CPG4>
__device__ __forceinline__ void attn_tc_body(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                             const TcAttn &p, const Kv4 &c4) {
  constexpr bool Q4 = NC4 > 0;
  constexpr int G4 = Q4 ? (NC4 + CPG4 - 1) / CPG4 : 1;
  static_assert(!Q4 || (PAGED && !STAGED), "a 4-bit cache is paged, and leaves no room to stage rows");
  using C = Tc<NCH, STAGED, Q4>;
  constexpr int kThreads = C::threads;
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
  auto raw_full = [&](int s) { return bars + kStageBars + 8 * (3 * NS + s); };
  auto raw_free = [&](int s) { return bars + kStageBars + 8 * (3 * NS + kRaw + s); };
  // queries in fp16: tile A by unit (not every warp waits for every unit's), tile B
  auto q_ready = [&](uint32_t n) { return bars + kStageBars + 8 * (3 * NS + 2 * kRaw + n % kUnits); };
  const uint32_t q_ready_b = bars + kStageBars + 8 * (3 * NS + 2 * kRaw + kUnits);
  Unit *units = reinterpret_cast<Unit *>(gbase + C::unit_off);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + C::misc_off);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + C::misc_off + 4);
  volatile int *bad_seen = reinterpret_cast<volatile int *>(gbase + C::misc_off + 8);
  volatile int *marked = reinterpret_cast<volatile int *>(gbase + C::misc_off + 16);  // [16]
  volatile uint32_t *raw_strips = reinterpret_cast<volatile uint32_t *>(gbase + C::misc_off + 80);  // [kRaw]
  float *xm = reinterpret_cast<float *>(gbase + C::misc_off + 96), *xl = xm + 128;
  // of tile t of this worker, slot t % key_slots: its warps' marks, its rows' factors
  auto key_marks = [&](int slot) { return reinterpret_cast<uint4 *>(gbase + C::key_off + slot * 528); };
  auto key_factors = [&](int slot) { return reinterpret_cast<float *>(gbase + C::key_off + slot * 528 + 16); };
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
      mbar_init(u_free(k), Q4 ? 18 : 11);  // warps 0-7, 8, 9, 10 (Q4: 12 to 19)
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(freed(s), Q4 ? 1 : 2);  // the tensor core's and warp 10's
      mbar_init(clean(s), Q4 ? 4 : 1);
    }
    if constexpr (Q4)
      for (int s = 0; s < kRaw; ++s) {
        mbar_init(raw_full(s), 1);
        mbar_init(raw_free(s), 8);
      }
    if constexpr (Q4)
      for (int k = 0; k <= kUnits; ++k) mbar_init(k < kUnits ? q_ready(k) : q_ready_b, 4);
    mbar_fence_init();
    *abort_flag = 0;
    *bad_seen = 0;
    for (int k = 0; k < 16; ++k) marked[k] = 0;
  }
  if (warp == kWarpMma) tmem_alloc(smem_addr(tmem_slot), 512);
  if (threadIdx.x == kWarpKv * 32) {
    prefetch_map(&tm_q);
    if constexpr (!Q4) {
      prefetch_map(&tm_k);
      prefetch_map(&tm_v);
    }
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

  // 384 threads launched with 168 registers: 2 x 208 + 88 = 3 x 168; 640 with 96:
  // 2 x 176 + 32 + 2 x 48 = 5 x 96
  if (Q4 && warp >= kWarpCodes) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if constexpr (Q4) {
      // ------------------------- codes to tiles of keys (fp16) and values (bf16)
      // A word of a key's codes is eight dimensions, 16 bytes of its row in the
      // tile; two words of values are eight dimensions of two rows.
      const int tid = threadIdx.x & 127, strip = kv4_strip(c4), ng = c4.ng;
      const bool values = warp >= kWarpCodes + 4;
      // This thread's part of 64 keys: eight dimensions (which: part) of every chunk of
      // two rows.  Keys: rows kr of strips ks and ks + 2; values: rows 2 vr and the next
      // of strip vs, which share their words.
      const int part = tid & 3, ks = tid >> 6, kr = tid >> 2 & 15, vs = tid >> 5, vr = lane >> 2;
      int s = values ? 1 : 0, rs = 0;
      uint32_t phase = 1, raw_phase = 0;
      bool ok = true;
      for (uint32_t un = 0; ok; ++un) {
        if (!wait_warp(u_full(un), (un / kUnits) & 1u)) break;
        const Unit &ur = units[un % kUnits];
        if (!ur.valid) break;
        const int tile = ur.tile, stop = ur.stop, all = ur.all, end = ur.end;
        for (int kt = tile; kt < stop; ++kt) {
          if (!(ok = wait_warp(freed(s), phase))) break;
          uint8_t *const dst = gbase + C::kv_off + s * C::tile;
          const int slot = s / 2 + (phase ? 0 : C::key_slots / 2);  // (keys: s is even)
          bool found = false;
          uint32_t scaled = 0;  // halves of which this warp has written factors
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            const bool some = kt * kKT + 64 * half < end;
            if (some && !(ok = wait_warp(raw_full(rs), raw_phase))) break;
            const uint32_t have = some ? raw_strips[rs] : 0u;
            const uint8_t *const raw = gbase + C::raw_off + rs * C::raw;
            uint32_t w[2][NC4], par[2][G4], wide = 0;
            int key[2];  // rows in the tile
            if (!values) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int st = ks + 2 * i;
                key[i] = 64 * half + 16 * st + kr;
                const bool in = (have >> st & 1u) && kt * kKT + key[i] < end;
                lds_words<NC4>(w[i], reinterpret_cast<const uint32_t *>(raw + st * strip) + (kr * 4 + part) * NC4);
                lds_words<G4>(par[i], reinterpret_cast<const uint32_t *>(raw + st * strip + 512 * NC4) + kr * ng);
#pragma unroll
                for (int g = 0; g < G4; ++g) par[i][g] = in ? par[i][g] : kZeros;
              }
            } else {
              const uint32_t *const words = reinterpret_cast<const uint32_t *>(raw + vs * strip + 256 * NC4) +
                                            (((vr >> 2) * 8 + 2 * part) * 4 + (vr & 3)) * NC4;
              lds_words<NC4>(w[0], words);
              lds_words<NC4>(w[1], words + 4 * NC4);
#pragma unroll
              for (int c = 0; c < NC4; ++c) {
                const uint32_t lo = w[0][c], hi = w[1][c];
                w[0][c] = __byte_perm(lo, hi, 0x5410u);
                w[1][c] = __byte_perm(lo, hi, 0x7632u);
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                key[i] = 64 * half + 16 * vs + 2 * vr + i;
                const int j = kt * kKT + key[i];
                const bool in = (have >> vs & 1u) && j < end;
                lds_words<G4>(par[i], reinterpret_cast<const uint32_t *>(raw + vs * strip + 512 * NC4 + 64 * ng) +
                                          (2 * vr + i) * ng);
#pragma unroll
                for (int g = 0; g < G4; ++g) {
                  // a value that is not finite stays out of a tile that some row sees only in part
                  const bool out = j >= all && (par[i][g] & 0x7F800000u) == 0x7F800000u;
                  found |= in && out;
                  par[i][g] = in && !out ? par[i][g] : 0u;
                }
              }
            }
            if (!values) {
#pragma unroll
              for (int g = 0; g < G4; ++g) wide |= !plain_keys(par[0][g]) | !plain_keys(par[1][g]);
              if (!__any_sync(0xFFFFFFFFu, wide)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) put_key<false, NC4, CPG4>(dst, key[i], part, w[i], par[i], 1.0f);
              } else {
                scaled |= 1u << half;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int e = key_exponent<G4>(par[i]);
                  if (part == 0) key_factors(slot)[key[i]] = pow2_of(e);
                  put_key<true, NC4, CPG4>(dst, key[i], part, w[i], par[i], pow2_of(-e));
                }
              }
            } else {
#pragma unroll
              for (int g = 0; g < G4; ++g) wide |= wide_values(par[0][g]) | wide_values(par[1][g]);
              if (!__any_sync(0xFFFFFFFFu, wide)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) put_row<false, NC4, CPG4>(dst, key[i], part, w[i], par[i]);
              } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) put_row<true, NC4, CPG4>(dst, key[i], part, w[i], par[i]);
              }
            }
            __syncwarp();
            if (some) {
              if (lane == 0) mbar_arrive(raw_free(rs));
              if (++rs == kRaw) {
                rs = 0;
                raw_phase ^= 1u;
              }
            }
          }
          if (!ok) break;
          if (found) marked[un & 15u] = static_cast<int>(un + 1);
          if (!values && lane == 0) reinterpret_cast<uint32_t *>(key_marks(slot))[warp & 3] = scaled;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(clean(s));
          s += 2;
          if (s >= NS) {  // (the stages are even in number)
            s -= NS;
            phase ^= 1u;
          }
        }
        if (lane == 0) mbar_arrive(u_free(un));
      }
    }
  } else if (warp >= 8) {
    if constexpr (Q4)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    else
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
    } else if (Q4 && warp == kWarpKv) {
      // ------------------------------- codes of keys and values, 64 keys at a time
      const int strip = kv4_strip(c4), bmask = (1 << p.block_shift) - 1;
      const int64_t head_bytes = kv4_head_bytes(c4);
      uint32_t n = 0;  // half tiles loaded so far
      int rs = 0;
      uint32_t phase = 1;
      bool ok = true;
      for (uint32_t un = 0; ok; ++un) {
        if (!wait_warp(u_full(un), (un / kUnits) & 1u)) break;
        const Unit u = units[un % kUnits];
        if (!u.valid) break;
        const int32_t *table = p.a.block_table + u.r * p.a.table_stride;
        // lane = strip of the half tile
        auto block_of = [&](int hf) {
          const int k = hf * 64 + 16 * lane;
          return lane < 4 && hf < 2 * u.stop && k < u.end ? table[k >> p.block_shift] : 0;
        };
        int id = block_of(2 * u.tile);
        for (int hf = 2 * u.tile; hf < 2 * u.stop && hf * 64 < u.end; ++hf) {
          const int mine = id, k = hf * 64 + 16 * lane;
          id = block_of(hf + 1);
          const bool in = lane < 4 && k < u.end, there = in && mine >= 0 && mine < c4.num_blocks;
          if (in && !there) {
            *bad_seen = 1;
            atomicOr(p.status, kDevBadBlock);
          }
          const uint32_t have = __ballot_sync(0xFFFFFFFFu, there);
          if (!(ok = wait_warp(raw_free(rs), phase))) break;
          if (lane == 0) {
            raw_strips[rs] = have;
            mbar_arrive_expect_tx(raw_full(rs), __popc(have) * strip);
          }
          __syncwarp();
          if (there)
            bulk_g2s(base + C::raw_off + rs * C::raw + lane * strip,
                     c4.data + mine * c4.block_stride + u.h * head_bytes + ((k & bmask) >> 4) * strip, strip,
                     raw_full(rs));
          __syncwarp();
          ++n;
          if (++rs == kRaw) {
            rs = 0;
            phase ^= 1u;
          }
        }
        if (lane == 0) mbar_arrive(u_free(un));
      }
      // copies still landing (after an abort; otherwise all have been consumed)
      for (uint32_t k = n > kRaw ? n - kRaw : 0; k < n; ++k)
        mbar_wait_bounded(raw_full(k % kRaw), (k / kRaw) & 1u, p.status);
    } else if (!Q4 && warp == kWarpKv) {
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
    } else if (Q4 && warp == kWarpClean) {
      // (its work is that of the warps that make the tiles)
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
      const uint32_t id_s = idesc_bf16(kKT, false, Q4), id_o = idesc_bf16(ksteps * 16, true);
      const uint64_t kd0 = smem_desc_sw128(base + C::kv_off), vd0 = desc_values(base + C::kv_off);
      const uint64_t qd0 = smem_desc_sw128(base + C::q_off);
      uint32_t n0 = 0;                    // loads before the unit
      uint32_t ready = 0;                 // loads known to have passed warp 10
      uint32_t ready_v = 0;               // values known to be there
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
        if (!(ok = wait(Q4 ? q_ready(un) : q_full(0), (Q4 ? un / kUnits : un) & 1u))) break;
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
          // (4-bit values are made by other warps than keys, and may be behind them)
          if (Q4 && held && static_cast<int>(nv - ready_v) >= 0) {
            if (!(ok = wait(clean(nv % NS), (nv / NS) & 1u))) break;
            ready_v = nv + 1;
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
            if (pair && w && cur == 0 && !(ok = wait(Q4 ? q_ready_b : q_full(1), pairs & 1u))) break;
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
    if constexpr (Q4)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---------------------------------------------------------- warpgroups
    const int w = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 (warp % 4)
    const uint32_t ts = tmem + lanes + w * 128, to = tmem + lanes + C::o_col + w * C::o_step;
    const int ochunks = (hd + 31) / 32;
    // rows of a tile are (token, head) with gsub heads a token, of which g count
    const int tok = row / p.gsub, hq = row - tok * p.gsub;
    uint32_t nt = 0, no = 0, nx = 0;
    uint32_t loaded = 0, two = 0;  // (4-bit keys) key tiles of earlier units; units with two query tiles
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
      float m = -INFINITY, l = 0.0f, sl2 = p.sl2;
      if constexpr (Q4) {
        // the tile's queries to fp16, each row times a power of two that its scores lose again
        if (w == 0 || pair) {
          if (!(ok = wait_warp(q_full(w), (w ? two : un) & 1u))) break;
          const int E = scale_query(gbase + C::q_off + w * C::tile, row, nch, p.most_e);
          sl2 *= pow2_of(-E);
          if (!pair) xl[row] = sl2;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(w ? q_ready_b : q_ready(un));
        } else if (first < last) {
          if (!(ok = wait_warp(q_ready(un), (un / kUnits) & 1u))) break;
          sl2 = xl[row];
        }
        two += pair ? 1u : 0u;
      }
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
          if constexpr (Q4) {
            const int slot = (loaded + (kt - u.tile)) % C::key_slots;
            const uint4 marks = *key_marks(slot);
            if (marks.x | marks.y | marks.z | marks.w) {
              // row j of the tile was made by warp 2 (strip % 2) + (row of the strip) / 8
              const float *const by = key_factors(slot);
              const uint32_t mark[4] = {marks.x, marks.y, marks.z, marks.w};
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t v[32];
                tmem_ld32(ts + 32 * c, v);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (mark[j >> 3] >> (c >> 1) & 1u) v[j] = __float_as_uint(__uint_as_float(v[j]) * by[32 * c + j]);
                tmem_st32(ts + 32 * c, v);
              }
              tmem_wait_st();
            }
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
          const bool grow = (top - m) * sl2 > kRescale;  // -inf - -inf: NaN, no
          if (__any_sync(0xFFFFFFFFu, grow)) {
            const float mn = grow ? top : m;
            const float f = mn == m ? 1.0f : ex2((m - mn) * sl2);
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
          const float ref = m == -INFINITY ? 0.0f : m * sl2;
          const f32x2 a2 = pack2(sl2, sl2), b2 = pack2(-ref, -ref);
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
      loaded += u.stop - u.tile;
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
                      make_uint4(o[dim_at<Q4>(4 * j)], o[dim_at<Q4>(4 * j + 1)], o[dim_at<Q4>(4 * j + 2)],
                                 o[dim_at<Q4>(4 * j + 3)]);
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
            f0 = ex2((m - r) * sl2);
            f1 = ex2((m1 - r) * sl2);
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
            p.parts.ml[slot + line] = make_float2(m == -INFINITY ? m : m * sl2, l);
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
              for (int j = 0; j < 32; ++j) v[j] = have ? __uint_as_float(o[dim_at<Q4>(j)]) * k0 : 0.0f;
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
          if (live && marked[un & 15u] == static_cast<int>(un + 1)) {
            if constexpr (Q4)
              add_marked4(p, c4, u, vis, out, bf16);
            else
              add_marked<PAGED>(p, u, vis, out, bf16);
          }
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
inline bool map_rows(CUtensorMap *m, const void *p, int64_t rows, int64_t stride, int heads, int hd,
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

}  // namespace
}  // namespace qmm
