// kv4_rows.cu -- rows of a paged cache held in 4 bits (layout: kv4.h): rotary
// positions with the quantising write, and reading rows back.
//
// A key (rotated as in rope_append.cu, in fp32) or value row is quantised per
// head and group of 32 or 64 dimensions:
//   lo, hi = min, max;  top = max(|lo|, |hi|)
//   s  = the next bf16 at or above max((hi - lo) / 15, top / 2048, 2^-100)
//   zp = -rint(lo / s), code = clamp(rint(v / s) + zp, 0, 15)
// with 1 / s rounded to fp32 once and multiplied, every step one rounding, so
// that the codes are defined bit for bit.  Rounding the scale up costs no
// range, and codes are taken with the scale as it is stored.  top / 2048 holds
// |zp| to 2048, which fp16 has exactly; a group so narrow that this decides is
// off by at most top / 4096, less than bf16's own rounding.  A group with a
// NaN or an infinity gets the scale NaN: all of it reads as NaN.
//
// Four lanes hold a row of a head, each eight dimensions of every chunk of 32:
// a lane's codes of a key are consecutive words of the cache, and a group's
// extremes meet in two shuffles.  A warp takes four heads of two tokens at a time;
// where they are neighbours in the cache (prompts), each lane stores or loads
// whole words of both, which share the words of values.
//
// Measured, 32 heads of 128 over 8, groups of 64:
//   append  16384 tokens in bf16, 354 MB in and out: 81 us, 4.4 TB/s.  One token and
//           eight heads a warp took 195 us: half words of values were stored one by
//           one.  Four blocks an SM: 3, 5 and 6 took 122, 102 and 126 (four: 87).
//           Nothing is full (issue slots 54 %, DRAM 53 %, integer pipe 49 %): warps
//           wait for their rows, 8 of the 13 cycles between two instructions, with
//           nothing of the next pair in flight.  87 -> 81 by a look for infinities on
//           the FMA pipe and no clamp at 0; positions and slots fetched a turn ahead
//           change nothing.
//   read    100000 rows to bf16, 525 MB in and out: 101 us, 5.2 TB/s (a copy 6.8).
//           Issue slots 65 %, integer pipe 62 %, DRAM 56 %; half of a warp's time is
//           waiting for words.  111 us where a warp took a row of eight heads after the
//           other; 108 with a 64-bit division a step and codes shifted and converted
//           one by one (issue slots 67 %, DRAM 52 %); 119 where 40 registers left six
//           blocks of the eight of a grid resident.
// A few rows are launch-bound: 3 us (300 rows to fp32).
#include <cuda_fp16.h>

#include <cstdint>

#include "attn_batch.h"
#include "kv4.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer, half to even

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Eight elements as they lie in memory, and as floats.
template <bool BF16>
struct Raw8 {
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void *p, int64_t i) {
    const uint4 *b = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) + i * (BF16 ? 2 : 4));
#pragma unroll
    for (int k = 0; k < (BF16 ? 1 : 2); ++k) w[k] = __ldg(b + k);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < (BF16 ? 1 : 2); ++k) w[k] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float *x) const {
    if constexpr (BF16) {
      const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(v[k] << 16);
        x[2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        x[4 * k] = __uint_as_float(w[k].x);
        x[4 * k + 1] = __uint_as_float(w[k].y);
        x[4 * k + 2] = __uint_as_float(w[k].z);
        x[4 * k + 3] = __uint_as_float(w[k].w);
      }
    }
  }
};

__device__ __forceinline__ void store8(void *p, int64_t i, const float *x, bool bf16) {
  if (bf16) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  } else {
    float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// The rule above for a group of which four lanes hold N values each (n of them
// count): this lane's codes, eight to a word, and the group's parameters.
template <int N>
__device__ __forceinline__ uint32_t quantise(const float *x, int n, uint32_t *words) {
  float lo = INFINITY, hi = -INFINITY;
  float zero = 0.0f;  // until something is not finite
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i < n) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
      zero = fmaf(x[i], 0.0f, zero);
    }
  }
  bool bad = zero != 0.0f;
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
  }
  bad = __ballot_sync(0xFFFFFFFFu, bad) >> (threadIdx.x & 28) & 15u;
  const float top = fmaxf(fabsf(lo), fabsf(hi));
  float s = __fmul_rn(__fsub_rn(__fmul_rn(hi, 0.0625f), __fmul_rn(lo, 0.0625f)), 16.0f / 15.0f);
  s = fmaxf(fmaxf(s, __fmul_rn(top, 0x1p-11f)), 0x1p-100f);
  const uint32_t sb = (__float_as_uint(s) + 0xFFFFu) & 0xFFFF0000u;
  const float inv = __frcp_rn(__uint_as_float(sb));
  // rint(v / s) as an integer: the sum's bits less the magic number's.  No code of a
  // finite group is below 0: every step grows with v, and lo gives 0.
  const int z = __float_as_int(kMagic) - __float_as_int(__fadd_rn(__fmul_rn(lo, inv), kMagic));
#pragma unroll
  for (int w = 0; w < N / 8; ++w) {
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = __float_as_int(__fadd_rn(__fmul_rn(x[8 * w + j], inv), kMagic)) + (z - __float_as_int(kMagic));
      v += static_cast<uint32_t>(min(c, 15)) << (4 * j);
    }
    words[w] = bad || 8 * w >= n ? 0u : v;
  }
  if (bad) return 0x7FC00000u;
  return sb | __half_as_ushort(__int2half_rn(z));
}

template <int NC>
__device__ __forceinline__ void store_words(uint32_t *p, const uint32_t *w) {
  if constexpr (NC % 4 == 0) {
#pragma unroll
    for (int c = 0; c < NC; c += 4) *reinterpret_cast<uint4 *>(p + c) = make_uint4(w[c], w[c + 1], w[c + 2], w[c + 3]);
  } else if constexpr (NC % 2 == 0) {
#pragma unroll
    for (int c = 0; c < NC; c += 2) *reinterpret_cast<uint2 *>(p + c) = make_uint2(w[c], w[c + 1]);
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) p[c] = w[c];
  }
}

template <int NC>
__device__ __forceinline__ void load_words(uint32_t *w, const uint32_t *p) {
  if constexpr (NC % 4 == 0) {
#pragma unroll
    for (int c = 0; c < NC; c += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p + c));
      w[c] = v.x, w[c + 1] = v.y, w[c + 2] = v.z, w[c + 3] = v.w;
    }
  } else if constexpr (NC % 2 == 0) {
#pragma unroll
    for (int c = 0; c < NC; c += 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p + c));
      w[c] = v.x, w[c + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) w[c] = __ldg(p + c);
  }
}

// CPG: chunks of a group.
template <int NC, int CPG, bool BF16>
__global__ void __launch_bounds__(kThreads, NC <= 4 ? 4 : 2) rope_append_kv4_kernel(RopeAppend a, Kv4 cache, uint32_t *status) {
  constexpr int G = (NC + CPG - 1) / CPG;
  pdl_enter();
  const int lane = threadIdx.x & 31, t4 = lane & 3, team = lane >> 2;
  const int heads = a.n_head + 2 * a.n_kv, turned = a.n_head + a.n_kv, hd = a.head_dim;
  const int64_t rows = cache.num_blocks << cache.block_shift;
  const int strip = kv4_strip(cache);
  // (two tokens, four heads) by turns: a few tokens still spread over many warps
  const int quads = (heads + 3) / 4, odd = team & 1;
  const int64_t pairs = (a.T + 1) / 2, step = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t dt = step / quads;
  const int dp = static_cast<int>(step - dt * quads);
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  int64_t pair = item / quads;
  int part = static_cast<int>(item - pair * quads);
  for (; pair < pairs; pair += dt, part += dp) {
    if (part >= quads) {
      part -= quads;
      if (++pair >= pairs) break;
    }
    const int64_t t = 2 * pair + odd;
    const int64_t p = t < a.T ? a.positions[t] : -1, slot = t < a.T ? a.slots[t] : -1;
    // a padding row (position below 0) or one the table does not reach: zeros, no cache row
    const bool live = p >= 0 && p < a.max_seq;
    const bool put = live && slot >= 0 && slot < rows;
    if (lane - 4 * odd == 0 && part == 0) {
      if (p >= a.max_seq) atomicOr(status, kDevBadPosition);
      if (live && slot >= rows) atomicOr(status, kDevBadBlock);
    }
    {
      const int h = 4 * part + (team >> 1);
      const bool on = h < heads && t < a.T;
      Raw8<BF16> raw[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int d = 32 * c + 8 * t4;
        if (on && d < hd)
          raw[c].load(a.qkv, t * a.stride + static_cast<int64_t>(h) * hd + d);
        else
          raw[c].zero();
      }
      const bool query = h < a.n_head, key = !query && h < turned;
      const int hk = h - a.n_head - (key ? 0 : a.n_kv);
      void *const packed = query ? a.q : key ? a.k : a.v;
      const int64_t base = query ? (t * a.n_head + h) * hd : (t * a.n_kv + hk) * hd;
      // eight dimensions of chunk c, turned, and stored where they go out as numbers
      auto turn = [&](int c, float *y) {
        const int d = 32 * c + 8 * t4;
        raw[c].get(y);
        if (!on || d >= hd) return false;
        if (!live) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = 0.0f;
        } else if (h < turned) {
          const int64_t at = p * (hd / 2) + d / 2;
          const float4 cs = __ldg(reinterpret_cast<const float4 *>(a.cos_t + at));
          const float4 sn = __ldg(reinterpret_cast<const float4 *>(a.sin_t + at));
          const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = y[2 * i], o = y[2 * i + 1];
            y[2 * i] = fmaf(e, cc[i], -__fmul_rn(o, ss[i]));
            y[2 * i + 1] = fmaf(e, ss[i], __fmul_rn(o, cc[i]));
          }
        }
        if (packed) store8(packed, base + d, y, a.y_bf16);
        return true;
      };
      if (4 * part + 4 <= a.n_head || !__any_sync(0xFFFFFFFFu, put)) {  // nothing here is quantised
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float y[8];
          turn(c, y);
        }
        continue;
      }
      uint32_t words[G * CPG], params[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float x[8 * CPG];
        int n = 0;
#pragma unroll
        for (int k = 0; k < CPG; ++k) {
          const int c = g * CPG + k;
          if (c < NC) {
            if (turn(c < NC ? c : 0, x + 8 * k)) n = 8 * k + 8;
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[8 * k + i] = 0.0f;
          }
        }
        params[g] = quantise<8 * CPG>(x, n, words + g * CPG);
      }
      // Rows 2 j and 2 j + 1 share the words of values: where the pair's tokens go
      // there, each lane stores whole words of both.
      const int64_t other = __shfl_xor_sync(0xFFFFFFFFu, slot, 4);
      const bool both = __shfl_xor_sync(0xFFFFFFFFu, put, 4) && put && (slot ^ other) == 1;
      uint32_t theirs[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) theirs[c] = __shfl_xor_sync(0xFFFFFFFFu, words[c], 4);
      if (on && put && !query) {
        const int row = static_cast<int>(slot & ((1 << cache.block_shift) - 1)), r = row & 15;
        uint8_t *const s = cache.data + (slot >> cache.block_shift) * cache.block_stride + (row >> 4) * strip +
                           static_cast<int64_t>(hk) * kv4_head_bytes(cache);
        uint32_t *const v = reinterpret_cast<uint32_t *>(s + 256 * NC) +
                            (((r >> 3) * 8 + 2 * t4) * 4 + ((r & 7) >> 1)) * NC;
        if (key) {
          store_words<NC>(reinterpret_cast<uint32_t *>(s) + (r * 4 + t4) * NC, words);
        } else if (both) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
            words[c] = r & 1 ? __byte_perm(theirs[c], words[c], 0x7632u) : __byte_perm(words[c], theirs[c], 0x5410u);
          store_words<NC>(v + (r & 1) * 4 * NC, words);
        } else {
          uint16_t *const v16 = reinterpret_cast<uint16_t *>(v) + (r & 1);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            v16[2 * c] = static_cast<uint16_t>(words[c]);
            v16[2 * (4 * NC + c)] = static_cast<uint16_t>(words[c] >> 16);
          }
        }
        uint32_t *const q = reinterpret_cast<uint32_t *>(s + 512 * NC) + (key ? 0 : 16 * cache.ng) + r * cache.ng;
#pragma unroll
        for (int g = 0; g < G; ++g)
          if ((g & 3) == t4 && g < cache.ng) q[g] = params[g];
      }
    }
  }
}

template <int NC>
__global__ void __launch_bounds__(kThreads, NC <= 4 ? 8 : 4)
    kv4_read_kernel(Kv4 cache, const int64_t *slots, int64_t n, void *k, void *v, bool bf16, uint32_t *status) {
  pdl_enter();
  const int lane = threadIdx.x & 31, t4 = lane & 3, team = lane >> 2, hd = cache.head_dim, odd = team & 1;
  const int64_t rows = cache.num_blocks << cache.block_shift;
  const int strip = kv4_strip(cache);
  // A warp takes two rows of four heads, its CTA sixteen: neighbours share sectors.
  const unsigned quads = (2 * cache.n_kv + 3) / 4;
  const int64_t pairs = (n + 1) / 2;
  const unsigned di = gridDim.x / quads, dp = gridDim.x - di * quads;
  int64_t pair = static_cast<int64_t>(blockIdx.x / quads) * kWarps + (threadIdx.x >> 5);
  unsigned part = blockIdx.x % quads;
  for (; pair < pairs; pair += static_cast<int64_t>(di) * kWarps, part += dp) {
    if (part >= quads) {
      part -= quads;
      pair += kWarps;
      if (pair >= pairs) break;
    }
    const int64_t i = 2 * pair + odd;
    const int64_t slot = i < n ? slots[i] : -1;
    const bool live = slot >= 0 && slot < rows;
    if (lane - 4 * odd == 0 && part == 0 && slot >= rows) atomicOr(status, kDevBadBlock);
    const int64_t other = __shfl_xor_sync(0xFFFFFFFFu, slot, 4);
    const bool both = live && other < rows && (slot ^ other) == 1;
    const int h = 4 * part + (team >> 1);
    const bool key = h < cache.n_kv;
    const int hk = key ? h : h - cache.n_kv;
    void *const out = key ? k : v;
    const bool on = h < 2 * cache.n_kv && i < n && out;
    const int row = static_cast<int>(slot & ((1 << cache.block_shift) - 1)), r = row & 15;
    const uint8_t *const s = cache.data + (slot >> cache.block_shift) * cache.block_stride + (row >> 4) * strip +
                             static_cast<int64_t>(hk) * kv4_head_bytes(cache);
    uint32_t w[NC], par[NC], hi[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) w[c] = par[c] = hi[c] = 0u;
    if (live && on) {
      const uint32_t *const q =
          reinterpret_cast<const uint32_t *>(s + 512 * NC) + (key ? 0 : 16 * cache.ng) + r * cache.ng;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        par[c] = c % 2 && cache.cpg == 2 ? par[c - c % 2] : __ldg(q + min(c / cache.cpg, cache.ng - 1));
      if (key) {
        load_words<NC>(w, reinterpret_cast<const uint32_t *>(s) + (r * 4 + t4) * NC);
      } else {
        // words of two rows, of which this one has one half
        const uint32_t *const vw =
            reinterpret_cast<const uint32_t *>(s + 256 * NC) + (((r >> 3) * 8 + 2 * t4) * 4 + ((r & 7) >> 1)) * NC;
        load_words<NC>(w, vw + (both ? (r & 1) * 4 * NC : 0));
        if (!both) load_words<NC>(hi, vw + 4 * NC);
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const uint32_t theirs = __shfl_xor_sync(0xFFFFFFFFu, w[c], 4);
      if (!key) {
        const uint32_t lo = both && (r & 1) ? theirs : w[c], up = !both ? hi[c] : r & 1 ? w[c] : theirs;
        w[c] = __byte_perm(lo, up, r & 1 ? 0x7632u : 0x5410u);
      }
    }
    if (!on) continue;
    const int64_t base = (i * cache.n_kv + hk) * hd;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = 32 * c + 8 * t4;
      if (d >= hd) continue;
      const float scale = __uint_as_float(par[c] & 0xFFFF0000u);
      const float zp = __half2float(__ushort_as_half(static_cast<unsigned short>(par[c])));
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // the code where it is, as low bits of 2^23: code 16^(j % 4), exact, and with
        // the zero point taken off rounded once
        const uint32_t half = j < 4 ? w[c] : w[c] >> 16;
        const float at = __uint_as_float((half & 15u << 4 * (j % 4)) | 0x4B000000u) - 8388608.0f;
        y[j] = fmaf(at, 1.0f / (1 << 4 * (j % 4)), -zp) * scale;
      }
      store8(out, base + d, y, bf16);
    }
  }
}

unsigned grid_of(int64_t rows, int per_sm) {
  const int64_t most = static_cast<int64_t>(sm_count()) * per_sm, want = (rows + kWarps - 1) / kWarps;
  return static_cast<unsigned>(want < most ? want : most);
}

template <int NC, int CPG>
cudaError_t run_append(const RopeAppend &a, const Kv4 &c, uint32_t *status, cudaStream_t s) {
  auto kern = a.x_bf16 ? rope_append_kv4_kernel<NC, CPG, true> : rope_append_kv4_kernel<NC, CPG, false>;
  return launch_pdl(kern, dim3(grid_of((a.T + 1) / 2 * ((a.n_head + 2 * a.n_kv + 3) / 4), 4)), dim3(kThreads), 0, s, a, c, status);
}

template <int NC>
cudaError_t run_append_nc(const RopeAppend &a, const Kv4 &c, uint32_t *status, cudaStream_t s) {
  if constexpr (NC > 1)
    if (c.cpg == 2) return run_append<NC, 2>(a, c, status, s);
  return run_append<NC, 1>(a, c, status, s);
}

}  // namespace

cudaError_t launch_rope_append_kv4(const RopeAppend &a, const Kv4 &c, cudaStream_t s) {
  uint32_t *status = device_status();
  if (!status) return cudaErrorInvalidDevice;
  switch (c.nc) {
    case 1: return run_append_nc<1>(a, c, status, s);
    case 2: return run_append_nc<2>(a, c, status, s);
    case 3: return run_append_nc<3>(a, c, status, s);
    case 4: return run_append_nc<4>(a, c, status, s);
    case 6: return run_append_nc<6>(a, c, status, s);
    default: return run_append_nc<8>(a, c, status, s);
  }
}

cudaError_t launch_kv4_read(const Kv4 &c, const int64_t *slots, int64_t n, void *k, void *v, bool bf16,
                            cudaStream_t s) {
  uint32_t *status = device_status();
  if (!status) return cudaErrorInvalidDevice;
  auto kern = c.nc == 1   ? kv4_read_kernel<1>
              : c.nc == 2 ? kv4_read_kernel<2>
              : c.nc == 3 ? kv4_read_kernel<3>
              : c.nc == 4 ? kv4_read_kernel<4>
              : c.nc == 6 ? kv4_read_kernel<6>
                          : kv4_read_kernel<8>;
  return launch_pdl(kern, dim3(grid_of((n + 15) / 16 * kWarps * ((2 * c.n_kv + 3) / 4), c.nc <= 4 ? 8 : 4)), dim3(kThreads), 0, s, c, slots, n, k, v, bf16,
                    status);
}

}  // namespace qmm
