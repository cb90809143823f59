// rope_append.cu -- rotary positions of a batch of tokens, and their keys and
// values into the paged cache.
//
// Row t of qkv holds the n_head query, n_kv key and n_kv value heads of a
// token at position p = positions[t]; every pair (2i, 2i + 1) of a query or
// key head turns by the angle whose cos and sin stand in row p of the table:
//   (a, b) -> (a c - b s, a s + b c)
// in fp32, each product sum formed with one fma, and rounded once to the
// output type.  The rotated queries go to q; the rotated keys and the values
// go to row slots[t] of the cache and, where asked, packed to k and v.
//
// The work is bound by HBM: every element is read once and written once.
// One CTA per token and pass: thread (u, j) holds column unit u (8 elements,
// or 4 where head_dim is no multiple of 8) of the heads j, j + J, ..., so that
// one load of cos and sin serves all of them.  Its loads are 16 bytes wide,
// wait for nothing (the position is only needed to use them, and the next
// token's is read ahead) and are held as they come until they are used, so
// that many threads fit an SM.
#include <cstdint>

#include "attn_batch.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;
// Resident CTAs per SM, each over many tokens (16384 tokens of 48 heads of 128, bf16,
// three heads in flight a thread: 74 us, 6.4 TB/s; one or two heads in flight 83 to 90).
// Five leave a thread 48 registers, and up to 31 words of it are spilled and read again from
// L1; with four CTAs almost nothing is, and the same call takes 83 us (fp32 rows into a bf16
// cache, which spill most: 104 us with five, 96 with four).
constexpr int kPerSm = 5;

// V elements as they lie in memory, and as floats.
template <int V, bool BF16>
struct Raw {
  static constexpr int n = V * (BF16 ? 2 : 4) / 8;  // 8-byte words
  uint2 w[n];
  __device__ __forceinline__ void load(const void *p, int64_t i) {
    const uint8_t *b = static_cast<const uint8_t *>(p) + i * (BF16 ? 2 : 4);
    if constexpr (n == 1) {
      w[0] = __ldg(reinterpret_cast<const uint2 *>(b));
    } else {
#pragma unroll
      for (int k = 0; k < n; k += 2) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(b) + k / 2);
        w[k] = make_uint2(v.x, v.y);
        w[k + 1] = make_uint2(v.z, v.w);
      }
    }
  }
  __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
    for (int k = 0; k < n; ++k) {
      if constexpr (BF16) {
        x[4 * k] = __uint_as_float(w[k].x << 16);
        x[4 * k + 1] = __uint_as_float(w[k].x & 0xFFFF0000u);
        x[4 * k + 2] = __uint_as_float(w[k].y << 16);
        x[4 * k + 3] = __uint_as_float(w[k].y & 0xFFFF0000u);
      } else {
        x[2 * k] = __uint_as_float(w[k].x);
        x[2 * k + 1] = __uint_as_float(w[k].y);
      }
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

template <int V>
__device__ __forceinline__ void store_unit(void *p, int64_t i, const float (&x)[V], bool bf16) {
  if (bf16) {
    uint16_t *d = static_cast<uint16_t *>(p) + i;
    if constexpr (V == 8)
      *reinterpret_cast<uint4 *>(d) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                 pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    else
      *reinterpret_cast<uint2 *>(d) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  } else {
    float *d = static_cast<float *>(p) + i;
#pragma unroll
    for (int k = 0; k < V; k += 4)
      *reinterpret_cast<float4 *>(d + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
  }
}

template <int V, bool BF16>
__global__ void __launch_bounds__(kThreads, kPerSm) rope_append_kernel(RopeAppend a, uint32_t *status) {
  constexpr int H = 3;  // heads of a thread at a time
  pdl_enter();
  const int units = a.head_dim / V, J = blockDim.x / units;
  const int u = threadIdx.x % units, j0 = threadIdx.x / units;
  const int heads = a.n_head + 2 * a.n_kv, turned = a.n_head + a.n_kv;
  const int64_t rows = a.num_blocks << a.block_shift;
  int64_t t = blockIdx.x;
  int64_t p = t < a.T ? a.positions[t] : -1, slot = t < a.T && a.slots ? a.slots[t] : -1;
  for (; t < a.T; t += gridDim.x) {
    const int64_t next = t + gridDim.x;
    const int64_t p_next = next < a.T ? a.positions[next] : -1;
    const int64_t slot_next = next < a.T && a.slots ? a.slots[next] : -1;
    // a padding row (position below 0) or one the table does not reach: zeros, no cache row
    const bool live = p >= 0 && p < a.max_seq;
    const bool put = live && a.cached && slot >= 0 && slot < rows;
    if (threadIdx.x == 0) {
      if (p >= a.max_seq) atomicOr(status, kDevBadPosition);
      if (a.cached && live && slot >= rows) atomicOr(status, kDevBadBlock);
    }
    float c[V / 2], s[V / 2];
    const int64_t at = live ? p * (a.head_dim / 2) + u * (V / 2) : 0;
#pragma unroll
    for (int i = 0; i < V / 2; i += 2) {
      const float2 cc = live ? __ldg(reinterpret_cast<const float2 *>(a.cos_t + at + i)) : make_float2(0.f, 0.f);
      const float2 ss = live ? __ldg(reinterpret_cast<const float2 *>(a.sin_t + at + i)) : make_float2(0.f, 0.f);
      c[i] = cc.x;
      c[i + 1] = cc.y;
      s[i] = ss.x;
      s[i + 1] = ss.y;
    }
    const int64_t row0 = put ? ((slot >> a.block_shift) * a.block_stride +
                                (slot & ((1 << a.block_shift) - 1)) * a.head_dim)
                             : 0;
    for (int h0 = j0; h0 < heads; h0 += H * J) {
      Raw<V, BF16> raw[H];
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const int h = min(h0 + k * J, heads - 1);
        raw[k].load(a.qkv, t * a.stride + static_cast<int64_t>(h) * a.head_dim + u * V);
      }
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const int h = h0 + k * J;
        if (h >= heads) break;
        float x[V];
        raw[k].get(x);
        if (h < turned) {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const float e = x[2 * i], o = x[2 * i + 1];
            x[2 * i] = fmaf(e, c[i], -o * s[i]);
            x[2 * i + 1] = fmaf(e, s[i], o * c[i]);
          }
        }
        if (!live)
#pragma unroll
          for (int i = 0; i < V; ++i) x[i] = 0.0f;
        if (h < a.n_head) {
          store_unit<V>(a.q, (t * a.n_head + h) * a.head_dim + u * V, x, a.y_bf16);
          continue;
        }
        const bool key = h < turned;
        const int hk = h - a.n_head - (key ? 0 : a.n_kv);
        void *packed = key ? a.k : a.v;
        if (packed) store_unit<V>(packed, (t * a.n_kv + hk) * a.head_dim + u * V, x, a.y_bf16);
        if (put)
          store_unit<V>(key ? a.k_cache : a.v_cache,
                        row0 + (static_cast<int64_t>(hk) << a.block_shift) * a.head_dim + u * V, x,
                        a.y_bf16);
      }
    }
    p = p_next;
    slot = slot_next;
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppend &a, cudaStream_t s) {
  uint32_t *status = device_status();
  if (!status) return cudaErrorInvalidDevice;
  // 16-byte bf16 units need rows and blocks that keep their alignment
  const bool wide = a.head_dim % 8 == 0 && a.stride % 8 == 0 && a.block_stride % 8 == 0;
  const int units = a.head_dim / (wide ? 8 : 4);
  const int threads = units >= kThreads ? units : units * (kThreads / units);
  int64_t blocks = a.T;
  const int64_t most = static_cast<int64_t>(sm_count()) * kPerSm;
  if (blocks > most) blocks = most;
  auto kern = wide ? (a.x_bf16 ? rope_append_kernel<8, true> : rope_append_kernel<8, false>)
                   : (a.x_bf16 ? rope_append_kernel<4, true> : rope_append_kernel<4, false>);
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, s, a, status);
}

}  // namespace qmm
