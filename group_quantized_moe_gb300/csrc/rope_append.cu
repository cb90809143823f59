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
// one load of cos and sin serves all of them, and its loads are 16 bytes
// wide and all in flight before the first use.
#include <cstdint>

#include "attn_batch.h"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;

template <int V, bool BF16>
__device__ __forceinline__ void load_unit(const void *p, int64_t i, float (&x)[V]) {
#pragma unroll
  for (int k = 0; k < V; k += 4) {
    if constexpr (BF16 && V == 8) {
      if (k == 0) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[2 * j] = __uint_as_float(w[j] << 16);
          x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      }
    } else {
      const float4 v = load_x4<BF16>(p, i + k);
      x[k] = v.x;
      x[k + 1] = v.y;
      x[k + 2] = v.z;
      x[k + 3] = v.w;
    }
  }
}

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
__global__ void __launch_bounds__(kThreads) rope_append_kernel(RopeAppend a, uint32_t *status) {
  pdl_enter();
  const int units = a.head_dim / V, J = blockDim.x / units;
  const int u = threadIdx.x % units, j0 = threadIdx.x / units;
  const int heads = a.n_head + 2 * a.n_kv;
  const int64_t rows = a.num_blocks << a.block_shift;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t p = a.positions[t], slot = a.slots ? a.slots[t] : -1;
    // a padding row (position below 0) or one the table does not reach: zeros, no cache row
    const bool live = p >= 0 && p < a.max_seq;
    const bool put = live && a.k_cache && slot >= 0 && slot < rows;
    if (threadIdx.x == 0) {
      if (p >= a.max_seq) atomicOr(status, kDevBadPosition);
      if (a.k_cache && live && slot >= rows) atomicOr(status, kDevBadBlock);
    }
    float c[V / 2], s[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const int64_t o = p * (a.head_dim / 2) + u * (V / 2) + i;
      c[i] = live ? __ldg(a.cos_t + o) : 0.0f;
      s[i] = live ? __ldg(a.sin_t + o) : 0.0f;
    }
    const int64_t block = put ? slot >> a.block_shift : 0;
    const int row = put ? static_cast<int>(slot & ((1 << a.block_shift) - 1)) : 0;
    for (int h0 = j0; h0 < heads; h0 += 4 * J) {
      float x[4][V];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int h = h0 + k * J;
        if (h < heads && live)
          load_unit<V, BF16>(a.qkv, t * a.stride + static_cast<int64_t>(h) * a.head_dim + u * V, x[k]);
        else
#pragma unroll
          for (int i = 0; i < V; ++i) x[k][i] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int h = h0 + k * J;
        if (h >= heads) break;
        if (h < a.n_head + a.n_kv) {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const float e = x[k][2 * i], o = x[k][2 * i + 1];
            if (live) {
              x[k][2 * i] = fmaf(e, c[i], -o * s[i]);
              x[k][2 * i + 1] = fmaf(e, s[i], o * c[i]);
            }
          }
        }
        if (h < a.n_head) {
          store_unit<V>(a.q, (t * a.n_head + h) * a.head_dim + u * V, x[k], a.y_bf16);
          continue;
        }
        const bool key = h < a.n_head + a.n_kv;
        const int hk = h - a.n_head - (key ? 0 : a.n_kv);
        void *packed = key ? a.k : a.v;
        if (packed)
          store_unit<V>(packed, (t * a.n_kv + hk) * a.head_dim + u * V, x[k], a.y_bf16);
        if (put)
          store_unit<V>(key ? a.k_cache : a.v_cache,
                        block * a.block_stride +
                            ((static_cast<int64_t>(hk) << a.block_shift) + row) * a.head_dim + u * V,
                        x[k], a.y_bf16);
      }
    }
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
  const int64_t most = static_cast<int64_t>(sm_count()) * 64;
  if (blocks > most) blocks = most;
  auto kern = wide ? (a.x_bf16 ? rope_append_kernel<8, true> : rope_append_kernel<8, false>)
                   : (a.x_bf16 ? rope_append_kernel<4, true> : rope_append_kernel<4, false>);
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, s, a, status);
}

}  // namespace qmm
