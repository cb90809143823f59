// attn_tile.cu -- batched attention for many query rows in fp32 (head sizes up
// to 128): prompts and chunks, on the CUDA cores' fused multiply-adds.
//
// A unit has 128 query rows (tokens times the query heads that share the
// key/value head) against 32-key tiles, copied to shared memory two stages
// ahead of their use (cp.async).  256 threads; a warp owns 16 rows and sees
// every key, so the weights P go from the lanes that form them to the lanes
// that use them inside the warp, and the only block-wide barriers are the two
// that hand the stages over.  Lane (y, x), y < 4, x < 8: scores of rows
// 4 p + y and keys x + 8 k (4 x 4), results of those rows in columns
// 4 x + 32 j.  A load from shared memory costs the SM a cycle per 4 bytes a
// lane, whoever shares them, and four multiply-adds a lane take one: with 4 x 4
// scores a lane Q K^T reads 8 floats for 16 multiply-adds, which bounds it at
// half the FMA rate (measured 38 TFLOP/s at 4096 tokens, 48% of the FMA pipe;
// three prompts, 1500 tokens together, 32 heads of 128, 263 us or 25 TFLOP/s; 8 x 4 and
// 8 x 8 scores a lane, which spill, gain nothing).
// Multiply-adds are issued in pairs (f32x2), 8% on short prompts.  A warp skips
// the tiles that none of its rows sees.
#include <cstdint>

#include "attn_batch.h"
#include "attn_internal.h"
#include "attn_sched.cuh"
#include "qmm_device.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 128;
constexpr int kKeys = 32;
constexpr int kPld = 40;  // floats of a row of P: four rows 8 banks apart

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 16 bytes global -> shared, or zeros.
__device__ __forceinline__ void copy16(float *dst, const float *src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}

template <int NC>  // 64-column groups of the head size
struct Tile {
  static constexpr int W = NC * 64, LD = W + 4;  // rows of Q and K 4 banks apart
  static constexpr int stage = kKeys * LD + kKeys * W;
  static constexpr int smem = (kRows * LD + 2 * stage + 8 * 16 * kPld) * 4;
  // two CTAs of 128 registers a thread spill ten words of them: three prompts of 500
  // tokens, 32 heads over 8 of 64 columns, 115 us; 130 us with one that spills none
  static constexpr int per_sm = NC == 1 ? 2 : 1;
};

template <int NC>
__global__ void __launch_bounds__(kThreads, Tile<NC>::per_sm)
    attn_tile_kernel(AttnBatch a, AttnSched sc, int gsub, int nsub, AttnParts parts,
                     uint32_t *status) {
  using C = Tile<NC>;
  constexpr int LD = C::LD, W = C::W, NJ = W / 32;
  extern __shared__ __align__(16) float sm[];
  __shared__ int64_t scratch[kThreads / 32 + 4];
  __shared__ int bad[3];  // keys of tile kt in blocks outside the cache, one bit each, in kt % 3
  float *Qs = sm, *stages = sm + kRows * LD;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, x8 = lane & 7, y4 = lane >> 3;
  float *Pw = stages + 2 * C::stage + warp * 16 * kPld;
  const int hd = a.head_dim, d4 = hd / 4, grp = a.n_head / a.n_kv;
  const float *gk = static_cast<const float *>(a.k), *gv = static_cast<const float *>(a.v);
  pdl_enter();
  const AttnRun run = sched_run<kThreads>(sc, blockIdx.x, scratch);
  if (tid == 0) parts.open[blockIdx.x].rows_tok = 0;
  const float sl2 = a.scale * 1.4426950408889634f;
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
    if (tid == 0 && sched_short(sc, q, i)) atomicOr(status, kDevBadBlock);
    // Copies tile kt into stage kt & 1: eight threads a key.
    const int ck = tid >> 3;  // this thread's key
    auto fetch = [&](int kt) {
      const int st = kt & 1, k = kt * kKeys + ck;
      float *ks = stages + st * C::stage, *vs = ks + kKeys * LD;
      int64_t kp = 0, vp = 0;
      bool real = k < end;
      if (a.block_table) {
        if (real) {
          const int b = k / a.block_size;
          const int32_t id = a.block_table[r * a.table_stride + b];
          real = id >= 0 && id < a.num_blocks;
          if (real)
            kp = vp = id * a.block_stride +
                      static_cast<int64_t>(h * a.block_size + k - b * a.block_size) * hd;
          else
            atomicOr(status, kDevBadBlock);
        }
      } else if (real) {
        kp = (static_cast<int64_t>(q.q0) + k) * a.k_stride + static_cast<int64_t>(h) * hd;
        vp = (static_cast<int64_t>(q.q0) + k) * a.v_stride + static_cast<int64_t>(h) * hd;
      }
      const uint32_t none = __ballot_sync(0xFFFFFFFFu, !real && k < end && (tid & 7) == 0);
      if (lane == 0 && none) {  // lanes 0, 8, 16, 24: keys 4 warp ..
        uint32_t m = 0;
        for (int j = 0; j < 4; ++j) m |= (none >> (8 * j) & 1u) << j;
        atomicOr(&bad[kt % 3], static_cast<int>(m << (4 * warp)));
      }
#pragma unroll
      for (int c = tid & 7; c < W / 4; c += 8) {
        const bool in = real && c < d4;
        copy16(ks + ck * LD + 4 * c, gk + (in ? kp + 4 * c : 0), in);
        copy16(vs + ck * W + 4 * c, gv + (in ? vp + 4 * c : 0), in);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncthreads();  // the previous unit is done with all of shared memory
    if (tid < 3) bad[tid] = 0;
    __syncthreads();
    fetch(tile);
    // eight loads in flight a thread: one after another they cost 0.6 us each
#pragma unroll 1
    for (int e0 = tid; e0 < kRows * (W / 4); e0 += 8 * kThreads) {
      float4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = e0 + j * kThreads, row = e / (W / 4), c = e - row * (W / 4);
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < rows && c < d4) {
          const int t = row / g, hq = row - t * g;
          v[j] = load_x4<false>(a.q, static_cast<int64_t>(q.q0 + t0 + t) * a.q_stride +
                                         static_cast<int64_t>(head0 + hq) * hd + 4 * c);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = e0 + j * kThreads, row = e / (W / 4), c = e - row * (W / 4);
        *reinterpret_cast<float4 *>(Qs + row * LD + 4 * c) = make_float4(
            v[j].x * sl2, v[j].y * sl2, v[j].z * sl2, v[j].w * sl2);  // scores in log2 units
      }
    }
    // this lane's rows 16 warp + 4 p + y4: keys they see, running maximum and sum, results
    int vis[4];
    float m[4], l[4];
    ulonglong2 o[4][NJ];  // four columns as two packed pairs
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int row = 16 * warp + 4 * p + y4;
      vis[p] = row < rows ? min(all + row / g, end) : 0;
      m[p] = -INFINITY;
      l[p] = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) o[p][j] = make_ulonglong2(0ull, 0ull);
    }
    const int first_row = 16 * warp, last_row = min(rows, first_row + 16) - 1;
    // keys any row of the warp sees, and every row
    const int most = last_row >= first_row ? min(all + last_row / g, end) : 0;
    const int least = last_row == first_row + 15 ? min(all + first_row / g, end) : 0;
    for (int kt = tile; kt < stop; ++kt) {
      const int st = kt & 1, k0 = kt * kKeys;
      if (kt + 1 < stop) {
        fetch(kt + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();
      if (k0 < most) {
        const float *Ks = stages + st * C::stage, *Vs = Ks + kKeys * LD;
        const float *Qw = Qs + (16 * warp + y4) * LD;
        f32x2 s2[4][4];
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int k = 0; k < 4; ++k) s2[p][k] = 0ull;
#pragma unroll 4
        for (int c = 0; c < W / 4; ++c) {
          ulonglong2 kk[4], qq[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            kk[k] = *reinterpret_cast<const ulonglong2 *>(Ks + (x8 + 8 * k) * LD + 4 * c);
#pragma unroll
          for (int p = 0; p < 4; ++p) qq[p] = *reinterpret_cast<const ulonglong2 *>(Qw + 4 * p * LD + 4 * c);
#pragma unroll
          for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              s2[p][k] = fma2(qq[p].x, kk[k].x, s2[p][k]);
              s2[p][k] = fma2(qq[p].y, kk[k].y, s2[p][k]);
            }
        }
        float s[4][4];
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float lo, hi;
            unpack2(s2[p][k], lo, hi);
            s[p][k] = lo + hi;
          }
        const uint32_t gone = static_cast<uint32_t>(bad[kt % 3]);
        const bool guard = k0 + kKeys > least || gone;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          if (guard) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = x8 + 8 * k;
              if (k0 + j >= vis[p] || (gone >> j & 1u)) s[p][k] = -INFINITY;
            }
          }
          float top = fmaxf(fmaxf(s[p][0], s[p][1]), fmaxf(s[p][2], s[p][3]));
#pragma unroll
          for (int w = 4; w >= 1; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, w));
          const float mn = fmaxf(m[p], top);
          const float ref = mn == -INFINITY ? 0.0f : mn;
          const float f = ex2(m[p] - ref);
          float sum = 0.0f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float e = s[p][k] == -INFINITY ? unseen_weight() : ex2(s[p][k] - ref);
            sum += e;
            Pw[(4 * p + y4) * kPld + x8 + 8 * k] = e;
          }
          l[p] = fmaf(l[p], f, sum);  // this lane's keys; summed over the lanes at the end
          m[p] = mn;
          if (__any_sync(0xFFFFFFFFu, f != 1.0f)) {
            const f32x2 f2 = pack2(f, f);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              o[p][j].x = mul2(o[p][j].x, f2);
              o[p][j].y = mul2(o[p][j].y, f2);
            }
          }
        }
        __syncwarp();
        auto add = [&](float w, const ulonglong2 &v, ulonglong2 &t) {
          const f32x2 w2 = pack2(w, w);
          t.x = fma2(w2, v.x, t.x);
          t.y = fma2(w2, v.y, t.y);
        };
        // Where some row misses some key, P is a zero there, which a non-finite
        // value would still turn into NaN: then (and only then) key by key.
        bool plain = true;
        if (guard) {
          float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int c = lane; c < kKeys * W / 4; c += 32) {
            const float4 v = *reinterpret_cast<const float4 *>(Vs + 4 * c);
            z.x = fmaf(v.x, 0.0f, z.x);
            z.y = fmaf(v.y, 0.0f, z.y);
            z.z = fmaf(v.z, 0.0f, z.z);
            z.w = fmaf(v.w, 0.0f, z.w);
          }
          plain = __all_sync(0xFFFFFFFFu, z.x + z.y + z.z + z.w == 0.0f);
        }
        if (plain) {
#pragma unroll 2
          for (int k = 0; k < kKeys; k += 4) {
            float4 w[4];
#pragma unroll
            for (int p = 0; p < 4; ++p)
              w[p] = *reinterpret_cast<const float4 *>(Pw + (4 * p + y4) * kPld + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int j = 0; j < NJ; ++j) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(Vs + (k + kk) * W + 32 * j + 4 * x8);
#pragma unroll
                for (int p = 0; p < 4; ++p)
                  add(kk == 0 ? w[p].x : kk == 1 ? w[p].y : kk == 2 ? w[p].z : w[p].w, v, o[p][j]);
              }
          }
        } else {
          const int nk = min(kKeys, most - k0);
#pragma unroll 1
          for (int k = 0; k < nk; ++k) {
            float w[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) w[p] = Pw[(4 * p + y4) * kPld + k];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(Vs + k * W + 32 * j + 4 * x8);
#pragma unroll
              for (int p = 0; p < 4; ++p)
                if (!is_unseen(w[p])) add(w[p], v, o[p][j]);
            }
          }
        }
        __syncwarp();
      }
      // last read a barrier ago, next written a barrier from here
      if (tid == 0) bad[(kt + 2) % 3] = 0;
      __syncthreads();
    }
    const bool whole = tile == 0 && stop == ntile;
    const int slot = 2 * blockIdx.x + (tile == 0 ? 1 : 0);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
#pragma unroll
      for (int w = 4; w >= 1; w >>= 1) l[p] += __shfl_xor_sync(0xFFFFFFFFu, l[p], w);
      const int row = 16 * warp + 4 * p + y4;
      if (row >= rows) continue;
      const int t = row / g, hq = row - t * g;
      const float inv = whole ? (l[p] > 0.0f || l[p] != l[p] ? 1.0f / l[p] : 0.0f) : 1.0f;
      const int64_t y0 = (static_cast<int64_t>(q.q0 + t0 + t) * a.n_head + head0 + hq) * hd;
      const int64_t base = static_cast<int64_t>(slot) * parts.rows + row;
      if (!whole && x8 == 0) parts.ml[base] = make_float2(m[p], l[p]);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int d = 32 * j + 4 * x8;
        if (d >= hd) continue;
        float4 v;
        unpack2(o[p][j].x, v.x, v.y);
        unpack2(o[p][j].y, v.z, v.w);
        v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        if (whole)
          store_y4(a.y, y0 + d, v, a.y_bf16);
        else
          *reinterpret_cast<float4 *>(parts.o + base * hd + d) = v;
      }
    }
    if (tid == 0 && tile == 0 && !whole)
      parts.open[blockIdx.x] =
          AttnOpen{q.q0 + t0, nt, vh, sched_last(sc, run, x, ntile)};
  }
  zero_loose_rows(a, sc, blockIdx.x, gridDim.x, kThreads);
}

template <int NC>
cudaError_t run_tile(const AttnBatch &a, const AttnPlan &p, const AttnSched &sc,
                     const AttnParts &parts, cudaStream_t s) {
  auto kern = attn_tile_kernel<NC>;
  const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), Tile<NC>::smem);
  if (e != cudaSuccess) return e;
  uint32_t *status = device_status();
  if (!status) return cudaErrorInvalidDevice;
  return launch_pdl(kern, dim3(p.workers), dim3(kThreads), Tile<NC>::smem, s, a, sc, p.gsub, p.nsub,
                    parts, status);
}

}  // namespace

// fp32, head sizes up to 128, with more query rows a request and key/value head
// than attn_rows_plan, which is asked first, takes: 8 on average of packed
// prompts, 32 over a paged cache (below, a 128-row unit would be mostly empty).
bool attn_tile_plan(bool bf16, int64_t T, int n_head, int n_kv, int head_dim, int R, AttnPlan *p) {
  const int grp = n_head / n_kv;
  if (bf16 || head_dim > 128) return false;
  p->rows = kRows;
  p->gsub = grp < kRows ? grp : kRows;
  p->nsub = (grp + p->gsub - 1) / p->gsub;
  p->U = kRows / p->gsub;
  p->KT = kKeys;
  // A tile takes 8 us, more than the join of a divided unit: runs may be short
  // (6 heads over one, 2 prompts of 300 tokens: 47 us; runs of four tiles 58).
  p->fixed = kKeys;
  p->min_run = kKeys;
  // a prompt of 200 tokens (32 heads over 8) divided 39 us, whole 54; four of 64
  // tokens 35 and 24
  p->whole = 128;
  p->workers = sm_count() * (head_dim <= 64 ? 2 : 1);
  return true;
}

cudaError_t launch_attn_tile(const AttnBatch &a, const AttnPlan &p, const AttnSched &sc,
                             const AttnParts &parts, cudaStream_t s) {
  return a.head_dim <= 64 ? run_tile<1>(a, p, sc, parts, s) : run_tile<2>(a, p, sc, parts, s);
}

}  // namespace qmm
