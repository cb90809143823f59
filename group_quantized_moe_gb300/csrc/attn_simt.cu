// attn_simt.cu -- batched causal attention (packed prompts, or new tokens over
// a paged cache) in fp32 on the CUDA cores, for the types and head sizes that
// the faster kernels leave (bf16 of any head size, fp32 of more than 128
// columns), and the merge of divided units.
//
//   s_j = scale q . k_j,  m = max_j s_j,  l = sum_j 2^((s_j - m) log2 e),
//   o = sum_j 2^((s_j - m) log2 e) v_j / l
// over the keys j that the token sees, in one pass over KT-key tiles with the
// running maximum and sum (o and l are rescaled when the maximum moves).
//
// A unit's query rows are the tokens of a block times the query heads that
// share the key/value head (up to TR rows), so that a key or value is read
// once for all of them.  256 threads as 16 x 16: thread (ty, tx) forms the
// scores of rows ty RP .. + RP - 1 and keys tx, tx + 16, ... and accumulates
// those rows' output columns 4 tx + 64 j.
//
// Bound by reading shared memory: each product of 4 x 4 scores (or rows by
// columns) takes eight 16-byte reads.  It serves what the faster kernels do
// not take; where attn_tile_kernel takes over (three fp32 prompts, 1500 tokens
// together, 32 heads of 128: 263 us), it needed 392 us, 17 TFLOP/s.  Prompts of
// three times 300 tokens, 8 heads of 256: 115 us (bf16), 107 us (fp32).  Single
// bf16 tokens, 64 query heads over one key/value head of 512 columns, 48 requests
// of 4096 keys: 1547 us, 0.26 TB/s of the cache, bound by the same reads.
#include <cstdint>

#include "attn_batch.h"
#include "attn_sched.cuh"
#include "qmm_device.cuh"
#include "qmm_internal.h"
#include "attn_internal.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// NC: 64-column groups of the head size; TR: query rows of a unit.
template <int NC, int TR>
struct Simt {
  static constexpr int KT = NC <= 2 ? 64 : (NC == 4 ? 32 : 16);
  static constexpr int LD = NC * 64 + 4;  // floats a row: rows 4 banks apart
  static constexpr int PLD = KT + 4;
  static constexpr int RP = TR / 16;
  static constexpr int smem = (TR * LD + KT * LD + KT * NC * 64 + TR * PLD) * 4 + KT * 8;
};

template <bool BF16, int NC, int TR>
__global__ void __launch_bounds__(kThreads) attn_simt_kernel(AttnBatch a, AttnSched sc, int gsub,
                                                             int nsub, AttnParts parts,
                                                             uint32_t *status) {
  using C = Simt<NC, TR>;
  constexpr int KT = C::KT, LD = C::LD, PLD = C::PLD, RP = C::RP, KP = KT / 16;
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm, *Ks = Qs + TR * LD, *Vs = Ks + KT * LD, *Ps = Vs + KT * NC * 64;
  int64_t *krow = reinterpret_cast<int64_t *>(Ps + TR * PLD);  // element offset of a key row, -1: none
  __shared__ int64_t scratch[kThreads / 32 + 4];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int hd = a.head_dim, d4 = hd / 4;
  const int grp = a.n_head / a.n_kv;
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
    const int g = min(gsub, grp - sub * gsub);  // query heads of this unit
    const int t0 = i * sc.U, nt = min(sc.U, q.n - t0);
    const int rows = nt * g, head0 = h * grp + sub * gsub;
    const int end = sched_end(sc, q, i);        // keys the last token sees
    const int all = sched_seen(sc, q, t0);      // keys the first token sees
    if (tid == 0 && sched_short(sc, q, i)) atomicOr(status, kDevBadBlock);
    __syncthreads();                            // the previous unit is done with Qs
    constexpr int QB = TR * NC / 16 < 8 ? TR * NC / 16 : 8;  // loads in flight a thread
#pragma unroll 1
    for (int e0 = tid; e0 < TR * NC * 16; e0 += QB * kThreads) {
      float4 v[QB];
#pragma unroll
      for (int j = 0; j < QB; ++j) {
        const int e = e0 + j * kThreads, row = e / (NC * 16), c = e - row * (NC * 16);
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < rows && c < d4) {
          const int t = row / g, hq = row - t * g;
          v[j] = load_x4<BF16>(a.q, static_cast<int64_t>(q.q0 + t0 + t) * a.q_stride +
                                        static_cast<int64_t>(head0 + hq) * hd + 4 * c);
        }
      }
#pragma unroll
      for (int j = 0; j < QB; ++j) {
        const int e = e0 + j * kThreads, row = e / (NC * 16), c = e - row * (NC * 16);
        *reinterpret_cast<float4 *>(Qs + row * LD + 4 * c) = v[j];
      }
    }
    float m[RP], l[RP];
    float4 o[RP][NC];
#pragma unroll
    for (int p = 0; p < RP; ++p) {
      m[p] = -INFINITY;
      l[p] = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) o[p][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int kt = tile; kt < stop; ++kt) {
      const int k0 = kt * KT, nk = min(KT, end - k0);  // keys of the tile any row sees
      bool bad = false;
      for (int k = tid; k < KT; k += kThreads) {
        int64_t off = -1;
        if (k < nk) {
          if (a.block_table) {
            const int j = k0 + k, b = j / a.block_size;
            const int32_t id = a.block_table[r * a.table_stride + b];
            if (id >= 0 && id < a.num_blocks)
              off = id * a.block_stride +
                    static_cast<int64_t>(h * a.block_size + j - b * a.block_size) * hd;
            else
              bad = true;
          } else {
            off = k0 + k;
          }
        }
        krow[k] = off;
      }
      // keys without a block, or that some row does not see: the guarded form
      const bool guard = __syncthreads_or(bad) || k0 + KT > all;
      if (bad) atomicOr(status, kDevBadBlock);
      constexpr int KB = KT * NC / 16 < 4 ? KT * NC / 16 : 4;  // keys and values in flight a thread
#pragma unroll 1
      for (int e0 = tid; e0 < KT * NC * 16; e0 += KB * kThreads) {
        float4 kv[KB], vv[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const int e = e0 + j * kThreads, k = e / (NC * 16), c = e - k * (NC * 16);
          const int64_t off = krow[k];
          kv[j] = vv[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (off >= 0 && c < d4) {
            if (a.block_table) {
              kv[j] = load_x4<BF16>(a.k, off + 4 * c);
              vv[j] = load_x4<BF16>(a.v, off + 4 * c);
            } else {
              const int64_t row = q.q0 + off, col = static_cast<int64_t>(h) * hd + 4 * c;
              kv[j] = load_x4<BF16>(a.k, row * a.k_stride + col);
              vv[j] = load_x4<BF16>(a.v, row * a.v_stride + col);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const int e = e0 + j * kThreads, k = e / (NC * 16), c = e - k * (NC * 16);
          *reinterpret_cast<float4 *>(Ks + k * LD + 4 * c) = kv[j];
          *reinterpret_cast<float4 *>(Vs + k * NC * 64 + 4 * c) = vv[j];
        }
      }
      __syncthreads();
      float s[RP][KP];
#pragma unroll
      for (int p = 0; p < RP; ++p)
#pragma unroll
        for (int k = 0; k < KP; ++k) s[p][k] = 0.0f;
#pragma unroll 2
      for (int c = 0; c < d4; ++c) {
        float4 kk[KP];
#pragma unroll
        for (int k = 0; k < KP; ++k)
          kk[k] = *reinterpret_cast<const float4 *>(Ks + (tx + 16 * k) * LD + 4 * c);
#pragma unroll
        for (int p = 0; p < RP; ++p) {
          const float4 qq = *reinterpret_cast<const float4 *>(Qs + (ty * RP + p) * LD + 4 * c);
#pragma unroll
          for (int k = 0; k < KP; ++k) {
            s[p][k] = fmaf(qq.x, kk[k].x, s[p][k]);
            s[p][k] = fmaf(qq.y, kk[k].y, s[p][k]);
            s[p][k] = fmaf(qq.z, kk[k].z, s[p][k]);
            s[p][k] = fmaf(qq.w, kk[k].w, s[p][k]);
          }
        }
      }
#pragma unroll
      for (int p = 0; p < RP; ++p) {
        const int row = ty * RP + p;
        const int vis = min(all + row / g, end);  // keys this row sees
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
          const int j = tx + 16 * k;
          s[p][k] *= sl2;
          if (guard && (k0 + j >= vis || krow[j] < 0)) s[p][k] = -INFINITY;
          mx = fmaxf(mx, s[p][k]);
        }
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, w));
        const float mn = fmaxf(m[p], mx);
        const float ref = mn == -INFINITY ? 0.0f : mn;  // no key so far: every term is 0
        const float f = ex2(m[p] - ref);
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < KP; ++k) {
          const float e = guard && s[p][k] == -INFINITY ? unseen_weight() : ex2(s[p][k] - ref);
          sum += e;
          Ps[row * PLD + tx + 16 * k] = e;
        }
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, w);
        l[p] = fmaf(l[p], f, sum);
        m[p] = mn;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          o[p][c].x *= f;
          o[p][c].y *= f;
          o[p][c].z *= f;
          o[p][c].w *= f;
        }
      }
      __syncthreads();
      const int steps = guard ? nk : KT;
      for (int k = 0; k < steps; ++k) {
        float pr[RP];
#pragma unroll
        for (int p = 0; p < RP; ++p) pr[p] = Ps[(ty * RP + p) * PLD + k];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float4 vv = *reinterpret_cast<const float4 *>(Vs + k * NC * 64 + 64 * c + 4 * tx);
#pragma unroll
          for (int p = 0; p < RP; ++p) {
            if (guard && is_unseen(pr[p])) continue;  // not even as 0 * NaN
            o[p][c].x = fmaf(pr[p], vv.x, o[p][c].x);
            o[p][c].y = fmaf(pr[p], vv.y, o[p][c].y);
            o[p][c].z = fmaf(pr[p], vv.z, o[p][c].z);
            o[p][c].w = fmaf(pr[p], vv.w, o[p][c].w);
          }
        }
      }
      __syncthreads();
    }
    const bool whole = tile == 0 && stop == ntile;
    const int slot = 2 * blockIdx.x + (tile == 0 ? 1 : 0);
#pragma unroll
    for (int p = 0; p < RP; ++p) {
      const int row = ty * RP + p;
      if (row >= rows) continue;
      if (whole) {
        const float inv = l[p] > 0.0f || l[p] != l[p] ? 1.0f / l[p] : 0.0f;
        const int t = row / g, hq = row - t * g;
        const int64_t y0 = (static_cast<int64_t>(q.q0 + t0 + t) * a.n_head + head0 + hq) * hd;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int d = 64 * c + 4 * tx;
          if (d < hd) store_y4(a.y, y0 + d, make_float4(o[p][c].x * inv, o[p][c].y * inv,
                                                        o[p][c].z * inv, o[p][c].w * inv), a.y_bf16);
        }
      } else {
        const int64_t base = static_cast<int64_t>(slot) * parts.rows + row;
        if (tx == 0) parts.ml[base] = make_float2(m[p], l[p]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int d = 64 * c + 4 * tx;
          if (d < hd) *reinterpret_cast<float4 *>(parts.o + base * hd + d) = o[p][c];
        }
      }
    }
    if (tid == 0 && tile == 0 && !whole) {
      parts.open[blockIdx.x] = AttnOpen{q.q0 + t0, nt, vh, sched_last(sc, run, x, ntile)};
    }
  }
  zero_loose_rows(a, sc, blockIdx.x, gridDim.x, kThreads);
}

// Units divided between workers: worker w (blockIdx.x) started one and left
// its part in slot 2 w + 1; the workers after it, up to `last`, left theirs
// in slots 2 w'.  out = sum_w 2^(m_w - M) o_w / sum_w 2^(m_w - M) l_w with
// M = max_w m_w, in worker order (not in order of arrival), so that a call
// repeated gives the same bits.  A warp per row; reads are a few rows per
// worker and stay in L2.  A launch of its own costs 2 to 3 us and needs no
// counters or flags between workers, which would have to be reset.
__global__ void __launch_bounds__(128) attn_join_kernel(AttnBatch a, int gsub, int nsub,
                                                        AttnParts parts) {
  pdl_enter();
  const AttnOpen u = parts.open[blockIdx.x];
  if (u.rows_tok == 0) return;
  const int grp = a.n_head / a.n_kv, hd = a.head_dim;
  const int h = u.vh / nsub, sub = u.vh - h * nsub, g = min(gsub, grp - sub * gsub);
  const int rows = u.rows_tok * g, d4 = hd / 4;
  const int w0 = blockIdx.x;
  const int lanes = blockDim.x / 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int row = blockIdx.y * lanes + warp; row < rows; row += gridDim.y * lanes) {
    auto at = [&](int w) {
      return static_cast<int64_t>(w == w0 ? 2 * w + 1 : 2 * w) * parts.rows + row;
    };
    float M = -INFINITY;
    for (int w = w0 + lane; w <= u.last; w += 32) M = fmaxf(M, parts.ml[at(w)].x);
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, k));
    const float ref = M == -INFINITY ? 0.0f : M;
    const int t = row / g, hq = row - t * g;
    const int64_t y0 =
        (static_cast<int64_t>(u.q0 + t) * a.n_head + h * grp + sub * gsub + hq) * hd;
    for (int c = lane; c < d4; c += 32) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.0f;
#pragma unroll 4
      for (int w = w0; w <= u.last; ++w) {
        const float2 ml = parts.ml[at(w)];
        const float4 v = *reinterpret_cast<const float4 *>(parts.o + at(w) * hd + 4 * c);
        // A part that saw no key is all zeros, and counts nothing; one that holds a
        // NaN makes the row NaN, however small its factor is (NaN scores do not
        // show in the maximum).
        const float f = ex2(ml.x - ref);
        L = fmaf(f, ml.y, L);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;
      store_y4(a.y, y0 + 4 * c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv),
               a.y_bf16);
    }
  }
}

template <bool BF16, int NC, int TR>
cudaError_t launch_simt(const AttnBatch &a, const AttnSched &sc, int gsub, int nsub,
                        const AttnParts &parts, int workers, cudaStream_t s) {
  auto kern = attn_simt_kernel<BF16, NC, TR>;
  constexpr int smem = Simt<NC, TR>::smem;
  static_assert(smem <= 227 * 1024, "shared memory");
  const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  uint32_t *status = device_status();
  if (!status) return cudaErrorInvalidDevice;
  return launch_pdl(kern, dim3(workers), dim3(kThreads), smem, s, a, sc, gsub, nsub, parts, status);
}

// Column groups of the form that takes a call: the plan's tiles and the launch
// both follow from it.  fp32 has no forms below four (such calls go to
// attn_rows_kernel or attn_tile_kernel); the wider one would compute the same.
int simt_nc(bool bf16, int head_dim) {
  if (head_dim > 256) return 8;
  return head_dim > 128 || !bf16 ? 4 : head_dim > 64 ? 2 : 1;
}

template <bool BF16, int TR>
cudaError_t launch_simt_nc(int nc, const AttnBatch &a, const AttnSched &sc, int gsub, int nsub,
                           const AttnParts &parts, int workers, cudaStream_t s) {
  if constexpr (BF16) {
    if (nc == 1) return launch_simt<BF16, 1, TR>(a, sc, gsub, nsub, parts, workers, s);
    if (nc == 2) return launch_simt<BF16, 2, TR>(a, sc, gsub, nsub, parts, workers, s);
  }
  if (nc == 4) return launch_simt<BF16, 4, TR>(a, sc, gsub, nsub, parts, workers, s);
  return launch_simt<BF16, 8, TR>(a, sc, gsub, nsub, parts, workers, s);
}

}  // namespace

AttnPlan attn_simt_plan(bool bf16, int64_t T, int n_head, int n_kv, int head_dim, int R) {
  const int grp = n_head / n_kv;
  AttnPlan p;
  p.rows = T * grp <= static_cast<int64_t>(16) * R ? 16 : 64;
  p.gsub = grp < p.rows ? grp : p.rows;
  p.nsub = (grp + p.gsub - 1) / p.gsub;
  p.U = p.rows / p.gsub;
  const int nc = simt_nc(bf16, head_dim);
  p.KT = nc <= 2 ? 64 : (nc == 4 ? 32 : 16);
  p.fixed = p.KT;
  p.min_run = p.KT;
  p.whole = 128;  // four prompts of 40 tokens, 512 columns: whole 47 us, divided 64
  p.workers = sm_count() * 2;
  return p;
}

cudaError_t launch_attn_simt(const AttnBatch &a, const AttnPlan &p, const AttnSched &sc,
                             const AttnParts &parts, cudaStream_t s) {
  const int nc = simt_nc(a.bf16, a.head_dim);
  if (a.bf16)
    return p.rows == 16 ? launch_simt_nc<true, 16>(nc, a, sc, p.gsub, p.nsub, parts, p.workers, s)
                        : launch_simt_nc<true, 64>(nc, a, sc, p.gsub, p.nsub, parts, p.workers, s);
  return p.rows == 16 ? launch_simt_nc<false, 16>(nc, a, sc, p.gsub, p.nsub, parts, p.workers, s)
                      : launch_simt_nc<false, 64>(nc, a, sc, p.gsub, p.nsub, parts, p.workers, s);
}

cudaError_t launch_attn_join(const AttnBatch &a, const AttnPlan &p, const AttnParts &parts,
                             cudaStream_t s) {
  // rows of the largest unit, 32 to a block
  const int64_t rows = a.T * p.gsub < p.rows ? a.T * p.gsub : p.rows;
  const int ny = static_cast<int>((rows + 31) / 32);
  return launch_pdl(attn_join_kernel, dim3(p.workers, ny), dim3(128), 0, s, a, p.gsub, p.nsub,
                    parts);
}

}  // namespace qmm
