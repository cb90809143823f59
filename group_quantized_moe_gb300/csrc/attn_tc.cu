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
#include "attn_tc_body.cuh"

namespace qmm {
namespace {

template <int NCH, bool PAGED, bool STAGED>
__global__ void __launch_bounds__(Tc<NCH, STAGED, false>::threads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TcAttn p) {
  attn_tc_body<NCH, PAGED, STAGED, 0, 1>(tm_q, tm_k, tm_v, p, Kv4{});
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
  constexpr uint32_t smem = Tc<NCH, STAGED, false>::bytes;
  static_assert(smem <= 227 * 1024, "shared memory");
  const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(workers), dim3(Tc<NCH, STAGED, false>::threads), smem, s, q, k, v, p);
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
