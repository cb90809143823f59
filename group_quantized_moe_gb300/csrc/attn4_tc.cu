// attn4_tc.cu -- batched attention over a paged cache held in 4 bits (layout:
// kv4.h) for many query rows: chunks of prompts, beside single tokens.
//
// The tensor-core kernel of attn_tc.cu (tcgen05, scores and results in tensor
// memory), whose tiles of 128 keys and values are made here from the codes: warp
// 8 fetches the strips of 64 keys by bulk copies, three such halves in flight,
// and two more warpgroups turn the codes of keys and of values into tiles in
// shared memory, (code - zp) s rounded once: keys to fp16 (2^-11 of a value), as
// scores magnify what is lost, values to bf16 (2^-8), as they come in any range.
// Keys in fp16 need queries in fp16: a tile's rows are turned where they lie, each
// times a power of two that brings its largest element to [2^14, 2^15) and that
// its scores lose again; a key row out of fp16's range is divided by one, and the
// warpgroups multiply its column of scores (a mark per tile says so).
//
// What bounds it: making the tiles, beside the exponentials, for every query tile
// pair again: issue slots are 51 % busy, the tensor cores 41 % of the time.  20
// requests, 4076 tokens in four chunks over up to 21000 keys, 32 heads over 8 of
// 128: 1.02 ms, 0.6 without conversions.  One warpgroup for both kinds of codes took
// 1.56 ms with bf16 keys, two 1.01 (fp16 keys 0.06 more); conversions with a branch
// a word 2.4; codes put back into the dimensions' order 1.07; words read only after
// their parameters 1.04.
// Registers: 176 a thread for the warpgroups that compute the weights, 48 for those
// of the codes, 32 for the others (168, 32 and 56: the same; 160, 32 and 64: 1.53 ms;
// 168, 48 and 48, before the dimensions' order: 1.13 against 1.07).
#include "attn_tc_body.cuh"
#include "kv4.h"

namespace qmm {
namespace {

// NC: chunks of 32 dimensions; CPG: chunks of a group.
template <int NC>
using Tc4 = Tc<(NC + 1) / 2, false, true>;

template <int NC, int CPG>
__global__ void __launch_bounds__(Tc4<NC>::threads, 1)
    attn4_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ TcAttn p,
                    const __grid_constant__ Kv4 c) {
  attn_tc_body<(NC + 1) / 2, true, false, NC, CPG>(tm_q, tm_q, tm_q, p, c);
}

template <int NC, int CPG>
cudaError_t run_tc(const CUtensorMap &q, const TcAttn &p, const Kv4 &c, int workers, cudaStream_t s) {
  auto kern = attn4_tc_kernel<NC, CPG>;
  constexpr uint32_t smem = Tc4<NC>::bytes;
  static_assert(smem <= 227 * 1024, "shared memory");
  const cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(workers), dim3(Tc4<NC>::threads), smem, s, q, p, c);
}

}  // namespace

bool attn4_tc_takes(const AttnBatch &a) {
  return a.bf16 && a.head_dim <= 128 && a.q_stride % 8 == 0 && a.q_stride <= (int64_t(1) << 38);
}

cudaError_t launch_attn4_tc(const AttnBatch &a, const Kv4 &c, const AttnPlan &pl, const AttnSched &sc,
                            const AttnParts &parts, cudaStream_t s) {
  TcAttn p{};
  p.a = a;
  p.a.num_blocks = c.num_blocks;
  p.sc = sc;
  p.parts = parts;
  p.gsub = pl.gsub;
  p.nsub = pl.nsub;
  p.tpt = pl.U / 2;
  p.block_shift = c.block_shift;
  p.sl2 = a.scale * 1.4426950408889634f;
  p.most_e = kv4_most_exponent(p.sl2);
  p.status = device_status();
  if (!p.status) return cudaErrorInvalidDevice;
  CUtensorMap q;
  if (!map_rows(&q, a.q, a.T, a.q_stride, a.n_head, a.head_dim, p.gsub, p.tpt)) return cudaErrorInvalidValue;
  const bool two = c.cpg == 2;
  switch (c.nc) {
    case 1: return run_tc<1, 1>(q, p, c, pl.workers, s);
    case 2: return two ? run_tc<2, 2>(q, p, c, pl.workers, s) : run_tc<2, 1>(q, p, c, pl.workers, s);
    case 3: return two ? run_tc<3, 2>(q, p, c, pl.workers, s) : run_tc<3, 1>(q, p, c, pl.workers, s);
    default: return two ? run_tc<4, 2>(q, p, c, pl.workers, s) : run_tc<4, 1>(q, p, c, pl.workers, s);
  }
}

}  // namespace qmm
