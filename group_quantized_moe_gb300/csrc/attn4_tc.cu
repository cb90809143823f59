// attn4_tc.cu -- batched attention over a paged cache held in 4 bits (layout:
// kv4.h) for many query rows: chunks of prompts, beside single tokens.
//
// The tensor-core kernel of attn_tc.cu (tcgen05, scores and results in tensor
// memory), whose tiles of 128 keys and values are made here from the codes: warp
// 8 fetches the strips of 64 keys by bulk copies, three such halves in flight,
// and two more warpgroups turn the codes of keys and of values into bf16 tiles in
// shared memory, (code - zp) s rounded once (2^-8 of a value).
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
