// Launch of the backward's score-modified instances (BwdScoreArgs): whole
// units, one CTA per key tile (two at d = 256).
#pragma once
#include "bwd_kernel.cuh"
#include "ops.h"

namespace attn {

template <int DT, int D, int kScore>
cudaError_t launch_bwd_score_inst(const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q,
                                  const CUtensorMap& d, const CUtensorMap& dq, const BwdScoreArgs& a, int N, int nz,
                                  cudaStream_t st) {
  using C = BwdCfg<DT, D>;
  cudaError_t e = smem_attr_once<bwd_kernel<DT, D, true, false, false, kScore>>(C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  if ((e = reg_pool_once<bwd_kernel<DT, D, true, false, false, kScore>>(C::NTHREADS, C::kRegsSplit)) != cudaSuccess)
    return e;
  const dim3 grid(static_cast<unsigned>((N + C::BC - 1) / C::BC * C::DSPLIT), static_cast<unsigned>(a.Hkv),
                  static_cast<unsigned>(nz));
  BwdScoreArgs g = a;
  g.tiles_x = 0;
  g.unit0 = 0;
  g.nsplit = 1;
  bwd_kernel<DT, D, true, false, false, kScore><<<grid, C::NTHREADS, C::SMEM_BYTES, st>>>(k, v, q, d, dq, g);
  return cudaGetLastError();
}

// mode: kScoreCap, kScoreBias, kScoreRanges together, not 0
template <int DT, int D>
cudaError_t launch_bwd_score_mode(int mode, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q,
                                  const CUtensorMap& d, const CUtensorMap& dq, const BwdScoreArgs& a, int N, int nz,
                                  cudaStream_t st) {
  switch (mode) {
    case 1: return launch_bwd_score_inst<DT, D, 1>(k, v, q, d, dq, a, N, nz, st);
    case 2: return launch_bwd_score_inst<DT, D, 2>(k, v, q, d, dq, a, N, nz, st);
    case 3: return launch_bwd_score_inst<DT, D, 3>(k, v, q, d, dq, a, N, nz, st);
    case 4: return launch_bwd_score_inst<DT, D, 4>(k, v, q, d, dq, a, N, nz, st);
    case 5: return launch_bwd_score_inst<DT, D, 5>(k, v, q, d, dq, a, N, nz, st);
    case 6: return launch_bwd_score_inst<DT, D, 6>(k, v, q, d, dq, a, N, nz, st);
    case 7: return launch_bwd_score_inst<DT, D, 7>(k, v, q, d, dq, a, N, nz, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
