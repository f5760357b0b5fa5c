// Launch of the backward's score-modified instances (BwdArgs::sc set): whole
// units, one CTA per key tile (two at d = 256).
#include "bwd_kernel.cuh"
#include "ops.h"

namespace attn {

namespace {

template <int DT, int D>
cudaError_t launch_inst(const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q, const CUtensorMap& d,
                        const CUtensorMap& dq, const BwdArgs& a, int N, int nz, cudaStream_t st) {
  using C = BwdCfg<DT, D>;
  cudaError_t e = smem_attr_once<bwd_kernel<DT, D, true, false, false, true>>(C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  if ((e = reg_pool_once<bwd_kernel<DT, D, true, false, false, true>>(C::NTHREADS, C::kRegsSplit)) != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((N + C::BC - 1) / C::BC * C::DSPLIT), static_cast<unsigned>(a.Hkv),
                  static_cast<unsigned>(nz));
  BwdArgs g = a;
  g.tiles_x = 0;
  g.unit0 = 0;
  g.nsplit = 1;
  bwd_kernel<DT, D, true, false, false, true><<<grid, C::NTHREADS, C::SMEM_BYTES, st>>>(k, v, q, d, dq, g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd_score(int dt, int d, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q,
                             const CUtensorMap& dout, const CUtensorMap& dq_acc, const BwdArgs& a, int N, int nz,
                             cudaStream_t st) {
  switch (d) {
    case 64: return dt == kBF16 ? launch_inst<kBF16, 64>(k, v, q, dout, dq_acc, a, N, nz, st)
                                : launch_inst<kFP16, 64>(k, v, q, dout, dq_acc, a, N, nz, st);
    case 128: return dt == kBF16 ? launch_inst<kBF16, 128>(k, v, q, dout, dq_acc, a, N, nz, st)
                                 : launch_inst<kFP16, 128>(k, v, q, dout, dq_acc, a, N, nz, st);
    case 256: return dt == kBF16 ? launch_inst<kBF16, 256>(k, v, q, dout, dq_acc, a, N, nz, st)
                                 : launch_inst<kFP16, 256>(k, v, q, dout, dq_acc, a, N, nz, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
