// Score-modified backward instances at head dim 64.
#include "bwd_score.cuh"

namespace attn {

cudaError_t launch_bwd_score_64(int mode, int dt, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q,
                                const CUtensorMap& dout, const CUtensorMap& dq_acc, const BwdScoreArgs& a, int N, int nz,
                                cudaStream_t st) {
  return dt == kBF16 ? launch_bwd_score_mode<kBF16, 64>(mode, k, v, q, dout, dq_acc, a, N, nz, st)
                     : launch_bwd_score_mode<kFP16, 64>(mode, k, v, q, dout, dq_acc, a, N, nz, st);
}

}  // namespace attn
