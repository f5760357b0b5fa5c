// Score-modified forward instances with bf16 operands, tiled as the plain ones.
#include "fwd_launch.cuh"

namespace attn {

cudaError_t launch_fwd_score_bf16(int mode, int d, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                  const FwdArgs& a, int rows, int gy, int gz, cudaStream_t st) {
  switch (d) {
    case 64: return launch_fwd_score_inst<kBF16, 64, 2>(mode, q, k, v, a, rows, gy, gz, st);
    case 128: return launch_fwd_score_inst<kBF16, 128, 2>(mode, q, k, v, a, rows, gy, gz, st);
    case 256: return launch_fwd_score_inst<kBF16, 256, 1>(mode, q, k, v, a, rows, gy, gz, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace attn
