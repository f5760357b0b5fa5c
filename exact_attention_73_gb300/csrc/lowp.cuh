// Conversions shared by the kernels that read 16-bit rows or E4M3 codes.
#pragma once
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace attn {

// Largest e with amax * 2^e <= 448 (448 = 0.875 * 2^9), 0 for amax == 0.
__device__ __forceinline__ int e4m3_scale_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  int k;
  const float m = frexpf(amax, &k);   // amax = m * 2^k, m in [0.5, 1)
  return (m <= 0.875f) ? 9 - k : 8 - k;
}

template <typename T>
__device__ __forceinline__ float to_f32(uint32_t bits16) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(bits16 << 16);
  else return __half2float(__ushort_as_half(static_cast<unsigned short>(bits16)));
}

// Eight consecutive 16-bit elements (one 16-byte vector) as floats.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    v[2 * u] = to_f32<T>(wv[u] & 0xFFFFu);
    v[2 * u + 1] = to_f32<T>(wv[u] >> 16);
  }
}

}  // namespace attn
