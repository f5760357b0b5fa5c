// The forward softmax step of capped and biased scores (kScoreCap, kScoreBias).
//
// A thread has one row of a 128 x 128 score tile in tensor memory. The plain
// step holds the row in 128 registers and is unrolled over it; with a cap the
// unrolled code no longer fits the instruction caches (ncu: instruction
// fetch was the largest added stall, 0.9 of 8.3 warps per issue against 0.24
// for the plain step), so here every pass is a loop over four chunks of 32
// columns that reads them from tensor memory again.
//
// A tile goes straight from its raw scores to its weights, cap and bias folded
// into the exponent, unless a mask cuts it or it crosses the diagonal of a
// bias: such tiles get their final scores written back first. tanh rises, so
// the largest raw score gives the running max; even that is looked for only
// where an upper bound (the largest magnitude, and the nearest key's bias)
// passes the running max by the threshold that moves it.
#pragma once
#include <cmath>

#include "score.cuh"

namespace attn {

struct ScoreStep {
  float mx;        // the row's largest final score (log2 units), where keep_max is false
  bool keep_max;   // warp-uniform: no row's score passes the threshold
  int way;         // warp-uniform: 0 final scores in tensor memory, else raw, and the tanh's tier (1, 2, 3)
};

// Largest magnitude (kAbs) or value of the row's 128 raw scores.
template <bool kAbs>
__device__ __forceinline__ float score_rowmax(uint32_t tS) {
  uint32_t r0[32], r1[32];
  float m[2];
  tmem_ld32(tS, r0);
  m[0] = m[1] = kAbs ? 0.f : -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; c += 2) {
    tmem_wait_ld();
    reg_fence(r0);
    tmem_ld32(tS + 32 * (c + 1), r1);
    m[0] = fmaxf(m[0], kAbs ? rowmax_abs(r0) : rowmax(r0));
    tmem_wait_ld();
    reg_fence(r1);
    if (c == 0) tmem_ld32(tS + 64, r0);
    m[1] = fmaxf(m[1], kAbs ? rowmax_abs(r1) : rowmax(r1));
  }
  return fmaxf(m[0], m[1]);
}

// dist: key - row of column 0; columns lo <= c < hi are visible; limit: the
// running max plus the threshold.
template <bool kCap, bool kBias>
__device__ __forceinline__ ScoreStep score_step(uint32_t tS, const ScoreArgs& sc, float limit, bool edge, float slope2,
                                                int dist, int lo, int hi) {
  ScoreStep st;
  int tier = 1;
  bool keep = false;
  float near = 0.f;
  if constexpr (kBias) {   // keys before the row: the bias is linear, largest at the nearest key
    const float at = static_cast<float>(dist);
    near = fmaxf(slope2 * at, slope2 * (at + 127.f));
  }
  float mx;
  if constexpr (kCap) {
    const float big = score_rowmax<true>(tS);
    if (warp_any(!(big <= sc.s_small))) tier = warp_any(!(big * fabsf(sc.w_of_s) <= 1.f)) ? 3 : 2;
    mx = cap_by(tier, big, sc);
  } else {
    mx = score_rowmax<false>(tS) * sc.sl2;
  }
  keep = !warp_any(!(mx + near <= limit));
  bool straight = !edge;
  if constexpr (kBias) straight = straight && !warp_any(dist + 127 > 0);
  if (straight && !keep) {
    if constexpr (kCap) {   // the bound was of the magnitude: now the value
      mx = cap_by(tier, score_rowmax<false>(tS), sc);
      if constexpr (kBias) keep = !warp_any(!(mx + near <= limit));
    }
    if constexpr (kBias) straight = keep;   // which key has the largest biased score is not known from the raw ones
  }
  st.mx = mx;
  st.keep_max = keep && straight;
  st.way = straight ? tier : 0;
  if (!straight) {
    float top = -INFINITY;
    const float from = static_cast<float>(dist);
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t r[32];
      tmem_ld32(tS + 32 * c, r);
      tmem_wait_ld();
      reg_fence(r);
      if constexpr (kCap) {
        if (tier < 3) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = cap_pair(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), sc.w_of_s, sc.cap_log2);
            r[e] = __float_as_uint(y.x);
            r[e + 1] = __float_as_uint(y.y);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            r[e] = __float_as_uint(cap_any(__uint_as_float(r[e]), sc.w_of_s, sc.cap_log2));
        }
      }
      if constexpr (kBias) {
        const float f = from + static_cast<float>(32 * c);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float y = kCap ? __uint_as_float(r[e]) : __uint_as_float(r[e]) * sc.sl2;
          r[e] = __float_as_uint(fmaf(-slope2, fabsf(f + static_cast<float>(e)), y));
        }
      }
      if (edge) {
        const int l = lo - 32 * c, h = hi - 32 * c;
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (e >= h || e < l) r[e] = __float_as_uint(-INFINITY);
      }
      top = fmaxf(top, rowmax(r));
      tmem_st32(tS + 32 * c, r);
    }
    tmem_wait_st();
    st.mx = top;
  }
  return st;
}

// The row's weights exp2(x + bias) over its scores, 16-bit pairs, and their
// sums. Chunk c's weights take columns 16c .. 16c + 15: of its own or earlier
// chunks' scores, never of the one whose load is already under way.
template <bool kBF16, bool kCap, bool kBias, int kWay>
__device__ __forceinline__ void score_weights_way(uint32_t tS, const ScoreArgs& sc, float slope2, int dist, float bias,
                                                  float2 (&acc)[4]) {
  const float2 rise = make_float2(slope2, slope2);
  auto chunk = [&](int c, const uint32_t(&r)[32]) {
    float b0 = bias;
    if constexpr (kBias && kWay != 0) b0 += slope2 * static_cast<float>(dist + 32 * c);
    const float2 at = make_float2(b0, b0);
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 s = make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
      float2 b = at;
      if constexpr (kBias && kWay != 0)
        b = ffma2(rise, make_float2(static_cast<float>(2 * e), static_cast<float>(2 * e + 1)), at);
      float2 x;
      if constexpr (kWay == 0) {
        x = fadd2(s, b);
      } else if constexpr (!kCap) {
        x = ffma2(s, make_float2(sc.sl2, sc.sl2), b);
      } else if constexpr (kWay == 1) {
        x = ffma2(s, cap_small_factor(s, sc), b);
      } else if constexpr (kWay == 2) {
        float2 w;
        const float2 q = cap_factor(s, sc.w_of_s, w);
        x = ffma2(q, fmul2(w, make_float2(sc.cap_log2, sc.cap_log2)), b);
      } else {
        x = fadd2(make_float2(cap_any(s.x, sc.w_of_s, sc.cap_log2), cap_any(s.y, sc.w_of_s, sc.cap_log2)), b);
      }
      x = make_float2(ex2(x.x), ex2(x.y));
      acc[e & 3] = fadd2(acc[e & 3], x);
      pk[e] = kBF16 ? pack_bf16x2(x.x, x.y) : pack_f16x2(x.x, x.y);
    }
    tmem_st16(tS + 16 * c, pk);
  };
  uint32_t r0[32], r1[32];
  tmem_ld32(tS, r0);
#pragma unroll 1
  for (int c = 0; c < 4; c += 2) {
    tmem_wait_ld();
    reg_fence(r0);
    tmem_ld32(tS + 32 * (c + 1), r1);
    chunk(c, r0);
    tmem_wait_ld();
    reg_fence(r1);
    if (c == 0) tmem_ld32(tS + 64, r0);
    chunk(c + 1, r1);
  }
}
template <bool kBF16, bool kCap, bool kBias>
__device__ __forceinline__ void score_weights(uint32_t tS, const ScoreArgs& sc, int way, float slope2, int dist,
                                              float bias, float2 (&acc)[4]) {
  if (way == 0) score_weights_way<kBF16, kCap, kBias, 0>(tS, sc, slope2, dist, bias, acc);
  else if (!kCap || way == 1) score_weights_way<kBF16, kCap, kBias, 1>(tS, sc, slope2, dist, bias, acc);
  else if (way == 2) score_weights_way<kBF16, kCap, kBias, kCap ? 2 : 1>(tS, sc, slope2, dist, bias, acc);
  else score_weights_way<kBF16, kCap, kBias, kCap ? 3 : 1>(tS, sc, slope2, dist, bias, acc);
}

}  // namespace attn
