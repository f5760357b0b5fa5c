// Appending rows to a block-quantised KV cache, with the rotation of the keys.
//
// A cache block is 128 tokens of one KV head with one power-of-two factor. A
// call adds rows start .. start + n - 1 to each sequence; every block that
// gets a row then holds what attn_quantize_fp8's rule gives for the block's
// earlier rows (at the values that their codes stand for) and the new ones
// together: e = the largest integer with amax 2^e <= 448 over both, codes
// e4m3_rn(x 2^e), factor 2^-e. The earlier rows are written again only where
// e moved. Keys are rotated in FP32 first (each product and sum rounded on its
// own, as attn_quantize_fp8_rope does).
//
// One CTA per (block of the new rows, KV head, sequence and K or V). A
// block's rows belong to one CTA, so nothing is shared between CTAs and no
// atomics are needed. HBM-bound for prompts (2 bytes in, 1 out per element),
// latency-bound for single tokens, where the earlier rows' codes (at most 16
// KB at d = 128) are read for their largest magnitude: E4M3 magnitudes order
// as their low seven bits, so that maximum is taken on packed bytes.
#include <cstdint>

#include "../../include/libattn.h"
#include "lowp.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace attn {

namespace {

struct AppendArgs {
  const void* x[2];          // new rows of K and V, strides x_sb, x_sh, x_sn (elements)
  uint8_t* x8[2];
  float* scales[2];
  const int* seqlens;        // rows held before the call
  const int* new_lens;       // new rows per sequence (null: n_new)
  const int* table;          // [B, max_blocks] pages (null: dense cache)
  const float* cos;          // [n_pos, rot / 2] or null
  const float* sin;
  long long x_sb[2], x_sh[2], x_sn[2];
  int B, Hkv, n_new;
  int rows_max;              // rows a sequence can hold
  int limit;                 // first row that is dropped: rows_max, or the tables' end before it
  int blocks;                // blocks per sequence (of the table, or of the dense cache)
  int pages;                 // pages of a paged cache
  int rot, interleaved;
  int* status;
};

__device__ __forceinline__ uint32_t max_u8x4(uint32_t a, uint32_t b) { return __vmaxu4(a, b); }

// value of the E4M3 magnitude `m` (0 .. 126)
__device__ __forceinline__ float e4m3_magnitude(uint32_t m) {
  const uint32_t ex = m >> 3, man = m & 7u;
  return ex == 0 ? static_cast<float>(man) * 0.001953125f                       // man * 2^-9
                 : __uint_as_float(((ex + 120u) << 23) | (man << 20));          // 2^(ex-7) (1 + man/8)
}

// Element chunks of a row: 16 elements per thread. Rotated: 8 pairs (two
// vectors, half apart or adjacent); past `rot`, 16 consecutive elements.
template <typename T, int D>
__device__ __forceinline__ void load_chunk(const AppendArgs& a, const T* row, int c, bool turn, int pos, int& e0,
                                           int& e1, float (&v0)[8], float (&v1)[8]) {
  const int half = a.rot / 2;
  const bool split = turn && !a.interleaved;
  e0 = split ? 8 * c : 16 * c;
  e1 = split ? half + 8 * c : 16 * c + 8;
  unpack8<T>(*reinterpret_cast<const uint4*>(row + e0), v0);
  unpack8<T>(*reinterpret_cast<const uint4*>(row + e1), v1);
  if (!turn) return;
  const float* ct = a.cos + static_cast<long long>(pos) * half + 8 * c;
  const float* st = a.sin + static_cast<long long>(pos) * half + 8 * c;
  float cs[8], sn[8];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(ct) + q), w = __ldg(reinterpret_cast<const float4*>(st) + q);
    cs[4 * q] = u.x; cs[4 * q + 1] = u.y; cs[4 * q + 2] = u.z; cs[4 * q + 3] = u.w;
    sn[4 * q] = w.x; sn[4 * q + 1] = w.y; sn[4 * q + 2] = w.z; sn[4 * q + 3] = w.w;
  }
  auto turned = [](float& p, float& q, float c_, float s_) {
    const float u = __fsub_rn(__fmul_rn(p, c_), __fmul_rn(q, s_));
    q = __fadd_rn(__fmul_rn(q, c_), __fmul_rn(p, s_));
    p = u;
  };
  if (a.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turned(v0[2 * i], v0[2 * i + 1], cs[i], sn[i]);
      turned(v1[2 * i], v1[2 * i + 1], cs[4 + i], sn[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turned(v0[i], v1[i], cs[i], sn[i]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
  constexpr int CH = D / 16;            // chunks per row
  constexpr int RSTEP = 256 / CH;       // rows per pass
  __shared__ float red[8];
  const int h = blockIdx.y, b = static_cast<int>(blockIdx.z) >> 1, kv = blockIdx.z & 1;
  const int start = a.seqlens[b];
  int n = a.new_lens ? min(a.new_lens[b], a.n_new) : a.n_new;
  if (start < 0 || (n > 0 && static_cast<long long>(start) + n > a.limit)) {   // rows that do not fit are dropped
    if (threadIdx.x == 0) atomicExch(a.status, kDevBadIndex);
    if (start < 0) return;
    n = a.limit - start;
  }
  if (n <= 0) return;
  const int blk = (start >> 7) + static_cast<int>(blockIdx.x);
  if (blk > (start + n - 1) >> 7) return;
  // rows of the block: [0, r0) were there, [r0, r1) are new
  const int r0 = max(start - blk * 128, 0), r1 = min(start + n - blk * 128, 128);
  long long base, si;
  if (a.table) {
    const int page = a.table[static_cast<long long>(b) * a.blocks + blk];
    if (page < 0 || page >= a.pages) {   // no such page: its rows are dropped
      if (threadIdx.x == 0) atomicExch(a.status, kDevBadIndex);
      return;
    }
    si = static_cast<long long>(page) * a.Hkv + h;
    base = si * 128 * D;
  } else {
    si = (static_cast<long long>(b) * a.Hkv + h) * a.blocks + blk;
    base = ((static_cast<long long>(b) * a.Hkv + h) * a.rows_max + static_cast<long long>(blk) * 128) * D;
  }
  uint8_t* x8 = a.x8[kv] + base;
  const T* x = static_cast<const T*>(a.x[kv]) + b * a.x_sb[kv] + h * a.x_sh[kv] +
               static_cast<long long>(blk * 128 - start) * a.x_sn[kv];   // row r of the block at x + r * x_sn
  const bool rope = kv == 0 && a.cos != nullptr;
  const int c = threadIdx.x % CH, rt = threadIdx.x / CH;
  const bool turn = rope && 16 * c < a.rot;
  // largest magnitude of the rows that were there and of the new ones
  const float s_old = r0 > 0 ? a.scales[kv][si] : 1.f;
  float amax = 0.f;
  for (int r = r0 + rt; r < r1; r += RSTEP) {
    int e0, e1;
    float v0[8], v1[8];
    load_chunk<T, D>(a, x + r * a.x_sn[kv], c, turn, blk * 128 + r, e0, e1, v0, v1);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmax3(amax, fabsf(v0[i]), fabsf(v1[i]));
  }
  uint32_t held = 0;
  for (int i = threadIdx.x; i < r0 * (D / 16); i += 256) {
    const uint4 w = reinterpret_cast<const uint4*>(x8)[i];
    held = max_u8x4(held, max_u8x4(max_u8x4(w.x & 0x7f7f7f7fu, w.y & 0x7f7f7f7fu),
                                   max_u8x4(w.z & 0x7f7f7f7fu, w.w & 0x7f7f7f7fu)));
  }
  uint32_t m = max(max(held & 0xffu, (held >> 8) & 0xffu), max((held >> 16) & 0xffu, held >> 24));
  amax = fmaxf(amax, e4m3_magnitude(min(m, 126u)) * s_old);   // a NaN code (127) counts as 448
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) amax = fmaxf(amax, red[i]);
  const int e = e4m3_scale_exponent(amax);
  // 2^e in two factors, both normal floats whatever e is
  const float f1 = ldexpf(1.f, e / 2), f2 = ldexpf(1.f, e - e / 2);
  const float s_new = ldexpf(1.f, -e);
  if (threadIdx.x == 0) a.scales[kv][si] = s_new;
  if (r0 > 0 && s_new != s_old) {   // the earlier rows at the new factor
    for (int i = threadIdx.x; i < r0 * (D / 16); i += 256) {
      uint4 w = reinterpret_cast<const uint4*>(x8)[i];
      uint32_t* p = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t code = (p[q] >> (8 * k)) & 0xffu;
          const float mag = (code & 0x7fu) == 0x7fu ? __int_as_float(0x7fc00000) : e4m3_magnitude(code & 0x7fu);
          f[k] = (code & 0x80u ? -mag : mag) * s_old * f1 * f2;
        }
        p[q] = pack_e4m3x4(f[0], f[1], f[2], f[3]);
      }
      reinterpret_cast<uint4*>(x8)[i] = w;
    }
  }
  for (int r = r0 + rt; r < r1; r += RSTEP) {
    int e0, e1;
    float v0[8], v1[8];
    load_chunk<T, D>(a, x + r * a.x_sn[kv], c, turn, blk * 128 + r, e0, e1, v0, v1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v0[i] = v0[i] * f1 * f2;
      v1[i] = v1[i] * f1 * f2;
    }
    uint8_t* dst = x8 + r * D;
    *reinterpret_cast<uint2*>(dst + e0) = make_uint2(pack_e4m3x4(v0[0], v0[1], v0[2], v0[3]),
                                                     pack_e4m3x4(v0[4], v0[5], v0[6], v0[7]));
    *reinterpret_cast<uint2*>(dst + e1) = make_uint2(pack_e4m3x4(v1[0], v1[1], v1[2], v1[3]),
                                                     pack_e4m3x4(v1[4], v1[5], v1[6], v1[7]));
  }
}

template <typename T>
cudaError_t launch_append(int d, const AppendArgs& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((a.n_new + 126) / 128 + 1), static_cast<unsigned>(a.Hkv),
                  static_cast<unsigned>(2 * a.B));
  switch (d) {
    case 64: append_kernel<T, 64><<<grid, 256, 0, st>>>(a); break;
    case 128: append_kernel<T, 128><<<grid, 256, 0, st>>>(a); break;
    default: append_kernel<T, 256><<<grid, 256, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

}  // namespace attn

using namespace attn;

extern "C" attn_status attn_cache_append_fp8(const void* k, const void* v, const long long* k_strides,
                                             const long long* v_strides, void* k8, void* v8, float* sk, float* sv,
                                             const int* seqlens, const int* new_lens, const int* block_table,
                                             const float* rope_cos, const float* rope_sin, int B, int Hkv, int n_new,
                                             int Nmax, int num_pages, int d, int rot_dim, int n_pos, int interleaved,
                                             attn_dtype dtype, void* stream) {
  if (!k || !v || !k_strides || !v_strides || !k8 || !v8 || !sk || !sv || !seqlens) return ATTN_ERR_NULL;
  if ((rope_cos == nullptr) != (rope_sin == nullptr)) return ATTN_ERR_NULL;
  const void* ptrs[] = {k, v, k8, v8, sk, sv, seqlens, new_lens, block_table, rope_cos, rope_sin};
  for (const void* p : ptrs)
    if (!aligned16(p)) return ATTN_ERR_ALIGN;
  if (B < 1 || B > 32767 || Hkv < 1 || Hkv > 65535 || n_new < 1 || Nmax < 1 || Nmax > 0x7fffff00) return ATTN_ERR_SHAPE;
  if (block_table && (num_pages < 1 || Nmax % 128)) return ATTN_ERR_SHAPE;
  if (d != 64 && d != 128 && d != 256) return ATTN_ERR_HEADDIM;
  if (rope_cos && (rot_dim < 16 || rot_dim > d || rot_dim % 16 || n_pos < 1)) return ATTN_ERR_SHAPE;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_DTYPE;
  for (int i = 0; i < 3; ++i)
    if (k_strides[i] % 8 || v_strides[i] % 8) return ATTN_ERR_ALIGN;
  int* status;
  attn_status s = device_context(&status);
  if (s != ATTN_OK) return s;
  AppendArgs a{};
  a.x[0] = k;
  a.x[1] = v;
  a.x8[0] = static_cast<uint8_t*>(k8);
  a.x8[1] = static_cast<uint8_t*>(v8);
  a.scales[0] = sk;
  a.scales[1] = sv;
  a.seqlens = seqlens;
  a.new_lens = new_lens;
  a.table = block_table;
  a.cos = rope_cos;
  a.sin = rope_sin;
  for (int i = 0; i < 2; ++i) {
    const long long* st = i == 0 ? k_strides : v_strides;
    a.x_sb[i] = st[0];
    a.x_sh[i] = st[1];
    a.x_sn[i] = st[2];
  }
  a.B = B;
  a.Hkv = Hkv;
  a.n_new = n_new;
  a.rows_max = Nmax;
  a.limit = rope_cos && n_pos < Nmax ? n_pos : Nmax;
  a.blocks = (Nmax + 127) / 128;
  a.pages = num_pages;
  a.rot = rope_cos ? rot_dim : 0;
  a.interleaved = interleaved ? 1 : 0;
  a.status = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_status(dtype == ATTN_BF16 ? launch_append<__nv_bfloat16>(d, a, st) : launch_append<__half>(d, a, st));
}
