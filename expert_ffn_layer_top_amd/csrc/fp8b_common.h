// Block-128 E4M3 helpers (device).  A block's largest magnitude amax counts as at least 2^-100 (so an
// all-zero block has finite factors), its codes are E4M3(v * inv) rounded to nearest even with
// inv = 448 / amax rounded to fp32 (448: the largest E4M3 value), and its scale is amax * (1/448)
// rounded to fp32; the value a code stands for is code * scale.
//
// The product with inv is rounded to fp32 before it is rounded to E4M3's 4 significant bits; the first
// rounding is off by at most 2^-24 of the value, so it moves only values that close to a border.
#pragma once

#include "common.h"

namespace moe {

constexpr int kFp8bBlock = 128;

// ceil(x / 128): blocks along an axis (the last one may be partial).
__host__ __device__ __forceinline__ long long fp8b_blocks(long long x) { return (x + kFp8bBlock - 1) / kFp8bBlock; }

struct Fp8bScale {
  float inv, scale;
};

// From the magnitude bits of a block's bf16 amax.
__device__ __forceinline__ Fp8bScale fp8b_scale(uint32_t amax_bits) {
  const float amax = fmaxf(__uint_as_float(amax_bits << 16), 0x1p-100f);
  return {448.0f / amax, amax * (1.0f / 448.0f)};
}

// E4M3 codes of four fp32 values in [-448, 448] (clamped: v * inv can exceed 448 by a rounding).
__device__ __forceinline__ uint32_t fp8b_encode4(float a, float b, float c, float d) {
  a = __builtin_amdgcn_fmed3f(a, -448.0f, 448.0f);
  b = __builtin_amdgcn_fmed3f(b, -448.0f, 448.0f);
  c = __builtin_amdgcn_fmed3f(c, -448.0f, 448.0f);
  d = __builtin_amdgcn_fmed3f(d, -448.0f, 448.0f);
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

// Codes of 8 bf16 values (two per word) times inv.
__device__ __forceinline__ uint2 fp8b_encode8(const uint32_t (&w)[4], float inv) {
  return make_uint2(fp8b_encode4(bf16_lo(w[0]) * inv, bf16_hi(w[0]) * inv, bf16_lo(w[1]) * inv, bf16_hi(w[1]) * inv),
                    fp8b_encode4(bf16_lo(w[2]) * inv, bf16_hi(w[2]) * inv, bf16_lo(w[3]) * inv, bf16_hi(w[3]) * inv));
}

// Largest magnitude bits of 8 bf16 values.
__device__ __forceinline__ uint32_t fp8b_amax8(const uint32_t (&w)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int h = 0; h < 4; ++h) m = max(m, max(w[h] & 0x7fffu, (w[h] >> 16) & 0x7fffu));
  return m;
}

// Largest value over aligned groups of 16 lanes.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, 64)));
  return m;
}

}  // namespace moe
