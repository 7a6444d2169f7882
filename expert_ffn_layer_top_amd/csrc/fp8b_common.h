// Block-128 E4M3 helpers (device).  A block's largest magnitude amax counts as at least 2^-100 (so an
// all-zero block has finite factors), its codes are E4M3(v * inv) rounded to nearest even with
// inv = 448 / amax rounded to fp32 (448: the largest E4M3 value), and its scale is amax * (1/448)
// rounded to fp32; the value a code stands for is code * scale.  A block that holds an infinity (inv 0, scale
// inf) or a NaN is NaN throughout.
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
  float amax = __uint_as_float(amax_bits << 16);
  amax = amax < 0x1p-100f ? 0x1p-100f : amax;      // (a NaN stays)
  return {448.0f / amax, amax * (1.0f / 448.0f)};
}

// E4M3 codes of four fp32 products v * inv, rounded to nearest even.  No product of a finite block needs a
// clamp: |v| <= amax, and inv and the product are each off by at most 2^-24, so none exceeds 448 (1 + 2^-22),
// which still rounds to 448 (the next border is 464).
__device__ __forceinline__ uint32_t fp8b_encode4(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

// Codes of 8 bf16 values (two per word) times inv.
__device__ __forceinline__ uint2 fp8b_encode8(const uint32_t (&w)[4], float inv) {
  return make_uint2(fp8b_encode4(bf16_lo(w[0]) * inv, bf16_hi(w[0]) * inv, bf16_lo(w[1]) * inv, bf16_hi(w[1]) * inv),
                    fp8b_encode4(bf16_lo(w[2]) * inv, bf16_hi(w[2]) * inv, bf16_lo(w[3]) * inv, bf16_hi(w[3]) * inv));
}

// Magnitudes of bf16 pairs order as 16-bit integers, so a maximum takes both halves of a word at once.
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t abs_pair(uint32_t w) { return w & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t max_of_pair(uint32_t w) { return max(w & 0xffffu, w >> 16); }

// Largest magnitude bits of 8 bf16 values.
__device__ __forceinline__ uint32_t fp8b_amax8(const uint32_t (&w)[4]) {
  return max_of_pair(max_pair(max_pair(abs_pair(w[0]), abs_pair(w[1])), max_pair(abs_pair(w[2]), abs_pair(w[3]))));
}

// Largest value over aligned groups of 16 lanes, in all of them (rotations within the row of 16).
template <int CTRL>
__device__ __forceinline__ uint32_t max_ror(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false)));
}
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  m = max_ror<0x128>(m);
  m = max_ror<0x124>(m);
  m = max_ror<0x122>(m);
  return max_ror<0x121>(m);
}

// Lane I of the row of 16's value, in all 16 lanes.
template <int I>
__device__ __forceinline__ float row_lane(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + I, 0xf, 0xf, false));
}

}  // namespace moe
