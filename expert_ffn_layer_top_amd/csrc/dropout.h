// Dropout factors from a counter-based generator (device): nothing is stored, every kernel that needs the
// factor of an element computes it again.
//
// Element (r, c) of a matrix is dropped when 16 bits u(r, c) are below drop = round(p 2^16) and otherwise
// multiplied by 2^16 / (2^16 - drop).  The 8 elements of an aligned 16-byte chunk of bf16 take the 8 halves of
// one Philox4x32 block (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011) with 7
// rounds, the least that the paper finds to pass every test of its battery, of the counter (c / 8 + site 2^28, r, offset) under
// the seed as the key: a chunk costs 14 full 32 x 32 products, the slow part (quarter rate).  Kernels that read 2
// bytes an element and do little else notice it: the adapters' A x of 131072 rows of 7168 takes 323 us without and 350 to 390
// with dropout (part of it registers that do not fit), their weight gradient of 32768 rows of 2048 27 and 42.
#pragma once

#include "common.h"

namespace moe {

struct DropArgs {
  const int64_t* rng;   // [2]: seed, offset (read by the kernel, so that a replayed graph sees new ones)
  uint32_t drop;        // 0: nothing is dropped
  uint32_t site;
};

struct DropKey {
  uint32_t k0, k1, o0, o1, site, drop;
};

// (Without dropout rng may be null, and is not read.)
__device__ __forceinline__ DropKey drop_key(const DropArgs& a) {
  if (a.drop == 0) return {0, 0, 0, 0, 0, 0};
  const uint64_t s = static_cast<uint64_t>(a.rng[0]), o = static_cast<uint64_t>(a.rng[1]);
  return {static_cast<uint32_t>(s), static_cast<uint32_t>(s >> 32), static_cast<uint32_t>(o),
          static_cast<uint32_t>(o >> 32), a.site << 28, a.drop};
}

// 2^16 / (2^16 - drop).
__host__ __device__ __forceinline__ float drop_scale(uint32_t drop) { return 65536.0f / static_cast<float>(65536u - drop); }

// a ^ b ^ c in one instruction.
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

// The 8 pieces of 16 bits of chunk `chunk` of row `row`: elements 2i and 2i + 1 are the low and high half of word i.
__device__ __forceinline__ uint4 drop_bits(const DropKey& key, uint32_t row, uint32_t chunk) {
  uint32_t c0 = chunk | key.site, c1 = row, c2 = key.o0, c3 = key.o1, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t m0 = static_cast<uint64_t>(c0) * 0xD2511F53u, m1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = xor3(static_cast<uint32_t>(m1 >> 32), c1, k0);
    c2 = xor3(static_cast<uint32_t>(m0 >> 32), c3, k1);
    c1 = static_cast<uint32_t>(m1);
    c3 = static_cast<uint32_t>(m0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The chunk's 8 fp32 values, each times its factor (a dropped one is 0 whatever it was).
__device__ __forceinline__ void drop_apply(const DropKey& key, uint32_t row, uint32_t chunk, float scale, float (&f)[8]) {
  const uint4 b = drop_bits(key, row, chunk);
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = (w[i] & 0xffffu) >= key.drop ? f[2 * i] * scale : 0.f;
    f[2 * i + 1] = (w[i] >> 16) >= key.drop ? f[2 * i + 1] * scale : 0.f;
  }
}

// The chunk's 8 bf16 values with the dropped ones 0, the others as they are (the factor is left to the caller).
typedef uint32_t drop_u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ drop_u32x4 drop_zero(const DropKey& key, uint32_t row, uint32_t chunk, drop_u32x4 v) {
  // two 16-bit pieces at a time: min(max(u - (drop - 1), 0), 1) is 1 where u >= drop (drop > 0 here)
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const uint4 b = drop_bits(key, row, chunk);
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
  const unsigned short below = static_cast<unsigned short>(key.drop - 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u16x2 over = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, w[i]), u16x2{below, below});
    const u16x2 keep = __builtin_elementwise_min(over, u16x2{1, 1});
    const uint32_t x = v[i];
    v[i] = __builtin_bit_cast(uint32_t, static_cast<u16x2>(__builtin_bit_cast(u16x2, x) * keep));
  }
  return v;
}

// Host: the arguments of a call, checked.  p is rounded to a multiple of 2^-16; p = 0 needs no rng.
int make_drop(const int64_t* rng, float p, int site, DropArgs* out);

}  // namespace moe
