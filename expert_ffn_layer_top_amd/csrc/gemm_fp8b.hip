// Device-scheduled grouped GEMMs of the SwiGLU expert FFN on E4M3 codes with one fp32 scale per block
// of 128 along the contraction dimension, forward and backward, on the fp8 matrix cores
// (v_mfma_f32_16x16x128_f8f6f4: one instruction contracts exactly one block), or, for few rows, on the bf16 ones.
//
//   out[r][c] = sum over blocks b of  sa[b][r] * sb * sum over k in b of qa[r][k] qb[c][k]
//
// sb is one value per 128 x 128 block of a weight matrix (forward and dgrad products), or one per
// column and block (weight gradients, where both operands are blocks of 128 tokens).  A block's sum
// comes out of the matrix core in fp32 and is scaled into the running sum by fp32 FMAs; the result is rounded
// to bf16 once.  On the way there the fp8 core cuts: it adds aligned groups of 8 products along K and keeps of each
// the multiples of 2^(E - 13), E the largest sum of two operands' exponents in its group, which leaves a block's sum with an
// rms error of 2^-16 of its size (y 0.21% off, 0.17% with exact sums).  The bf16 core does not; where it runs is
// at exact_rows and grouped_skinny.
//
// Products and operands (all codes K-contiguous):
//   FWD1   xq [n][d]           x  W_gate, W_up [f][d]               -> G, U, A = silu(G) U
//   FWD2   aq [n][f]           x  W_down [d][f]                     -> Yexp
//   DGRAD1 dyq [n][d]          x  W_down^T [f][d]                   -> dG, dU (SwiGLU backward)
//   DGRAD2 dgq | duq [n][f]    x  W_gate^T | W_up^T [d][f]          -> dXp   (two contractions, one sum)
//   WGRAD_DOWN  dy^T [d][P]    x  a^T [f][P]                        -> dW_down[e]
//   WGRAD_GU    dg^T | du^T [f][P]  x  x^T [d][P]                   -> dW_gate[e], dW_up[e]
// where P is the padded token axis: expert e owns positions [offsets_pad[e], offsets_pad[e + 1]), whole
// blocks of 128 inside it.  An expert whose offsets say otherwise (another pad) has NaN gradients.
//
// Tile: 256 x 256 outputs per workgroup of eight waves, 64 rows x 128 columns each (two waves per
// SIMD).  The running sums must be plain vector registers, since vector instructions cannot use
// accumulation registers as operands: 128 of a wave's 256, which is why the waves are half the size of
// the MXFP8 kernel's, whose scales the matrix core applies.  While one wave's FMAs run (4 per MFMA), the
// other's MFMAs keep the matrix core busy.  K steps of 128 go through a two-stage LDS ring filled by
// LDS-DMA loads, XOR-swizzled 16-byte chunks, one barrier per step; the steps of a workgroup's tiles
// form one stream.  Lane l of a fragment holds row l % 16, bytes 16 (l / 16) .. + 15 and
// 64 + 16 (l / 16) .. + 15 of the step (any order serves, being the same for both operands); the product
// takes columns from the first operand, so a lane ends with 4 consecutive columns of one row and
// needs one row scale per 16 x 16 tile.
//
// Measured, 131072 rows of 64 experts, d 7168, f 2048, ms: gate/up 3.7 (4.0 after a pause), down 1.95, dgrad down 2.1, dgrad
// gate/up 3.7, wgrad down 2.2, wgrad gate/up 4.4, which is 1.7 to 2.1 PFLOP/s (a large library fp8 product with one scale
// for all: 2.7 to 3.1).  What bounds it: the matrix core is busy 54 to 56% of the cycles of the forward products and of dgrad
// gate/up, at 1.9 GHz.  An MFMA takes a SIMD 32 cycles and comes with 5.2 to 5.4 other vector instructions of 4 cycles (4 of
// them its FMAs); a SIMD spends 57 to 60 cycles per MFMA, little less than one after the other, although two waves
// share it.  A weight gradient's MFMA has 9.2 (each output's weight is a product of its own, sb sa) and takes 70: 45% busy.
// dgrad down, with the SwiGLU backward in its epilogue, has 5.9 and takes 69.  Leaving parts of the work out, each
// against the whole kernel of the same run: no FMAs -7%, no epilogue -7% (down -12%, dgrad down -20%, weight gradients -9%), loads
// that always hit the first-level cache -20%, column fragments not read from LDS -3%; all codes zero -10%.  Tried
// without gain: a load that touches the lines of the step after next (10% slower), a
// higher priority for half of the waves or for the MFMAs, stores left in flight over the next tile's first step.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <type_traits>

#include "common.h"
#include "fp8b_common.h"
#include "gemm_epilogue.h"
#include "gemm_sched.h"

namespace moe {
namespace g8b {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int BM = 256;
constexpr int BN = 256;
constexpr int BK = 128;                            // codes (bytes) per K step = one scale block
constexpr int NTH = 512;
constexpr int OP_BYTES = BM * BK;                  // 32 KiB per operand per stage
constexpr int SC_BYTES = BM * 4;                   // one scale per row per stage
constexpr int A_RING = 0;
constexpr int B_RING = 2 * OP_BYTES;
constexpr int SA_RING = 4 * OP_BYTES;
constexpr int SB_RING = SA_RING + 2 * SC_BYTES;
constexpr int LDS_TOTAL = SB_RING + 2 * SC_BYTES;  // 132 KiB
constexpr int STG_BYTES = 2 * OP_BYTES / 8;        // epilogue staging per wave, in the stage just consumed

__shared__ __attribute__((aligned(1024))) uint8_t lds_ring[LDS_TOTAL];
__shared__ int tile_map[256];                      // row tiles before each expert's

__device__ __forceinline__ uint32_t lds_addr(const uint8_t* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_u8*)(p)));
}

enum Mode { FWD1 = 0, FWD2 = 1, DGRAD1 = 2, DGRAD2 = 3, WGRAD_DOWN = 4, WGRAD_GU = 5 };

struct Params {
  int cm, cn;                   // tile order: cells of cm m-tiles x cn n-tiles
  const int32_t* offsets;
  const int32_t* offsets_pad;   // WGRAD: padded token offsets
  int E, n, d, f;
  int P;                        // WGRAD: length of the padded token axis
  const uint8_t* a0; const float* a0s;
  const uint8_t* a1; const float* a1s;
  const uint8_t* b0; const float* b0s;
  const uint8_t* b1; const float* b1s;
  const uint16_t* g;
  const uint16_t* u;
  uint16_t* o0;
  uint16_t* o1;
  uint16_t* o2;
};

template <int B, int E, class F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    static_for<B + 1, E>(f);
  }
}

constexpr bool is_wgrad(int mode) { return mode >= WGRAD_DOWN; }

// Row r (128 bytes = 8 chunks of 16), chunk c stored at position c ^ ((r >> 1) & 7).
__device__ __forceinline__ int kc_off(int r, int c) { return r * 128 + ((c ^ ((r >> 1) & 7)) << 4); }

struct Tile {
  int e, m0, m_end, n0, half;
  int k_begin;   // WGRAD: first padded token position of the expert
  int k_len;     // WGRAD: its padded tokens (-1: no whole blocks of the axis)
};

template <int MODE>
__host__ __device__ __forceinline__ int n_total(int d, int f) {
  return (MODE == FWD1 || MODE == DGRAD1 || MODE == WGRAD_DOWN) ? f : d;
}
template <int MODE>
__host__ __device__ __forceinline__ int n_tile_width() { return MODE == FWD1 ? BN / 2 : BN; }
// contraction length of one operand (DGRAD2 runs two of them); the padded tokens for weight gradients
template <int MODE>
__host__ __device__ __forceinline__ int k_one(int d, int f) { return (MODE == FWD1 || MODE == DGRAD1) ? d : f; }
template <int MODE>
__host__ __device__ __forceinline__ int m_total(int d, int f) { return MODE == WGRAD_DOWN ? d : f; }

using gsched::MTiles;

// The row tiles before each expert's, kept in LDS (in registers they spilled others): every wave writes all
// of it, the same values, and so reads back its own.  Returns the number of row tiles.
__device__ __forceinline__ int store_map(const Params& p) {
  const MTiles m = gsched::mtile_scan<BM>(p.offsets, p.E);
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < 4; ++r) tile_map[64 * r + lane] = 64 * r + lane < p.E ? m.excl[r] : INT32_MAX;
  return m.total;
}
// The expert that owns row tile mt: the last one with at most mt tiles before it (`first` of them).
__device__ __forceinline__ int map_find(int mt, int& first) {
  const int lane = threadIdx.x & 63;
  int count = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) count += __popcll(__ballot(tile_map[64 * r + lane] <= mt));
  first = tile_map[count - 1];
  return count - 1;
}

// Expert t.e's range of the padded token axis.  Offsets of a pad that the axis has no room for, or that splits
// blocks, can only be seen here, on the device; nothing is read through them.
__device__ __forceinline__ void token_range(const Params& p, Tile& t) {
  const int begin = p.offsets_pad[t.e], end = p.offsets_pad[t.e + 1];
  const bool whole = ((begin | end) & (BK - 1)) == 0 && 0 <= begin && begin <= end && end <= p.P;
  t.k_begin = __builtin_amdgcn_readfirstlane(whole ? begin : 0);
  t.k_len = __builtin_amdgcn_readfirstlane(whole ? end - begin : -1);
}

// What a tile's sums start from.
template <int MODE>
__device__ __forceinline__ float start_value(const Tile& t) {
  return is_wgrad(MODE) && t.k_len < 0 ? __builtin_nanf("") : 0.f;
}

// The tile with linear id `lid`: each expert owns a contiguous run of ids, its tiles in cell order.
template <int MODE>
__device__ __forceinline__ Tile tile_at(const Params& p, int ntiles_n, int lid) {
  Tile t{};
  int mi, nt;
  if constexpr (!is_wgrad(MODE)) {
    int first;
    const int e = __builtin_amdgcn_readfirstlane(map_find(lid / ntiles_n, first));
    first = __builtin_amdgcn_readfirstlane(first);
    const int r0 = p.offsets[e], r1 = p.offsets[e + 1];
    gsched::cell_order(lid - first * ntiles_n, (r1 - r0 + BM - 1) / BM, ntiles_n, p.cm, p.cn, mi, nt);
    t.e = e;
    t.m0 = r0 + mi * BM;
    t.m_end = r1;
  } else {
    const int Mtot = m_total<MODE>(p.d, p.f);
    const int mt = (Mtot + BM - 1) / BM, rows = mt * (MODE == WGRAD_GU ? 2 : 1);
    t.e = lid / (rows * ntiles_n);
    gsched::cell_order(lid - t.e * rows * ntiles_n, rows, ntiles_n, p.cm, p.cn, mi, nt);
    t.half = mi >= mt ? 1 : 0;
    t.m0 = (mi - t.half * mt) * BM;
    t.m_end = Mtot;
    token_range(p, t);
  }
  t.n0 = nt * n_tile_width<MODE>();
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
  t.m_end = __builtin_amdgcn_readfirstlane(t.m_end);
  t.n0 = __builtin_amdgcn_readfirstlane(t.n0);
  t.half = __builtin_amdgcn_readfirstlane(t.half);
  return t;
}

// One wave's DMA sources of a tile: the codes' descriptor, bounded to the operand's extent (r1: the
// second operand of DGRAD2), and where its row scales start (block 0, this tile's first row; row
// scales of block b are `pitch` floats further each, and `rows` of them exist).
struct TileSrc {
  __amdgpu_buffer_rsrc_t r0, r1;
  const float* s0;
  const float* s1;
  int rows;
  int nk;   // K steps
};

template <int MODE>
__device__ __forceinline__ TileSrc empty_src(const Params& p) {
  TileSrc s{};
  s.r0 = gep::rsrc(p.a0, 0);
  s.r1 = s.r0;
  s.s0 = p.a0s;
  s.s1 = p.a0s;
  return s;
}

template <int MODE>
__device__ __forceinline__ TileSrc tile_src(const Params& p, const Tile& t, bool role_b, int h) {
  TileSrc s{};
  const int Kone = k_one<MODE>(p.d, p.f);
  if constexpr (is_wgrad(MODE)) {
    s.nk = max(t.k_len, 0) / BK;
    const int C = role_b ? n_total<MODE>(p.d, p.f) : m_total<MODE>(p.d, p.f);
    const int c0 = role_b ? t.n0 : t.m0;
    const uint8_t* base = role_b ? p.b0 : (MODE == WGRAD_GU && t.half ? p.a1 : p.a0);
    const float* sbase = role_b ? p.b0s : (MODE == WGRAD_GU && t.half ? p.a1s : p.a0s);
    s.r0 = gep::rsrc(base + static_cast<long long>(c0) * p.P + t.k_begin, static_cast<long long>(C - c0) * p.P - t.k_begin);
    s.r1 = s.r0;
    s.s0 = sbase + static_cast<long long>(t.k_begin / BK) * C + c0;
    s.s1 = s.s0;
    s.rows = C - c0;
  } else {
    s.nk = static_cast<int>(fp8b_blocks(Kone)) * (MODE == DGRAD2 ? 2 : 1);
    if (!role_b) {
      const long long rows = static_cast<long long>(p.n) - t.m0;
      s.r0 = gep::rsrc(p.a0 + static_cast<long long>(t.m0) * Kone, rows * Kone);
      s.s0 = p.a0s + t.m0;
      s.r1 = s.r0;
      s.s1 = s.s0;
      if constexpr (MODE == DGRAD2) {
        s.r1 = gep::rsrc(p.a1 + static_cast<long long>(t.m0) * Kone, rows * Kone);
        s.s1 = p.a1s + t.m0;
      }
      s.rows = static_cast<int>(rows);
    } else {
      const int N = n_total<MODE>(p.d, p.f);
      const long long off = (static_cast<long long>(t.e) * N + t.n0) * Kone;
      const long long bytes = static_cast<long long>(N - t.n0) * Kone;
      s.r0 = gep::rsrc((MODE == FWD1 && h >= 2 ? p.b1 : p.b0) + off, bytes);
      s.r1 = s.r0;
      if constexpr (MODE == DGRAD2) s.r1 = gep::rsrc(p.b1 + off, bytes);
      s.s0 = p.a0s;
      s.s1 = p.a0s;
    }
  }
  return s;
}

// Scale of the weight block that K block kb (of operand half `half`) and the tile's columns from
// `col` on belong to; lane l asks for block kb + l.  Columns and blocks past the matrix read a
// neighbour's scale, which only meets codes that read as zero.
template <int MODE>
__device__ __forceinline__ float weight_scale(const Params& p, const Tile& t, int col, int half, int kb) {
  if constexpr (is_wgrad(MODE)) return 0.f;
  const int N = n_total<MODE>(p.d, p.f);
  const int nb = static_cast<int>(fp8b_blocks(N)), kbs = static_cast<int>(fp8b_blocks(k_one<MODE>(p.d, p.f)));
  const int c = min(col / kFp8bBlock, nb - 1);
  const int k = min(kb + static_cast<int>(threadIdx.x & 63), kbs - 1);
  const float* s = half ? p.b1s : p.b0s;
  return s[(static_cast<long long>(t.e) * nb + c) * kbs + k];
}

template <int OFF>
__device__ __forceinline__ void ds_b128(i32x4& v, uint32_t addr) {
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
}
template <int OFF>
__device__ __forceinline__ void ds_f128(f32x4& v, uint32_t addr) {
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
}
template <int OFF>
__device__ __forceinline__ void ds_f32(float& v, uint32_t addr) {
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
}

// Fragment Q (16 rows): both 16-byte chunks of this lane.
template <int Q>
__device__ __forceinline__ void read_frag(i32x8& v, uint32_t a0, uint32_t a1) {
  i32x4 lo, hi;
  ds_b128<2048 * Q>(lo, a0);
  ds_b128<2048 * Q>(hi, a1);
  v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Waits until at most N LDS reads are outstanding and ties the registers that have then landed.
template <int N>
__device__ __forceinline__ void wait_first(i32x8& b, i32x8& a) {
  asm volatile("s_waitcnt lgkmcnt(%2)" : "+v"(b), "+v"(a) : "n"(N));
}
template <int N>
__device__ __forceinline__ void wait_scales(float (&s)[4]) {
  asm volatile("s_waitcnt lgkmcnt(%4)" : "+v"(s[0]), "+v"(s[1]), "+v"(s[2]), "+v"(s[3]) : "n"(N));
}
template <int N>
__device__ __forceinline__ void wait_col(i32x8& b) {
  asm volatile("s_waitcnt lgkmcnt(%1)" : "+v"(b) : "n"(N));
}
template <int N>
__device__ __forceinline__ void wait_col(i32x8& b, f32x4& sb) {
  asm volatile("s_waitcnt lgkmcnt(%2)" : "+v"(b), "+v"(sb) : "n"(N));
}

__device__ __forceinline__ f32x4 mfma_block(const i32x8& x, const i32x8& y) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 codes of a fragment (dwords 2 I and 2 I + 1) as bf16.
template <int I>
__device__ __forceinline__ bf16x8 codes_bf16(const i32x8& v) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * I], 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * I], 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * I + 1], 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * I + 1], 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The same block sums, exact to fp32: every E4M3 value is a bf16 one, and the bf16 matrix core keeps what the fp8
// one cuts off beside a larger product (rms error of a sum 2^-27 of its size instead of 2^-16).
__device__ __forceinline__ f32x4 exact_block(const i32x8& x, const i32x8& y) {
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  static_for<0, 4>([&](auto h) { sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16<h>(x), codes_bf16<h>(y), sum, 0, 0, 0); });
  return sum;
}

// One K step of a wave: 64 rows (four fragments at a0, a1) by NF column fragments (at b0, b1; FWD1: the first
// half are the gate's, the others the up matrix's, from fragment UP on), its scaled block sums added to acc.
// `next` issues all loads of the step after, behind the first MFMAs (spread over the step, 5% more time: the
// last of them had an eighth of it to arrive).
template <int MODE, int NF, int UP, bool EXACT, class F>
__device__ __forceinline__ void multiply_step(f32x4 (&acc)[NF][4], uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1,
                                              uint32_t sa_at, uint32_t sb_at, float ws0, float ws1, F&& next) {
  constexpr bool WG = is_wgrad(MODE);
  i32x8 fa[4], fb[2];
  float sa[4], ca[4], cb[4];
  f32x4 sb[3], tmp[4];               // sb: column scales of the fragments i - 1 (whose sums are in tmp), i and i + 1
  auto col_frag = [&](auto i) {
    constexpr int q = MODE == FWD1 && i >= NF / 2 ? i - NF / 2 + UP : i;
    read_frag<q>(fb[i & 1], b0, b1);
    if constexpr (WG && i > 0) ds_f128<64 * i>(sb[i % 3], sb_at);
  };
  // reads return in order: the first MFMA starts on the first two fragments, the others follow as they come
  col_frag(std::integral_constant<int, 0>{});
  static_for<0, 4>([&](auto j) { read_frag<j>(fa[j], a0, a1); });
  static_for<0, 4>([&](auto j) { ds_f32<64 * j>(sa[j], sa_at); });
  if constexpr (WG) ds_f128<0>(sb[0], sb_at);
  static_for<0, NF>([&](auto i) {
    constexpr int after = i + 1 < NF ? (WG ? 3 : 2) : 0;     // reads of the next fragment
    if constexpr (i + 1 < NF) col_frag(std::integral_constant<int, i + 1>{});
    if constexpr (i > 0) {
      if constexpr (WG) wait_col<after>(fb[i & 1], sb[i % 3]);
      else wait_col<after>(fb[i & 1]);
    }
    if constexpr (i == 1) {
      wait_scales<after>(sa);
      if constexpr (WG) asm volatile("" : "+v"(sb[0]));       // has landed with them
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ca[j] = WG ? sa[j] : sa[j] * ws0;
        cb[j] = MODE == FWD1 ? sa[j] * ws1 : 0.f;
      }
    }
    // a block sum enters the running sum just before its register takes the next fragment's, three MFMAs after
    // its own was issued
    auto add = [&](auto ii, auto j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = WG ? sb[ii % 3][e] * sa[j] : (MODE == FWD1 && ii >= NF / 2 ? cb[j] : ca[j]);
        acc[ii][j][e] = fmaf(tmp[j][e], w, acc[ii][j][e]);
      }
    };
    static_for<0, 4>([&](auto j) {
      if constexpr (i > 0) add(std::integral_constant<int, i - 1>{}, j);
      if constexpr (i == 0) wait_first<after + (WG ? 5 : 4) + 2 * (3 - j)>(fb[0], fa[j]);
      tmp[j] = EXACT ? exact_block(fb[i & 1], fa[j]) : mfma_block(fb[i & 1], fa[j]);
      __builtin_amdgcn_sched_barrier(0);   // the compiler would pull the FMAs up to their MFMA and wait there
      if constexpr (i == 0 && j == 3) { next(); __builtin_amdgcn_sched_barrier(0); }
    });
    if constexpr (i == NF - 1) static_for<0, 4>([&](auto j) { add(i, j); });
  });
}

// Writes the tile's results, staged through this wave's 8 KiB of the stage just consumed.
template <int MODE>
__device__ __forceinline__ void epilogue(const Params& p, const Tile& t, f32x4 (&acc)[8][4], int wm, int wn, int lane,
                                         uint32_t stg) {
  using gep::u32x2;
  using gep::u32x4;
  const int row0 = t.m0 + 64 * wm;
  const int rows_valid = t.m_end - row0;
  if constexpr (MODE == FWD1) {
    const int col0 = t.n0 + 64 * wn, cv = p.f - col0;
    auto store = [&](uint16_t* out, auto&& val) {
      const auto r = gep::out_rsrc(out, p.n, p.f, row0, col0);
      gep::sfor<0, 2>([&](auto q) {
        u32x2 v[2][4];
        gep::sfor<0, 2>([&](auto jj) { gep::sfor<0, 4>([&](auto i) { v[jj][i] = val(i, std::integral_constant<int, 2 * q + jj>{}); }); });
        gep::stage_out_round<4, 2>(v, q, r, rows_valid, cv, p.f, stg, lane);
      });
    };
    if (p.o0 != nullptr) {
      store(p.o0, [&](auto i, auto j) { return gep::pack4(acc[i][j]); });
      store(p.o1, [&](auto i, auto j) { return gep::pack4(acc[i + 4][j]); });
    }
    store(p.o2, [&](auto i, auto j) {
      f32x4 av;
#pragma unroll
      for (int e = 0; e < 4; ++e) av[e] = acc[i][j][e] * gep::sigmoid(acc[i][j][e]) * acc[i + 4][j][e];
      return gep::pack4(av);
    });
  } else if constexpr (MODE == DGRAD1) {
    const int col0 = t.n0 + 128 * wn, cv = p.f - col0;
    const auto rg = gep::out_rsrc(p.g, p.n, p.f, row0, col0), ru = gep::out_rsrc(p.u, p.n, p.f, row0, col0);
    const auto rdg = gep::out_rsrc(p.o0, p.n, p.f, row0, col0), rdu = gep::out_rsrc(p.o1, p.n, p.f, row0, col0);
    // (8-byte loads straight into the product's layout, a round ahead, ran the product 13% slower)
    u32x4 gl[4], ul[4];
    gep::load_rows<1>(rg, std::integral_constant<int, 0>{}, rows_valid, cv, p.f, lane, gl);
    gep::load_rows<1>(ru, std::integral_constant<int, 0>{}, rows_valid, cv, p.f, lane, ul);
    gep::sfor<0, 4>([&](auto q) {
      u32x2 gm[1][8], um[1][8];
      gep::stage_in_round<1>(gl, gm, stg, lane);
      gep::stage_in_round<1>(ul, um, stg, lane);
      if constexpr (q < 3) {                     // the next round's, on their way while this one's are used
        gep::load_rows<1>(rg, std::integral_constant<int, q + 1>{}, rows_valid, cv, p.f, lane, gl);
        gep::load_rows<1>(ru, std::integral_constant<int, q + 1>{}, rows_valid, cv, p.f, lane, ul);
      }
      gep::sfor<0, 8>([&](auto i) {
        const u32x2 g2 = gm[0][i], u2 = um[0][i];
        const float gv[4] = {bf16_lo(g2.x), bf16_hi(g2.x), bf16_lo(g2.y), bf16_hi(g2.y)};
        const float uv[4] = {bf16_lo(u2.x), bf16_hi(u2.x), bf16_lo(u2.y), bf16_hi(u2.y)};
        float dgv[4], duv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float da = acc[i][q][e], sg = gep::sigmoid(gv[e]);
          dgv[e] = da * uv[e] * sg * (1.0f + gv[e] * (1.0f - sg));
          duv[e] = da * gv[e] * sg;
        }
        gm[0][i] = u32x2{pack_bf16x2(dgv[0], dgv[1]), pack_bf16x2(dgv[2], dgv[3])};
        um[0][i] = u32x2{pack_bf16x2(duv[0], duv[1]), pack_bf16x2(duv[2], duv[3])};
      });
      gep::stage_out_round<8, 1>(gm, q, rdg, rows_valid, cv, p.f, stg, lane);
      gep::stage_out_round<8, 1>(um, q, rdu, rows_valid, cv, p.f, stg, lane);
    });
  } else {
    const int N = n_total<MODE>(p.d, p.f);
    const int col0 = t.n0 + 128 * wn, cv = N - col0;
    uint16_t* out = p.o0;
    long long rows = p.n;
    if constexpr (is_wgrad(MODE)) {
      rows = m_total<MODE>(p.d, p.f);
      out = (MODE == WGRAD_GU && t.half ? p.o1 : p.o0) + static_cast<long long>(t.e) * rows * N;
    }
    const auto r = gep::out_rsrc(out, rows, N, row0, col0);
    gep::sfor<0, 4>([&](auto q) {
      u32x2 v[1][8];
      gep::sfor<0, 8>([&](auto i) { v[0][i] = gep::pack4(acc[i][q]); });
      gep::stage_out_round<8, 1>(v, q, r, rows_valid, cv, N, stg, lane);
    });
  }
}

// Where a K step is read from: codes and row scales, its byte offset in a row, and the bytes of the row
// from there on (TAIL: the contraction length is no multiple of 128, and the last step's rest reads zero).
struct Step {
  __amdgpu_buffer_rsrc_t r, rs;
  int soff, left;
};

template <int MODE, bool TAIL>
__device__ __forceinline__ void grouped_gemm(const Params& p) {
  constexpr bool WG = is_wgrad(MODE);
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const bool role_b = wave < 4;    // waves 0-3 stream the column operand, 4-7 the row operand
  const int h = wave & 3;          // 64 rows each

  // ---- device-side schedule (as the MXFP8 products)
  constexpr int NTW = MODE == FWD1 ? BN / 2 : BN;
  const int ntiles_n = (n_total<MODE>(p.d, p.f) + NTW - 1) / NTW;
  int total;
  bool deal = false;
  if constexpr (!WG) {
    total = store_map(p) * ntiles_n;
  } else {
    total = p.E * ((m_total<MODE>(p.d, p.f) + BM - 1) / BM) * (MODE == WGRAD_GU ? 2 : 1) * ntiles_n;
    deal = gsched::wgrad_skewed(p.offsets, p.E, p.n);
  }
  const int G = gridDim.x;   // a multiple of 8
  const int bid = blockIdx.x;
  int lid, lstep, lend;
  if (deal) {
    lid = bid;
    lstep = G;
    lend = total;
  } else {
    const int per = (total + 7) >> 3;
    const int x = bid & 7;
    lid = x * per + (bid >> 3);
    lstep = G >> 3;
    lend = (x + 1) * per < total ? (x + 1) * per : total;
  }
  lid = __builtin_amdgcn_readfirstlane(lid);
  lend = __builtin_amdgcn_readfirstlane(lend);
  if (lid >= lend) return;
  int rn = 1;
  auto deal_lid = [&](int r) { return r * G + ((r & 1) ? (G - 1 - bid) : bid); };
  int lid_n = deal ? deal_lid(1) : lid + lstep;

  const int Kone = k_one<MODE>(p.d, p.f);
  const int kb_one = static_cast<int>(fp8b_blocks(Kone));
  const int ld = WG ? p.P : Kone;                    // bytes per operand row
  const int spitch = WG ? (role_b ? n_total<MODE>(p.d, p.f) : m_total<MODE>(p.d, p.f)) : p.n;

  Tile t = tile_at<MODE>(p, ntiles_n, lid);
  TileSrc cur = tile_src<MODE>(p, t, role_b, h);
  Tile tn = t;
  TileSrc nxt = empty_src<MODE>(p);
  // weight scales: lane l of w0 holds K block l's (w1: of the up product / of the second contraction)
  const int wcol = MODE == FWD1 ? 0 : 128 * wn;
  float w0 = weight_scale<MODE>(p, t, t.n0 + wcol, 0, 0), w1 = 0.f, w0n = 0.f, w1n = 0.f;
  if constexpr (MODE == FWD1 || MODE == DGRAD2) w1 = weight_scale<MODE>(p, t, t.n0 + wcol, 1, 0);
  auto look_ahead = [&]() {
    tn = tile_at<MODE>(p, ntiles_n, lid_n);
    nxt = tile_src<MODE>(p, tn, role_b, h);
    w0n = weight_scale<MODE>(p, tn, tn.n0 + wcol, 0, 0);
    if constexpr (MODE == FWD1 || MODE == DGRAD2) w1n = weight_scale<MODE>(p, tn, tn.n0 + wcol, 1, 0);
  };
  if (lid_n < lend) look_ahead();

  // DMA: instruction i covers rows 64 h + 8 i + lane / 8 of the operand's 256 (FWD1's column operand:
  // rows of the gate's or the up matrix's 128), chunk position lane % 8
  const int row_h = (MODE == FWD1 && role_b) ? 64 * (h & 1) : 64 * h;
  const int chunk = (lane & 7) ^ (lane >> 4);        // of even instructions; odd ones: chunk ^ 4
  const int vo = (row_h + (lane >> 3)) * ld + 16 * chunk;
  const int vo_odd = (row_h + (lane >> 3)) * ld + 16 * (chunk ^ 4);
  uint8_t* const dst0 = lds_ring + (role_b ? B_RING : A_RING) + h * 8192;
  uint8_t* const sdst0 = lds_ring + (role_b ? SB_RING : SA_RING) + h * 256;

  auto step_of = [&](const TileSrc& s, int k) {
    Step st{s.r0, s.r0, k * BK, BK};
    const float* sc = s.s0;
    int kb = k;
    if constexpr (MODE == DGRAD2) {
      if (k >= kb_one) { st.r = s.r1; sc = s.s1; kb = k - kb_one; st.soff = kb * BK; }
    }
    if constexpr (TAIL) st.left = Kone - st.soff;
    if (k >= s.nk) { st.r = gep::rsrc(p.a0, 0); st.soff = 0; }
    const bool scales = (WG || !role_b) && k < s.nk;
    st.rs = gep::rsrc(sc + static_cast<long long>(kb) * spitch, scales ? 4LL * s.rows : 0);
    return st;
  };
  auto issue = [&](auto i, const Step& st, uint8_t* dst) {
    int off = (i & 1) ? vo_odd : vo;
    asm volatile("" : "+v"(off));      // added up here each time: kept, the eight offsets spilled other registers
    off += 8 * i * ld;
    if constexpr (TAIL) off = 16 * ((i & 1) ? chunk ^ 4 : chunk) < st.left ? off : static_cast<int>(gep::OOB);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(st.r, (lds_void*)(dst + i * 1024), 16, off, st.soff, 0, 0);
  };
  auto issue_scales = [&](const Step& st, uint8_t* dst) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(st.rs, (lds_void*)dst, 4, 4 * (64 * h + lane), 0, 0, 0);
  };

  const uint32_t ring = lds_addr(lds_ring);
  const uint32_t kc0 = kc_off(lane & 15, lane >> 4), kc1 = kc_off(lane & 15, 4 + (lane >> 4));
  const uint32_t a_off = A_RING + wm * 8192;
  const uint32_t b_off = B_RING + (MODE == FWD1 ? 8192 * wn : 16384 * wn);
  const uint32_t sa_off = SA_RING + 4 * (64 * wm + (lane & 15));
  const uint32_t sb_off = SB_RING + 4 * (128 * wn + 4 * (lane >> 4));

  f32x4 acc[8][4];
  auto start_acc = [&]() {
    const float v = start_value<MODE>(t);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{v, v, v, v};
  };
  start_acc();
  int st = 0, kt = 0;
  bool ready = false;
  for (;;) {
    if (!ready && cur.nk > 0) {
      const Step s0 = step_of(cur, 0);
      static_for<0, 8>([&](auto i) { issue(i, s0, dst0 + st * OP_BYTES); });
      if (WG || !role_b) issue_scales(s0, sdst0 + st * SC_BYTES);
      ready = true;
    }
    bool next_ready = false;
    while (kt < cur.nk) {
      // step kt is in LDS everywhere, and every wave is done with step kt - 1, whose stage takes the next
      asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
      const bool here = kt + 1 < cur.nk;
      next_ready = !here && nxt.nk > 0;
      const Step ns = here ? step_of(cur, kt + 1) : step_of(nxt, 0);
      // this step's weight scales (each 64 K blocks the registers are filled again)
      float ws0 = 1.f, ws1 = 1.f;
      if constexpr (!WG) {
        const bool second = MODE == DGRAD2 && kt >= kb_one;
        const int kb = second ? kt - kb_one : kt;
        if (kb >= 64 && (kb & 63) == 0) {
          if (MODE != DGRAD2 || !second) w0 = weight_scale<MODE>(p, t, t.n0 + wcol, 0, kb);
          if (MODE == FWD1 || second) w1 = weight_scale<MODE>(p, t, t.n0 + wcol, 1, kb);
        }
        ws0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(second ? w1 : w0), kb & 63));
        if constexpr (MODE == FWD1) ws1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w1), kb & 63));
      }
      const uint32_t so = ring + st * OP_BYTES, sso = ring + st * SC_BYTES;
      const uint32_t fa0 = so + a_off + kc0, fa1 = so + a_off + kc1, fb0 = so + b_off + kc0, fb1 = so + b_off + kc1;
      uint8_t* const dst = dst0 + (st ^ 1) * OP_BYTES;
      multiply_step<MODE, 8, 8, false>(acc, fa0, fa1, fb0, fb1, sso + sa_off, sso + sb_off, ws0, ws1, [&]() {
        if (WG || !role_b) issue_scales(ns, sdst0 + (st ^ 1) * SC_BYTES);
        static_for<0, 8>([&](auto i) { issue(i, ns, dst); });
      });
      st ^= 1;
      ++kt;
    }
    // ---- tile done (or empty): once every wave has read the last step, its stage serves as staging
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const uint32_t spent = ring + (st ^ 1) * OP_BYTES + (wave < 4 ? A_RING : B_RING) + (wave & 3) * STG_BYTES;
    epilogue<MODE>(p, t, acc, wm, wn, lane, spent);
    if (lid_n >= lend) break;
    ready = next_ready;
    t = tn;
    start_acc();
    cur = nxt;
    w0 = w0n;
    w1 = w1n;
    kt = 0;
    lid_n = deal ? deal_lid(++rn) : lid_n + lstep;
    if (lid_n < lend) look_ahead();
    else nxt = empty_src<MODE>(p);
  }
  // no LDS-DMA may still be writing when the workgroup ends
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}

template <int MODE, bool TAIL>
__global__ __launch_bounds__(NTH, 2) void grouped_gemm_fp8b_kernel(Params p) {
  grouped_gemm<MODE, TAIL>(p);
}

// Tile cells per product, as measured for the MXFP8 products of the same tile and operand bytes.  On these kernels, at the
// size above, cells of 1 x all, 8 x 2, 4 x 4, 8 x 4, 4 x 8 and 6 x 5 are within 4% of each other; the ones taken are not the
// fastest for the weight gradients (gate/up 5.09 ms in 1 x all, 4.90 in 8 x 2; down 2.47 in 8 x 4, 2.38 in 4 x 4) and
// dgrad gate/up (3.67 in 8 x 2, 3.60 in 4 x 4).
template <int MODE>
void tile_cells(Params& p) {
  p.cm = 1;
  p.cn = 1 << 20;
  if (MODE == FWD1 || MODE == DGRAD2) { p.cm = 8; p.cn = 2; }
  if (MODE == WGRAD_DOWN) { p.cm = 8; p.cn = 4; }
}

template <int MODE>
int launch(const Params& p0, hipStream_t s) {
  Params p = p0;
  tile_cells<MODE>(p);
  const long long nt = (n_total<MODE>(p.d, p.f) + n_tile_width<MODE>() - 1) / n_tile_width<MODE>();
  long long upper;
  if (is_wgrad(MODE)) {
    upper = static_cast<long long>(p.E) * ((m_total<MODE>(p.d, p.f) + BM - 1) / BM) * (MODE == WGRAD_GU ? 2 : 1) * nt;
    MOE_REQUIRE(static_cast<long long>(p.P) * BM < 0x7fffffffLL, MOE_ERR_UNSUPPORTED, "padded token axis too long");
  } else {
    upper = (static_cast<long long>(p.n / BM) + p.E) * nt;
    MOE_REQUIRE(static_cast<long long>(k_one<MODE>(p.d, p.f)) * BM < 0x7fffffffLL, MOE_ERR_UNSUPPORTED, "rows too long");
  }
  MOE_REQUIRE(upper < (1LL << 31), MOE_ERR_UNSUPPORTED, "too many tiles");
  const unsigned g = static_cast<unsigned>(gemm_workgroups(upper));
  if constexpr (is_wgrad(MODE)) {
    grouped_gemm_fp8b_kernel<MODE, false><<<g, NTH, 0, s>>>(p);
  } else {
    if (k_one<MODE>(p.d, p.f) % BK != 0) grouped_gemm_fp8b_kernel<MODE, true><<<g, NTH, 0, s>>>(p);
    else grouped_gemm_fp8b_kernel<MODE, false><<<g, NTH, 0, s>>>(p);
  }
  return check_launch("grouped_gemm_fp8b");
}

// ------------------------------------------------------------------ few rows per expert
//
// What the forms for few rows write per lane: 4 consecutive columns of one row (`second`: FWD1's up
// accumulators, which with `v` make the activation).
template <int MODE>
__device__ __forceinline__ void store4(const Params& p, long long at, const f32x4& v, const f32x4& second) {
  typedef gep::u32x2 u32x2;
  if constexpr (MODE == FWD1) {
    if (p.o0 != nullptr) {
      *reinterpret_cast<u32x2*>(p.o0 + at) = gep::pack4(v);
      *reinterpret_cast<u32x2*>(p.o1 + at) = gep::pack4(second);
    }
    f32x4 av;
#pragma unroll
    for (int e = 0; e < 4; ++e) av[e] = v[e] * gep::sigmoid(v[e]) * second[e];
    *reinterpret_cast<u32x2*>(p.o2 + at) = gep::pack4(av);
  } else if constexpr (MODE == DGRAD1) {
    const u32x2 g2 = *reinterpret_cast<const u32x2*>(p.g + at), u2 = *reinterpret_cast<const u32x2*>(p.u + at);
    const float gv[4] = {bf16_lo(g2.x), bf16_hi(g2.x), bf16_lo(g2.y), bf16_hi(g2.y)};
    const float uv[4] = {bf16_lo(u2.x), bf16_hi(u2.x), bf16_lo(u2.y), bf16_hi(u2.y)};
    f32x4 dg, du;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float sg = gep::sigmoid(gv[e]);
      dg[e] = v[e] * uv[e] * sg * (1.0f + gv[e] * (1.0f - sg));
      du[e] = v[e] * gv[e] * sg;
    }
    *reinterpret_cast<u32x2*>(p.o0 + at) = gep::pack4(dg);
    *reinterpret_cast<u32x2*>(p.o1 + at) = gep::pack4(du);
  } else {
    *reinterpret_cast<u32x2*>(p.o0 + at) = gep::pack4(v);
  }
}

// The expert of row group mu (groups of R rows, an expert's last one partial; experts in order) and the
// group's place in it; false past the last group.  Lane l of round r holds expert 64 r + l; prefix sums by
// row shifts, as this stands between the launch and the first load of a weight.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
template <int R>
__device__ __forceinline__ bool find_group(const int32_t* __restrict__ offsets, int E, int mu, int& e, int& r0, int& r1) {
  const int lane = threadIdx.x & 63;
  int carry = 0;
  for (int base = 0; base < E; base += 64) {
    const int ex = min(base + lane, E - 1);
    const int lo = offsets[ex], hi = offsets[ex + 1];
    const int groups = base + lane < E ? (hi - lo + R - 1) / R : 0;
    int incl = groups;
    incl = dpp_add<0x111, 0xf>(incl);
    incl = dpp_add<0x112, 0xf>(incl);
    incl = dpp_add<0x114, 0xf>(incl);
    incl = dpp_add<0x118, 0xf>(incl);
    incl = dpp_add<0x142, 0xa>(incl);
    incl = dpp_add<0x143, 0xc>(incl);
    const int before = carry + incl - groups;
    const unsigned long long hit = __ballot(groups > 0 && before <= mu && mu < before + groups);
    if (hit) {
      const int src = __ffsll(static_cast<long long>(hit)) - 1;
      e = base + src;
      r0 = __builtin_amdgcn_readlane(lo, src) + (mu - __builtin_amdgcn_readlane(before, src)) * R;
      r1 = __builtin_amdgcn_readlane(hi, src);
      return true;
    }
    carry += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// A few rows per expert on average (single tokens, small decoding batches): a product reads every weight
// of the experts that have rows once and does next to nothing with it, so the kernel is a stream of weights.
// Each wave takes up to 16 rows of one expert and 32 weight rows: 32 output columns, or in FWD1 the gate
// and the up rows of 16.  It loads weight fragments straight into registers (no LDS: a weight is used by one
// wave only), D K steps ahead and together with the rows' codes and scales (loads return in order, so what
// is used together is loaded together).  The 4 waves of a workgroup split the contraction KS ways, summed in
// wave order through LDS, where the columns alone make too few waves.
// It has time to spare (4% of it), so its block sums are the exact ones, for the reason given at exact_rows.
constexpr int SKINNY_ROWS = 16;

struct SkinnyStep {
  i32x8 w[2];
  i32x8 x;
  float sx;
};

template <int MODE, int KS>
__device__ __forceinline__ void grouped_skinny(const Params& p) {
  constexpr int D = 3;                             // (4 take 146 registers instead of 120: 88 us for 64 tokens of 64 experts, 85 here)
  constexpr int WC = MODE == FWD1 ? 16 : 32;       // columns of a wave
  constexpr int CBW = 4 / KS;                      // column blocks per workgroup
  __shared__ float s_sum[4][8][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ks = wave % KS;
  const int N = n_total<MODE>(p.d, p.f), K = k_one<MODE>(p.d, p.f);
  const int KB = static_cast<int>(fp8b_blocks(K)), NB = static_cast<int>(fp8b_blocks(N));
  const int groups = (N / WC + CBW - 1) / CBW;
  const int mu = blockIdx.x / groups;
  const int cb = (blockIdx.x - mu * groups) * CBW + wave / KS;
  int e, r0, r1;
  if (!find_group<SKINNY_ROWS>(p.offsets, p.E, mu, e, r0, r1)) return;
  r1 = min(r1, p.n);                               // (as the other forms' descriptors: no row past the buffers)
  if (r0 >= r1) return;
  const int rows = min(SKINNY_ROWS, r1 - r0);
  const bool active = cb * WC < N;
  const int n0 = active ? cb * WC : 0;
  const int lr = lane & 15, lk = 16 * (lane >> 4);

  const long long woff = (static_cast<long long>(e) * N + n0 + lr) * K + lk;
  const uint8_t* const wp[2] = {p.b0 + woff, MODE == FWD1 ? p.b1 + woff : p.b0 + woff + 16LL * K};
  const int row = r0 + min(lr, rows - 1);          // lanes past the rows repeat the last one
  const uint8_t* const xp = p.a0 + static_cast<long long>(row) * K + lk;
  const float* const sp = p.a0s + row;
  auto load = [&](SkinnyStep& s, int kb) {
    const long long at = static_cast<long long>(kb) * BK;
    const bool tail = at + 64 >= K;                  // only the block's first half exists
    auto frag = [&](const uint8_t* q) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(q + at);
      i32x4 hi = {0, 0, 0, 0};
      if (!tail) hi = *reinterpret_cast<const i32x4*>(q + at + 64);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
#pragma unroll
    for (int w = 0; w < 2; ++w) s.w[w] = frag(wp[w]);
    s.x = frag(xp);
    s.sx = sp[static_cast<long long>(kb) * p.n];
  };
  f32x4 acc[2] = {};
  const long long sw_row = (static_cast<long long>(e) * NB + n0 / kFp8bBlock) * KB;
  if (active) {
    for (int base = 0; base < KB; base += 64) {      // lane l holds the weight scale of block base + l
      const int at = min(base + lane, KB - 1);
      const float ws0 = p.b0s[sw_row + at], ws1 = MODE == FWD1 ? p.b1s[sw_row + at] : ws0;
      const int end = min(KB, base + 64);
      SkinnyStep s[D];
      int kb = base + ks;
#pragma unroll
      for (int i = 0; i < D; ++i)
        if (kb + i * KS < end) load(s[i], kb + i * KS);
      while (kb < end) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
          if (kb < end) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const float sw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w ? ws1 : ws0), kb - base));
              const f32x4 t = exact_block(s[i].w[w], s[i].x);
              const float c = sw * s[i].sx;
#pragma unroll
              for (int q = 0; q < 4; ++q) acc[w][q] = fmaf(t[q], c, acc[w][q]);
            }
            if (kb + D * KS < end) load(s[i], kb + D * KS);
            kb += KS;
          }
        }
      }
    }
  }
  if constexpr (KS > 1) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int q = 0; q < 4; ++q) s_sum[wave][w * 4 + q][lane] = acc[w][q];
    __syncthreads();
    if (ks != 0) return;
#pragma unroll
    for (int o = 1; o < KS; ++o)
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[w][q] += s_sum[wave + o][w * 4 + q][lane];
  }
  if (!active || lr >= rows) return;
  const long long at = static_cast<long long>(r0 + lr) * N + n0 + 4 * (lane >> 4);
  store4<MODE>(p, at, acc[0], acc[1]);
  if constexpr (MODE != FWD1) store4<MODE>(p, at + 16, acc[1], acc[1]);
}

template <int MODE, int KS>
__global__ __launch_bounds__(256) void grouped_skinny_fp8b_kernel(Params p) {
  grouped_skinny<MODE, KS>(p);
}

template <int MODE>
int launch_skinny(const Params& p, hipStream_t s) {
  const int cols = n_total<MODE>(p.d, p.f) / (MODE == FWD1 ? 16 : 32);
  const long long units = p.n / SKINNY_ROWS + std::min(p.n, p.E);     // at least the row groups of all experts
  // as many ways to split the contraction as give every compute unit 8 waves, with 3 steps left for each
  const int kb = static_cast<int>(fp8b_blocks(k_one<MODE>(p.d, p.f)));
  int ks = 1;
  while (ks < 4 && units * cols * ks < 8LL * cu_count() && kb >= 6 * ks) ks *= 2;
  const long long blocks = units * ((cols + 4 / ks - 1) / (4 / ks));
  MOE_REQUIRE(blocks < (1LL << 31), MOE_ERR_UNSUPPORTED, "too many tiles");
  const unsigned g = static_cast<unsigned>(blocks);
  if (ks == 1) grouped_skinny_fp8b_kernel<MODE, 1><<<g, 256, 0, s>>>(p);
  else if (ks == 2) grouped_skinny_fp8b_kernel<MODE, 2><<<g, 256, 0, s>>>(p);
  else grouped_skinny_fp8b_kernel<MODE, 4><<<g, 256, 0, s>>>(p);
  return check_launch("grouped_gemm_fp8b (few rows)");
}

// The small tiles: 64 or 128 rows x 128 column rows (FWD1: the gate and the up rows of 64 columns), four
// waves, two LDS stages, one workgroup per tile, three (64 rows) or two (128) workgroups on a compute unit,
// so that each one's waits, prologue and epilogue are covered by the others' loads and products.  64-row
// tiles serve up to some 100 rows per expert, where the stream of weights sets the time but a weight meets
// enough rows that it should come through LDS once for all of them; 128-row tiles serve products whose
// 256-row tiles would be few, ragged, or short (few K steps for each epilogue, as the weight gradients of a
// few hundred tokens).  A wave has 64 rows x 32 columns, or 64 x 64.
constexpr int SM_BN = 128;
template <int BM>
struct Small {
  static constexpr int NF = BM / 32;                       // 16-column fragments of a wave
  static constexpr int A = BM * BK, B = SM_BN * BK;
  static constexpr int SA = A + B, SB = SA + BM * 4;       // the stage's scales, one float per row
  static constexpr int STAGE = SB + SM_BN * 4;
  static constexpr int PER_CU = BM == 64 ? 3 : 2;
};

template <int MODE, int BM, bool TAIL, bool EXACT>
__device__ __forceinline__ void grouped_small(const Params& p, uint8_t* lds) {
  constexpr bool WG = is_wgrad(MODE);
  using S = Small<BM>;
  constexpr int NF = S::NF;
  constexpr int TC = MODE == FWD1 ? SM_BN / 2 : SM_BN;     // output columns of a tile
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = BM == 128 ? wave >> 1 : 0, wn = BM == 128 ? wave & 1 : wave;
  const int N = n_total<MODE>(p.d, p.f), K = k_one<MODE>(p.d, p.f);
  const int nt = (N + TC - 1) / TC, kb_one = static_cast<int>(fp8b_blocks(K));
  // tiles dealt to the XCDs in contiguous runs, the row tiles of one column tile side by side
  MTiles mts{};
  int total, mtw = 0;
  if constexpr (WG) {
    mtw = (m_total<MODE>(p.d, p.f) + BM - 1) / BM * (MODE == WGRAD_GU ? 2 : 1);
    total = p.E * mtw * nt;
  } else {
    mts = gsched::mtile_scan<BM>(p.offsets, p.E);
    total = mts.total * nt;
  }
  // (round-robin for weight gradients of a hot expert, whose long tiles would otherwise share an XCD)
  const int per = (total + 7) >> 3;
  int lid = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (static_cast<int>(blockIdx.x >> 3) >= per) lid = total;
  if (WG && gsched::wgrad_skewed(p.offsets, p.E, p.n)) lid = blockIdx.x;
  if (lid >= total) return;
  Tile t{};
  int mi, ni, nk = kb_one * (MODE == DGRAD2 ? 2 : 1);
  if constexpr (WG) {
    const int Mtot = m_total<MODE>(p.d, p.f), mt = (Mtot + BM - 1) / BM;
    t.e = __builtin_amdgcn_readfirstlane(lid / (mtw * nt));
    gsched::cell_order(lid - t.e * mtw * nt, mtw, nt, 4, 4, mi, ni);
    t.half = __builtin_amdgcn_readfirstlane(mi >= mt ? 1 : 0);
    t.m0 = __builtin_amdgcn_readfirstlane((mi - t.half * mt) * BM);
    t.m_end = Mtot;
    token_range(p, t);
    nk = max(t.k_len, 0) / BK;
  } else {
    int e, first;
    gsched::mtile_find(mts, lid / nt, e, first);
    t.e = __builtin_amdgcn_readfirstlane(e);
    first = __builtin_amdgcn_readfirstlane(first);
    const int r0 = p.offsets[t.e], r1 = p.offsets[t.e + 1];
    gsched::cell_order(lid - first * nt, (r1 - r0 + BM - 1) / BM, nt, 1 << 20, 1, mi, ni);
    t.m0 = __builtin_amdgcn_readfirstlane(r0 + mi * BM);
    t.m_end = __builtin_amdgcn_readfirstlane(min(r1, p.n));
  }
  t.n0 = __builtin_amdgcn_readfirstlane(ni * TC);

  // DMA: each wave loads a quarter of both operands, 8 rows per instruction (FWD1: waves 0, 1 the gate's
  // rows, 2, 3 the up matrix's); the first BM / 64 waves the rows' scales, and of weight gradients waves
  // 2, 3 the columns'
  const int ld = WG ? p.P : K;
  const int wrow = MODE == FWD1 ? 32 * (wave & 1) : 32 * wave;
  const uint8_t *xb0, *xb1 = nullptr, *wb0, *wb1 = nullptr;
  const float *xs0, *xs1 = nullptr;
  long long xbytes, wbytes;
  int xrows, xpitch;
  if constexpr (WG) {
    const bool second = MODE == WGRAD_GU && t.half;
    xb0 = (second ? p.a1 : p.a0) + static_cast<long long>(t.m0) * p.P + t.k_begin;
    xbytes = static_cast<long long>(t.m_end - t.m0) * p.P - t.k_begin;
    wb0 = p.b0 + static_cast<long long>(t.n0) * p.P + t.k_begin;
    wbytes = static_cast<long long>(N - t.n0) * p.P - t.k_begin;
    xpitch = t.m_end;
    xrows = t.m_end - t.m0;
    xs0 = (second ? p.a1s : p.a0s) + static_cast<long long>(t.k_begin / BK) * t.m_end + t.m0;
  } else {
    const long long woff = (static_cast<long long>(t.e) * N + t.n0) * K;
    wb0 = (MODE == FWD1 && wave >= 2 ? p.b1 : p.b0) + woff;
    wb1 = p.b1 + woff;
    wbytes = static_cast<long long>(N - t.n0) * K;
    xrows = p.n - t.m0;
    xpitch = p.n;
    xb0 = p.a0 + static_cast<long long>(t.m0) * K;
    xb1 = p.a1 + static_cast<long long>(t.m0) * K;
    xbytes = static_cast<long long>(xrows) * K;
    xs0 = p.a0s + t.m0;
    xs1 = p.a1s + t.m0;
  }
  const int chunk = (lane & 7) ^ (lane >> 4);
  auto issue = [&](int k, int st) {
    const bool second = MODE == DGRAD2 && k >= kb_one;
    const int kb = second ? k - kb_one : k;
    const auto rw = gep::rsrc(second ? wb1 : wb0, wbytes);
    const auto rx = gep::rsrc(second ? xb1 : xb0, xbytes);
    uint8_t* const dst = lds + st * S::STAGE;
    const int left = K - kb * BK;
    auto load = [&](auto i, const __amdgpu_buffer_rsrc_t& r, int row, uint8_t* to) {
      const int c = (i & 1) ? chunk ^ 4 : chunk;
      int off = (row + 8 * i + (lane >> 3)) * ld + 16 * c;
      if (TAIL && 16 * c >= left) off = static_cast<int>(gep::OOB);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, off, kb * BK, 0, 0);
    };
    static_for<0, 4>([&](auto i) { load(i, rw, wrow, dst + S::A + (4 * wave + i) * 1024); });
    static_for<0, BM / 32>([&](auto i) { load(i, rx, BM / 4 * wave, dst + (BM / 32 * wave + i) * 1024); });
    if (wave < BM / 64) {
      const float* sc = (second ? xs1 : xs0) + static_cast<long long>(kb) * xpitch;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(gep::rsrc(sc, 4LL * xrows), (lds_void*)(dst + S::SA + 256 * wave), 4,
                                               4 * (64 * wave + lane), 0, 0, 0);
    }
    if (WG && wave >= 2) {
      const float* sc = p.b0s + static_cast<long long>(t.k_begin / BK + kb) * N + t.n0;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(gep::rsrc(sc, 4LL * (N - t.n0)), (lds_void*)(dst + S::SB + 256 * (wave - 2)),
                                               4, 4 * (64 * (wave - 2) + lane), 0, 0, 0);
    }
  };
  float w0 = 0.f, w1 = 0.f;                        // weight scales: lane l holds K block l's
  f32x4 acc[NF][4];
  const float start = start_value<MODE>(t);
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{start, start, start, start};
  if (nk > 0) issue(0, 0);
  const uint32_t base = lds_addr(lds);
  const uint32_t kc0 = kc_off(lane & 15, lane >> 4), kc1 = kc_off(lane & 15, 4 + (lane >> 4));
  const uint32_t a_off = 8192 * wm, b_off = S::A + (MODE == FWD1 ? 1024 : 2048) * NF * wn;
  const uint32_t sa_off = S::SA + 4 * (64 * wm + (lane & 15)), sb_off = S::SB + 4 * (16 * NF * wn + 4 * (lane >> 4));
  for (int k = 0; k < nk; ++k) {
    float ws0 = 1.f, ws1 = 1.f;
    if constexpr (!WG) {
      const bool second = MODE == DGRAD2 && k >= kb_one;
      const int kb = second ? k - kb_one : k;
      if ((kb & 63) == 0) {
        w0 = weight_scale<MODE>(p, t, t.n0, second ? 1 : 0, kb);
        if constexpr (MODE == FWD1) w1 = weight_scale<MODE>(p, t, t.n0, 1, kb);
      }
      ws0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w0), kb & 63));
      if constexpr (MODE == FWD1) ws1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w1), kb & 63));
    }
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    const uint32_t so = base + (k & 1) * S::STAGE;
    multiply_step<MODE, NF, 4, EXACT>(acc, so + a_off + kc0, so + a_off + kc1, so + b_off + kc0, so + b_off + kc1, so + sa_off,
                               so + sb_off, ws0, ws1, [&]() {
                                 if (k + 1 < nk) issue(k + 1, (k + 1) & 1);
                               });
  }
  const int row0 = t.m0 + 64 * wm;
  uint16_t* o0 = p.o0;
  long long out_rows = p.n;
  if constexpr (WG) {
    out_rows = t.m_end;
    o0 = (MODE == WGRAD_GU && t.half ? p.o1 : p.o0) + static_cast<long long>(t.e) * out_rows * N;
  }
  if constexpr (BM == 64) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = row0 + 16 * j + (lane & 15);
      if (r >= t.m_end) continue;
      const int col = t.n0 + (MODE == FWD1 ? 16 : 32) * wn + 4 * (lane >> 4);
      const long long at = static_cast<long long>(r) * N + col;
      if (col < N) store4<MODE>(p, at, acc[0][j], acc[1][j]);
      if (MODE != FWD1 && col + 16 < N) store4<MODE>(p, at + 16, acc[1][j], acc[1][j]);
    }
  } else {
    // staged through 4 KiB per wave of the stages, which every wave is done with
    using gep::u32x2;
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const uint32_t stg = base + 4096 * wave;
    const int rows_valid = t.m_end - row0;
    if constexpr (MODE == FWD1) {
      const int col0 = t.n0 + 32 * wn, cv = N - col0;
      auto store = [&](uint16_t* out, auto&& val) {
        u32x2 v[4][2];
        gep::sfor<0, 4>([&](auto j) { gep::sfor<0, 2>([&](auto i) { v[j][i] = val(i, j); }); });
        gep::stage_out_round<2, 4>(v, std::integral_constant<int, 0>{}, gep::out_rsrc(out, out_rows, N, row0, col0), rows_valid,
                                   cv, N, stg, lane);
      };
      if (p.o0 != nullptr) {
        store(p.o0, [&](auto i, auto j) { return gep::pack4(acc[i][j]); });
        store(p.o1, [&](auto i, auto j) { return gep::pack4(acc[i + 2][j]); });
      }
      store(p.o2, [&](auto i, auto j) {
        f32x4 av;
#pragma unroll
        for (int e = 0; e < 4; ++e) av[e] = acc[i][j][e] * gep::sigmoid(acc[i][j][e]) * acc[i + 2][j][e];
        return gep::pack4(av);
      });
    } else {
      const int col0 = t.n0 + 64 * wn, cv = N - col0;
      auto store = [&](auto q, uint16_t* out, const u32x2 (&v)[2][4]) {
        gep::stage_out_round<4, 2>(v, q, gep::out_rsrc(out, out_rows, N, row0, col0), rows_valid, cv, N, stg, lane);
      };
      if constexpr (MODE == DGRAD1) {
        // G and U straight into the product's layout (8 bytes of a row per lane), all rows' loads first
        gep::sfor<0, 2>([&](auto q) {
          u32x2 gm[2][4], um[2][4];
          const auto rg = gep::out_rsrc(p.g, p.n, N, row0, col0), ru = gep::out_rsrc(p.u, p.n, N, row0, col0);
          gep::sfor<0, 2>([&](auto jj) {
            gep::sfor<0, 4>([&](auto i) {
              const int rr = 16 * (2 * q + jj) + (lane & 15), cc = 16 * i + 4 * (lane >> 4);
              const int off = rr < rows_valid && cc < cv ? (rr * N + cc) * 2 : static_cast<int>(gep::OOB);
              gm[jj][i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rg, off, 0, 0));
              um[jj][i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(ru, off, 0, 0));
            });
          });
          gep::sfor<0, 2>([&](auto jj) {
            gep::sfor<0, 4>([&](auto i) {
              const u32x2 g2 = gm[jj][i], u2 = um[jj][i];
              const float gv[4] = {bf16_lo(g2.x), bf16_hi(g2.x), bf16_lo(g2.y), bf16_hi(g2.y)};
              const float uv[4] = {bf16_lo(u2.x), bf16_hi(u2.x), bf16_lo(u2.y), bf16_hi(u2.y)};
              f32x4 dg, du;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float da = acc[i][2 * q + jj][e], sg = gep::sigmoid(gv[e]);
                dg[e] = da * uv[e] * sg * (1.0f + gv[e] * (1.0f - sg));
                du[e] = da * gv[e] * sg;
              }
              gm[jj][i] = gep::pack4(dg);
              um[jj][i] = gep::pack4(du);
            });
          });
          store(q, p.o0, gm);
          store(q, p.o1, um);
        });
      } else {
        gep::sfor<0, 2>([&](auto q) {
          u32x2 v[2][4];
          gep::sfor<0, 2>([&](auto jj) { gep::sfor<0, 4>([&](auto i) { v[jj][i] = gep::pack4(acc[i][2 * q + jj]); }); });
          store(q, o0, v);
        });
      }
    }
  }
}

template <int MODE, int BM, bool TAIL, bool EXACT>
__global__ __launch_bounds__(256, Small<BM>::PER_CU) void grouped_small_fp8b_kernel(Params p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * Small<BM>::STAGE];
  grouped_small<MODE, BM, TAIL, EXACT>(p, lds);
}

template <int MODE, int BM, bool EXACT = false>
int launch_small(const Params& p, hipStream_t s) {
  const int K = k_one<MODE>(p.d, p.f), tc = MODE == FWD1 ? SM_BN / 2 : SM_BN;
  const long long nt = (n_total<MODE>(p.d, p.f) + tc - 1) / tc;
  const long long blocks =
      is_wgrad(MODE) ? static_cast<long long>(p.E) * ((m_total<MODE>(p.d, p.f) + BM - 1) / BM) * (MODE == WGRAD_GU ? 2 : 1) * nt
                     : (static_cast<long long>(p.n / BM) + std::min(p.n, p.E)) * nt;
  MOE_REQUIRE(blocks < (1LL << 31) - 8, MOE_ERR_UNSUPPORTED, "too many tiles");
  MOE_REQUIRE((is_wgrad(MODE) ? static_cast<long long>(p.P) : K) * SM_BN < 0x7fffffffLL, MOE_ERR_UNSUPPORTED, "rows too long");
  const unsigned g = static_cast<unsigned>((blocks + 7) / 8 * 8);
  if (!is_wgrad(MODE) && K % BK != 0) grouped_small_fp8b_kernel<MODE, BM, !is_wgrad(MODE), EXACT><<<g, 256, 0, s>>>(p);
  else grouped_small_fp8b_kernel<MODE, BM, false, EXACT><<<g, 256, 0, s>>>(p);
  return check_launch("grouped_gemm_fp8b (small tiles)");
}

// Which form runs a product, from host-visible sizes (the row counts stay on the device).
//   few rows:  forward products of at most 6 rows per expert on average.  Measured (gate/up + down with their
//              quantisers and combine, weights not in the last-level cache, us; 64-row tiles in brackets): 64
//              experts, d 2048, f 1024, 4 rows each 85 [101]; one token of 8 experts, d 4096, f 768 38 [56]; the
//              first with 16 rows each, products alone, weights cached: 47 + 27 [34 + 26].
//   else the tiling with the lowest estimate: rounds of tiles over the compute units, each KB = K / 128 steps
//   and an epilogue.  Bigger tiles move fewer bytes per product and cost less per output; smaller ones leave
//   less of the last round empty.  A tile of K blocks takes, in us: 256 rows 1.5 K + 6.5 (23 with the SwiGLU
//   backward's epilogue, 1.75 K + 6 for weight gradients), 128 rows 0.64 K + 3 (7.6; 0.72 K + 2.6), 64 rows
//   0.4 K + 2 (4); a unit's share of the tiles counts as whole rounds, and half a round more than the share
//   for the persistent 256-row kernel, whose units drift apart.  Fitted to 1 to 128 experts, d and f 512 to
//   7168, 64 to 8192 rows per expert, where the choice costs 1% over the best form on average, 20% at worst.
//   Both sides of it (gate/up + down, us, 64- / 128- / 256-row tiles): 64 experts, d 2048, f 1024, 128 rows
//   each 101 + 47 / 109 + 55 / 86 + 44, 1024 rows 531 + 314 / 438 + 253 / 348 + 191; 16 experts, d 2112, f 1344,
//   64 rows 31 + 15 / 27 + 18 / 37 + 24, 250 rows 52 + 30 / 48 + 29 / 41 + 26; one expert, d = f = 4096, 1024
//   rows 60 + 30 / 43 + 30 / 59 + 50, 4096 rows 203 + 97 / 160 + 79 / 122 + 61; weight gradients of 16 experts,
//   d 2112, f 1344, 64 rows 128-row tiles 28 + 52, 256-row 27 + 41.
// MOE_FP8B_FORM = few, mid, half or big sets the form (tests run every form on the same cases; a product without it
// takes the next).  It chooses a kernel, not a precision: see exact_rows for the one exception.
enum Form { FEW, MID, HALF, BIG, NONE, UNKNOWN };
Form forced_form() {
  const char* env = getenv("MOE_FP8B_FORM");
  if (env == nullptr || env[0] == '\0') return NONE;
  return !strcmp(env, "few") ? FEW : !strcmp(env, "mid") ? MID : !strcmp(env, "half") ? HALF : !strcmp(env, "big") ? BIG : UNKNOWN;
}
template <int MODE>
Form choose_form(const Params& p, Form forced) {
  constexpr bool WG = is_wgrad(MODE), FORWARD = MODE == FWD1 || MODE == FWD2;
  if (forced != NONE) {
    if (forced == FEW && !FORWARD) forced = MID;
    return forced == MID && WG ? HALF : forced;
  }
  if (FORWARD && p.n <= 6LL * p.E) return FEW;
  const double busy = std::min(p.n, p.E), mean = p.n / busy;
  const double kb = WG ? std::ceil(mean / BK) : static_cast<double>(fp8b_blocks(k_one<MODE>(p.d, p.f))) * (MODE == DGRAD2 ? 2 : 1);
  const int N = n_total<MODE>(p.d, p.f), cus = cu_count();
  auto tiles = [&](int bm, int cols) {           // per unit
    double mt;
    if (WG) mt = busy * ((m_total<MODE>(p.d, p.f) + bm - 1) / bm) * (MODE == WGRAD_GU ? 2 : 1);
    else if (p.E == 1) mt = (p.n + bm - 1) / bm;
    else mt = mean <= 0.84 * bm ? busy : static_cast<double>(p.n) / bm + 0.5 * busy;   // a last tile half full
    return mt * ((N + cols - 1) / cols) / cus;
  };
  const int cols = MODE == FWD1 ? SM_BN / 2 : SM_BN;
  const double tb = tiles(BM, n_tile_width<MODE>());
  const double big = (tb <= 1.0 ? 1.0 : tb + 0.5) * (WG ? 1.75 * kb + 6.0 : 1.5 * kb + (MODE == DGRAD1 ? 23.0 : 6.5));
  // (the 256-row kernel's 32-bit offsets span 256 rows of codes, the others' 128)
  const bool fits = (WG ? static_cast<long long>(p.P) : k_one<MODE>(p.d, p.f)) * BM < 0x7fffffffLL;
  const double half = std::ceil(tiles(128, cols)) * (WG ? 0.72 * kb + 2.6 : 0.64 * kb + (MODE == DGRAD1 ? 7.6 : 3.0)) - 1.5;
  if (WG) return half < big || !fits ? HALF : BIG;
  const double mid = std::ceil(tiles(64, cols)) * (0.4 * kb + (MODE == DGRAD1 ? 4.0 : 2.0)) + 2.5;
  return mid < half && (mid < big || !fits) ? MID : half < big || !fits ? HALF : BIG;
}

// A, dG and dU are quantised again by whoever uses them.  Where one is rounded to bf16 the other way at the
// largest value of a block, the block's scale moves by 2^-8 and some 5% of its codes by a step, 2% of its sum; the
// fp8 matrix core's cut does that to one block in 200.  Among many blocks it takes y from 0.17% (its own rounding)
// to 0.21% off, but one such block in 32 to 0.4%.  So a product of fewer than 2048 blocks has exact block sums:
// above, twice the expected number of moved blocks still leaves y within one and a half times its rounding.
// They cost (gate/up, us, 64-row tiles of the two kinds and the kernel of few rows): 16 experts, d 2112, f 1344, 16
// rows each 17 / 28 / 18; one expert, d = f = 4096, 16 rows 18 / 29 / 13, 64 rows 19 / 31 / 26; 8 experts, d 7168,
// f 2048, 16 rows 41 / 57 / 41, 30 rows 41 / 58 / 79.
// (128- and 256-row tiles have no exact form: where one of them is set by hand, its sums are the fp8 core's.)
template <int MODE>
bool exact_rows(const Params& p, Form forced) {
  return (MODE == FWD1 || MODE == DGRAD1) && p.n * static_cast<long long>(fp8b_blocks(p.f)) < 2048 && forced != HALF &&
         forced != BIG;
}

template <int MODE>
int launch_rows(const Params& p, hipStream_t s) {
  const Form forced = forced_form();
  MOE_REQUIRE(forced != UNKNOWN, MOE_ERR_INVALID_ARG, "MOE_FP8B_FORM must be few, mid, half or big");
  const Form form = choose_form<MODE>(p, forced);
  if constexpr (MODE == FWD1 || MODE == FWD2) {
    if (form == FEW) return launch_skinny<MODE>(p, s);
  }
  if constexpr (MODE == FWD1 || MODE == DGRAD1) {
    if (exact_rows<MODE>(p, forced)) {
      if constexpr (MODE == FWD1)
        if (forced == NONE && p.n <= 16LL * p.E) return launch_skinny<MODE>(p, s);
      return launch_small<MODE, 64, true>(p, s);
    }
  }
  if (form == HALF) return launch_small<MODE, 128>(p, s);
  if constexpr (!is_wgrad(MODE)) {
    if (form == MID) return launch_small<MODE, 64>(p, s);
  }
  return launch<MODE>(p, s);
}

int check_gemm(int E, int n, int d, int f, const int32_t* offsets) {
  MOE_REQUIRE(E >= 1 && E <= 256, MOE_ERR_UNSUPPORTED, "E must be in [1, 256] (got %d)", E);
  MOE_REQUIRE(n >= 1, MOE_ERR_UNSUPPORTED, "n must be >= 1 (got %d)", n);
  MOE_REQUIRE(d >= 64 && d % 64 == 0 && f >= 64 && f % 64 == 0, MOE_ERR_UNSUPPORTED,
              "d and f must be positive multiples of 64 (got %d, %d)", d, f);
  MOE_CHECK_PTR(offsets);
  return MOE_OK;
}

}  // namespace g8b
}  // namespace moe

using namespace moe;

#define FP8B_OPERAND(p) \
  do { MOE_CHECK_PTR(p); MOE_CHECK_ALIGN(p); } while (0)

extern "C" int moe_grouped_gemm_gate_up_fp8b(int E, int n, int d, int f, const int32_t* offsets, const uint8_t* xq,
                                             const float* xs, const uint8_t* w_gate, const float* w_gate_s,
                                             const uint8_t* w_up, const float* w_up_s, uint16_t* g, uint16_t* u,
                                             uint16_t* a, void* stream) {
  if (int st = g8b::check_gemm(E, n, d, f, offsets)) return st;
  FP8B_OPERAND(xq); FP8B_OPERAND(xs); FP8B_OPERAND(w_gate); FP8B_OPERAND(w_gate_s);
  FP8B_OPERAND(w_up); FP8B_OPERAND(w_up_s); FP8B_OPERAND(a);
  MOE_REQUIRE((g == nullptr) == (u == nullptr), MOE_ERR_INVALID_ARG, "g and u come together");
  if (g) { MOE_CHECK_ALIGN(g); MOE_CHECK_ALIGN(u); }
  g8b::Params p{};
  p.offsets = offsets; p.E = E; p.n = n; p.d = d; p.f = f;
  p.a0 = xq; p.a0s = xs; p.b0 = w_gate; p.b0s = w_gate_s; p.b1 = w_up; p.b1s = w_up_s;
  p.o0 = g; p.o1 = u; p.o2 = a;
  return g8b::launch_rows<g8b::FWD1>(p, as_stream(stream));
}

extern "C" int moe_grouped_gemm_down_fp8b(int E, int n, int d, int f, const int32_t* offsets, const uint8_t* aq,
                                          const float* as, const uint8_t* w_down, const float* w_down_s, uint16_t* yexp,
                                          void* stream) {
  if (int st = g8b::check_gemm(E, n, d, f, offsets)) return st;
  FP8B_OPERAND(aq); FP8B_OPERAND(as); FP8B_OPERAND(w_down); FP8B_OPERAND(w_down_s); FP8B_OPERAND(yexp);
  g8b::Params p{};
  p.offsets = offsets; p.E = E; p.n = n; p.d = d; p.f = f;
  p.a0 = aq; p.a0s = as; p.b0 = w_down; p.b0s = w_down_s; p.o0 = yexp;
  return g8b::launch_rows<g8b::FWD2>(p, as_stream(stream));
}

extern "C" int moe_grouped_gemm_dgrad_down_fp8b(int E, int n, int d, int f, const int32_t* offsets, const uint8_t* dyq,
                                                const float* dys, const uint8_t* w_down_t, const float* w_down_t_s,
                                                const uint16_t* g, const uint16_t* u, uint16_t* dg, uint16_t* du,
                                                void* stream) {
  if (int st = g8b::check_gemm(E, n, d, f, offsets)) return st;
  FP8B_OPERAND(dyq); FP8B_OPERAND(dys); FP8B_OPERAND(w_down_t); FP8B_OPERAND(w_down_t_s);
  FP8B_OPERAND(g); FP8B_OPERAND(u); FP8B_OPERAND(dg); FP8B_OPERAND(du);
  g8b::Params p{};
  p.offsets = offsets; p.E = E; p.n = n; p.d = d; p.f = f;
  p.a0 = dyq; p.a0s = dys; p.b0 = w_down_t; p.b0s = w_down_t_s; p.g = g; p.u = u; p.o0 = dg; p.o1 = du;
  return g8b::launch_rows<g8b::DGRAD1>(p, as_stream(stream));
}

extern "C" int moe_grouped_gemm_dgrad_gate_up_fp8b(int E, int n, int d, int f, const int32_t* offsets,
                                                   const uint8_t* dgq, const float* dgs, const uint8_t* duq,
                                                   const float* dus, const uint8_t* w_gate_t, const float* w_gate_t_s,
                                                   const uint8_t* w_up_t, const float* w_up_t_s, uint16_t* dxp,
                                                   void* stream) {
  if (int st = g8b::check_gemm(E, n, d, f, offsets)) return st;
  FP8B_OPERAND(dgq); FP8B_OPERAND(dgs); FP8B_OPERAND(duq); FP8B_OPERAND(dus);
  FP8B_OPERAND(w_gate_t); FP8B_OPERAND(w_gate_t_s); FP8B_OPERAND(w_up_t); FP8B_OPERAND(w_up_t_s); FP8B_OPERAND(dxp);
  g8b::Params p{};
  p.offsets = offsets; p.E = E; p.n = n; p.d = d; p.f = f;
  p.a0 = dgq; p.a0s = dgs; p.a1 = duq; p.a1s = dus;
  p.b0 = w_gate_t; p.b0s = w_gate_t_s; p.b1 = w_up_t; p.b1s = w_up_t_s; p.o0 = dxp;
  return g8b::launch_rows<g8b::DGRAD2>(p, as_stream(stream));
}

extern "C" int moe_grouped_gemm_wgrad_down_fp8b(int E, int n, int d, int f, const int32_t* offsets,
                                                const int32_t* offsets_pad, const uint8_t* dyT, const float* dyTs,
                                                const uint8_t* aT, const float* aTs, uint16_t* dw_down, void* stream) {
  if (int st = g8b::check_gemm(E, n, d, f, offsets)) return st;
  MOE_CHECK_PTR(offsets_pad);
  FP8B_OPERAND(dyT); FP8B_OPERAND(dyTs); FP8B_OPERAND(aT); FP8B_OPERAND(aTs); FP8B_OPERAND(dw_down);
  g8b::Params p{};
  p.offsets = offsets; p.offsets_pad = offsets_pad; p.E = E; p.n = n; p.d = d; p.f = f;
  p.P = moe_mx_pad_cap(n, E);
  MOE_REQUIRE(p.P > 0, MOE_ERR_UNSUPPORTED, "padded token axis too long");
  p.a0 = dyT; p.a0s = dyTs; p.b0 = aT; p.b0s = aTs; p.o0 = dw_down;
  return g8b::launch_rows<g8b::WGRAD_DOWN>(p, as_stream(stream));
}

extern "C" int moe_grouped_gemm_wgrad_gate_up_fp8b(int E, int n, int d, int f, const int32_t* offsets,
                                                   const int32_t* offsets_pad, const uint8_t* dgT, const float* dgTs,
                                                   const uint8_t* duT, const float* duTs, const uint8_t* xT,
                                                   const float* xTs, uint16_t* dw_gate, uint16_t* dw_up, void* stream) {
  if (int st = g8b::check_gemm(E, n, d, f, offsets)) return st;
  MOE_CHECK_PTR(offsets_pad);
  FP8B_OPERAND(dgT); FP8B_OPERAND(dgTs); FP8B_OPERAND(duT); FP8B_OPERAND(duTs); FP8B_OPERAND(xT); FP8B_OPERAND(xTs);
  FP8B_OPERAND(dw_gate); FP8B_OPERAND(dw_up);
  g8b::Params p{};
  p.offsets = offsets; p.offsets_pad = offsets_pad; p.E = E; p.n = n; p.d = d; p.f = f;
  p.P = moe_mx_pad_cap(n, E);
  MOE_REQUIRE(p.P > 0, MOE_ERR_UNSUPPORTED, "padded token axis too long");
  p.a0 = dgT; p.a0s = dgTs; p.a1 = duT; p.a1s = duTs; p.b0 = xT; p.b0s = xTs; p.o0 = dw_gate; p.o1 = dw_up;
  return g8b::launch_rows<g8b::WGRAD_GU>(p, as_stream(stream));
}
