// Quantisation of bf16 tensors to E4M3 codes with one fp32 scale per block of 128 (fp8b_common.h has
// the arithmetic), in the layouts the block-scaled grouped GEMMs read:
//   rows      blocks of 128 along the row, optionally on the way into the expert buffers (each token's
//             row to its k destinations); codes [n, C], scales [ceil(C/128), n]
//   grouped   blocks of 128 tokens of one expert, codes transposed [C, P] with every expert's tokens
//             starting at a multiple of 128 (the weight-gradient operands), scales [P/128, C];
//             together with the row layout from one read
//   weights   blocks of 128 x 128 of each matrix, codes as they lie and transposed, one set of scales
//             [E, ceil(R/128), ceil(C/128)] and its transpose
// Scales are block-major, so one K step of a product reads the scales of its 256 rows as one run.
// All are HBM-bound: 2 bytes read, 1 + 4/128 bytes written per element and layout.  Measured: rows of 8192 tokens
// of 2048 to 4 destinations 20 us (5.1 TB/s of its bytes); rows and tokens of 16384 x 4 of 1536 78 us; weights of 64
// matrices of 2048 x 7168 727 us (5.2 TB/s).
#include <type_traits>

#include "fp8b_common.h"

namespace moe {
namespace {

constexpr int kRowThreads = 256;

// ---- rows: 16 lanes per block, 8 elements (16 bytes read, 8 codes written) per lane.  Item: chunk c of
// row t, chunks padded to whole blocks per row so that a block's 16 lanes are one row's.
template <bool PERMUTE>
__global__ __launch_bounds__(kRowThreads) void fp8b_rows_kernel(const uint16_t* __restrict__ x,
                                                                const int32_t* __restrict__ dest, long long rows,
                                                                int C, int k, long long n, uint8_t* __restrict__ q,
                                                                float* __restrict__ s) {
  const int per_row = static_cast<int>(fp8b_blocks(C)) * 16;
  const long long item = static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x;
  const long long t = item / per_row;
  const int c = static_cast<int>(item - t * per_row);
  const bool live = t < rows && 8 * c < C;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (live) v = *reinterpret_cast<const uint4*>(x + t * C + 8 * c);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint32_t amax = max16(fp8b_amax8(w));
  if (!live) return;
  const Fp8bScale f = fp8b_scale(amax);
  const uint2 o = fp8b_encode8(w, f.inv);
  const int copies = PERMUTE ? k : 1;
  for (int j = 0; j < copies; ++j) {
    const long long r = PERMUTE ? dest[t * k + j] : t;
    if (PERMUTE && static_cast<unsigned long long>(r) >= static_cast<unsigned long long>(n)) continue;   // no row of the buffers
    *reinterpret_cast<uint2*>(q + r * C + 8 * c) = o;
    if ((c & 15) == 0) s[(c >> 4) * n + r] = f.scale;
  }
}

// ---- the tile forms: 128 positions x 128 columns per step of a 256-thread workgroup.  Thread t holds
// rows 8 (t / 16) .. + 7 of columns 8 (t % 16) .. + 7, so a row block is 16 adjacent lanes and a column
// block is 16 threads' 8 rows; transposed codes go through LDS into 128-byte runs.
constexpr int kTile = 128;
constexpr int kTileThreads = 256;

// 8 bytes (8 positions, chunk pg) of transposed column c: chunks XORed by the column's group of 8,
// so the 16 lanes that write one chunk of 16 column groups hit different banks.
__device__ __forceinline__ int tcode_off(int c, int pg) { return c * kTile + ((pg ^ ((c >> 3) & 15)) << 3); }

// Writes the staged transposed codes: column c's 128 positions to qT[(c0 + c) * pitch + p0 ..], for the
// columns below `cols` and the positions below `len` (both counted from the tile's corner; len a
// multiple of 64).
__device__ __forceinline__ void store_transposed(const uint8_t* s_t, uint8_t* __restrict__ qT, long long pitch, int cols,
                                                 int len) {
#pragma unroll
  for (int i = 0; i < kTile * kTile / 16 / kTileThreads; ++i) {
    const int item = threadIdx.x + kTileThreads * i;
    const int c = item >> 3, m = item & 7;       // 16 bytes: positions 16 m .. + 15
    if (c < cols && 16 * m < len) {
      const uint2 a = *reinterpret_cast<const uint2*>(s_t + tcode_off(c, 2 * m));
      const uint2 b = *reinterpret_cast<const uint2*>(s_t + tcode_off(c, 2 * m + 1));
      *reinterpret_cast<uint4*>(qT + c * pitch + 16 * m) = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
}

// Transposes 8 x 8 codes in registers (row i: 8 columns' codes) and stages them as 8 column chunks: four
// 4 x 4 byte blocks, eight byte permutes each.
__device__ __forceinline__ void stage_transposed(const uint2 (&o)[8], uint8_t* s_t, int cg, int pg) {
  uint32_t t[8][2];                                // [column][half of its 8 positions]
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t r0 = c ? o[4 * h].y : o[4 * h].x, r1 = c ? o[4 * h + 1].y : o[4 * h + 1].x;
      const uint32_t r2 = c ? o[4 * h + 2].y : o[4 * h + 2].x, r3 = c ? o[4 * h + 3].y : o[4 * h + 3].x;
      // bytes 0-3 of a permute's selector address its second operand, 4-7 its first
      const uint32_t a = __builtin_amdgcn_perm(r1, r0, 0x05010400u), b = __builtin_amdgcn_perm(r1, r0, 0x07030602u);
      const uint32_t d = __builtin_amdgcn_perm(r3, r2, 0x05010400u), e = __builtin_amdgcn_perm(r3, r2, 0x07030602u);
      t[4 * c + 0][h] = __builtin_amdgcn_perm(d, a, 0x05040100u);
      t[4 * c + 1][h] = __builtin_amdgcn_perm(d, a, 0x07060302u);
      t[4 * c + 2][h] = __builtin_amdgcn_perm(e, b, 0x05040100u);
      t[4 * c + 3][h] = __builtin_amdgcn_perm(e, b, 0x07060302u);
    }
#pragma unroll
  for (int j = 0; j < 8; ++j) *reinterpret_cast<uint2*>(s_t + tcode_off(8 * cg + j, pg)) = make_uint2(t[j][0], t[j][1]);
}

// Work item of block `id` when XCD x (block ids = x mod 8, each XCD with its own L2) takes a contiguous run
// of the items, so that neighbours of a band share an L2.
__device__ __forceinline__ long long run_item(long long id, long long total) {
  const long long per = total >> 3, extra = total & 7;
  const long long x = id & 7;
  return x * per + (x < extra ? x : extra) + (id >> 3);
}

// Grouped rows: padded position p of expert e holds grouped row r = offsets[e] + p - offsets_pad[e] while
// that is below offsets[e + 1]; its data is in[row_token ? row_token[r] : r], times row_gate[r] rounded
// to bf16 where given.  ROWS: also the real rows' row layout, q [n][C] and s [ceil(C/128)][n].  Offsets that are not
// whole blocks of the axis (of another pad than 128) would leave rows out: they make every scale NaN instead.
// A division per block: lane i of a row's 16 makes the factors of the thread group's row i, and one thread
// those of each column.  One tile per workgroup: walking four or eight along the band, as the MX quantisers
// do, measured level in time (81-88 us for 65536 rows of 1536, k = 4) and took 50 registers more.  Bound by
// its traffic: 38 us of reads (each token's row once per copy) and 21 us for each of the two outputs.
template <bool ROWS, bool GATE>
__global__ __launch_bounds__(kTileThreads, 6) void fp8b_grouped_kernel(
    const uint16_t* __restrict__ in, const int32_t* __restrict__ row_token, const float* __restrict__ row_gate,
    const int32_t* __restrict__ offsets, const int32_t* __restrict__ offsets_pad, int E, int C, long long n, long long P,
    uint8_t* __restrict__ q, float* __restrict__ s, uint8_t* __restrict__ qT, float* __restrict__ sT, int ctiles) {
  __shared__ __attribute__((aligned(16))) uint8_t s_t[kTile * kTile];
  __shared__ __attribute__((aligned(16))) uint32_t s_amax[kTileThreads / 64][kTile / 2];
  __shared__ __attribute__((aligned(16))) float s_inv[kTile];
  const int tid = threadIdx.x, cg = tid & 15, pg = tid >> 4;
  const long long item = run_item(blockIdx.x, gridDim.x);
  const long long p0 = item / ctiles * kTile;
  const int ct = static_cast<int>(item % ctiles), c0 = ct * kTile;
  // the band's expert: the last one that starts at or before it (every wave counts for itself: one round
  // of loads, where a search would wait for each of eight)
  int before = 0;
  const int end = offsets_pad[E];
  bool odd = end < 0 || end > P || (end & (kTile - 1)) != 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 64 * i + (tid & 63);
    const int start = e < E ? offsets_pad[e] : end;
    before += __popcll(__ballot(e < E && start <= p0));
    odd |= (start & (kTile - 1)) != 0 || start < 0 || start > end || (e == 0 && start != 0);
  }
  if (__ballot(odd) != 0ull) {                             // (the same in every workgroup)
    const float nan = __builtin_nanf("");
    if (tid < kTile) {
      if (ROWS && p0 + tid < n) s[ct * n + p0 + tid] = nan;
      if (c0 + tid < C) sT[(p0 / kTile) * C + c0 + tid] = nan;
    }
    return;
  }
  const int e = max(before - 1, 0);
  const int first = offsets[e];
  // the thread's eight positions: consecutive rows row0 .. of that expert, as far as it has them
  const int row0 = static_cast<int>(first + (p0 - offsets_pad[e]) + 8 * pg);
  const int rows = p0 < end ? min(max(static_cast<int>(min(static_cast<long long>(offsets[e + 1]), n)) - row0, 0), 8) : 0;
  const unsigned live = (1u << rows) - 1u;
  int src[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) src[i] = i < rows ? (row_token != nullptr ? row_token[row0 + i] : row0 + i) : -1;
  float gate[8];
  if constexpr (GATE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) gate[i] = (live >> i & 1u) ? row_gate[row0 + i] : 1.f;
  }
  const int col = c0 + 8 * cg;
  const bool in_cols = col < C;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if (src[i] >= 0 && in_cols) v[i] = *reinterpret_cast<const uint4*>(in + static_cast<long long>(src[i]) * C + col);
  }
  uint32_t cmax[4] = {0, 0, 0, 0};
  uint32_t my_amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (GATE) {
      uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int h = 0; h < 4; ++h) w[h] = pack_bf16x2(gate[i] * bf16_lo(w[h]), gate[i] * bf16_hi(w[h]));
      v[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    const uint32_t m[4] = {abs_pair(v[i].x), abs_pair(v[i].y), abs_pair(v[i].z), abs_pair(v[i].w)};
#pragma unroll
    for (int h = 0; h < 4; ++h) cmax[h] = max_pair(cmax[h], m[h]);
    if constexpr (ROWS) {
      const uint32_t rmax = max16(max_of_pair(max_pair(max_pair(m[0], m[1]), max_pair(m[2], m[3]))));
      my_amax = (cg & 7) == i ? rmax : my_amax;
    }
  }
  if constexpr (ROWS) {
    const Fp8bScale f = fp8b_scale(my_amax);
    if (cg < 8 && (live >> cg & 1u)) s[ct * n + row0 + cg] = f.scale;
    uint8_t* const qrow = q + static_cast<long long>(row0) * C + col;
    auto put = [&](auto i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      const uint2 o = fp8b_encode8(w, row_lane<i>(f.inv));
      if ((live >> i & 1u) && in_cols) *reinterpret_cast<uint2*>(qrow + static_cast<long long>(i) * C) = o;
      __builtin_amdgcn_sched_barrier(0);   // one row's codes at a time: all eight at once took 70 more registers
    };
    put(std::integral_constant<int, 0>{}); put(std::integral_constant<int, 1>{});
    put(std::integral_constant<int, 2>{}); put(std::integral_constant<int, 3>{});
    put(std::integral_constant<int, 4>{}); put(std::integral_constant<int, 5>{});
    put(std::integral_constant<int, 6>{}); put(std::integral_constant<int, 7>{});
  }
  // column maxima: over the wave's four position groups, then over the four waves
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    cmax[h] = max_pair(cmax[h], static_cast<uint32_t>(__shfl_xor(static_cast<int>(cmax[h]), 16, 64)));
    cmax[h] = max_pair(cmax[h], static_cast<uint32_t>(__shfl_xor(static_cast<int>(cmax[h]), 32, 64)));
  }
  if ((tid & 63) < 16) *reinterpret_cast<uint4*>(&s_amax[tid >> 6][4 * cg]) = make_uint4(cmax[0], cmax[1], cmax[2], cmax[3]);
  __syncthreads();
  if (tid < kTile) {
    const uint32_t m = max_pair(max_pair(s_amax[0][tid >> 1], s_amax[1][tid >> 1]),
                                max_pair(s_amax[2][tid >> 1], s_amax[3][tid >> 1]));
    const Fp8bScale f = fp8b_scale((tid & 1) ? m >> 16 : m & 0xffffu);
    s_inv[tid] = f.inv;
    if (c0 + tid < C) sT[(p0 / kTile) * C + c0 + tid] = f.scale;
  }
  __syncthreads();
  const float4 ia = *reinterpret_cast<const float4*>(&s_inv[8 * cg]), ib = *reinterpret_cast<const float4*>(&s_inv[8 * cg + 4]);
  uint2 o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i] = make_uint2(fp8b_encode4(bf16_lo(v[i].x) * ia.x, bf16_hi(v[i].x) * ia.y, bf16_lo(v[i].y) * ia.z,
                                   bf16_hi(v[i].y) * ia.w),
                      fp8b_encode4(bf16_lo(v[i].z) * ib.x, bf16_hi(v[i].z) * ib.y, bf16_lo(v[i].w) * ib.z,
                                   bf16_hi(v[i].w) * ib.w));
  stage_transposed(o, s_t, cg, pg);
  __syncthreads();
  store_transposed(s_t, qT + c0 * P + p0, P, C - c0, kTile);
}

// Weights [E][R][C]: one workgroup per 128 x 128 block.
__global__ __launch_bounds__(kTileThreads) void fp8b_weights_kernel(const uint16_t* __restrict__ w, int R, int C,
                                                                    int rblocks, int cblocks, uint8_t* __restrict__ q,
                                                                    float* __restrict__ s, uint8_t* __restrict__ qT,
                                                                    float* __restrict__ sT) {
  __shared__ __attribute__((aligned(16))) uint8_t s_t[kTile * kTile];
  __shared__ uint32_t s_amax[kTileThreads / 64];
  const int tid = threadIdx.x, cg = tid & 15, pg = tid >> 4;
  const long long item = blockIdx.x;
  const int cb = static_cast<int>(item % cblocks);
  const long long rest = item / cblocks;
  const int rb = static_cast<int>(rest % rblocks);
  const long long e = rest / rblocks;
  const long long plane = e * R * C;
  const int r0 = rb * kTile, c0 = cb * kTile, col = c0 + 8 * cg;
  uint4 v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 8 * pg + i;
    v[i] = make_uint4(0, 0, 0, 0);
    if (r < R && col < C) v[i] = *reinterpret_cast<const uint4*>(w + plane + static_cast<long long>(r) * C + col);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    m = max(m, fp8b_amax8(x));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, 64)));
  if ((tid & 63) == 0) s_amax[tid >> 6] = m;
  __syncthreads();
  m = max(max(s_amax[0], s_amax[1]), max(s_amax[2], s_amax[3]));
  const Fp8bScale f = fp8b_scale(m);
  if (tid == 0) {
    s[(e * rblocks + rb) * cblocks + cb] = f.scale;
    if (sT != nullptr) sT[(e * cblocks + cb) * rblocks + rb] = f.scale;
  }
  uint2 o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    o[i] = fp8b_encode8(x, f.inv);
    const int r = r0 + 8 * pg + i;
    if (r < R && col < C) *reinterpret_cast<uint2*>(q + plane + static_cast<long long>(r) * C + col) = o[i];
  }
  if (qT == nullptr) return;
  stage_transposed(o, s_t, cg, pg);
  __syncthreads();
  store_transposed(s_t, qT + plane + static_cast<long long>(c0) * R + r0, R, C - c0, R - r0);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_fp8b_quantize_rows(const uint16_t* x, const int32_t* dest, int T, int C, int k, uint8_t* q, float* s,
                                      void* stream) {
  MOE_CHECK_PTR(x); MOE_CHECK_PTR(q); MOE_CHECK_PTR(s);
  MOE_CHECK_ALIGN(x); MOE_CHECK_ALIGN(q); MOE_CHECK_ALIGN(s);
  if (dest) MOE_CHECK_ALIGN(dest);
  MOE_REQUIRE(T >= 1 && C >= 64 && C % 64 == 0, MOE_ERR_UNSUPPORTED, "need T >= 1 and C a multiple of 64");
  MOE_REQUIRE(k >= 1 && k <= 16 && (dest || k == 1), MOE_ERR_UNSUPPORTED, "k must be in [1, 16], and 1 without dest");
  const long long n = static_cast<long long>(T) * k;
  MOE_REQUIRE(n < (1LL << 31), MOE_ERR_UNSUPPORTED, "T*k must be < 2^31");
  const long long blocks = (static_cast<long long>(T) * fp8b_blocks(C) * 16 + kRowThreads - 1) / kRowThreads;
  MOE_REQUIRE(blocks * kRowThreads < (1LL << 32), MOE_ERR_UNSUPPORTED, "tensor too large (a launch has fewer than 2^32 threads)");
  if (dest)
    fp8b_rows_kernel<true><<<static_cast<unsigned>(blocks), kRowThreads, 0, as_stream(stream)>>>(x, dest, T, C, k, n, q, s);
  else
    fp8b_rows_kernel<false><<<static_cast<unsigned>(blocks), kRowThreads, 0, as_stream(stream)>>>(x, dest, T, C, k, n, q, s);
  return check_launch("fp8b_quantize_rows");
}

extern "C" int moe_fp8b_quantize_rows_grouped(const uint16_t* in, const int32_t* row_token, const float* row_gate,
                                              const int32_t* offsets, const int32_t* offsets_pad, int E, int n, int C,
                                              uint8_t* q, float* s, uint8_t* qT, float* sT, void* stream) {
  MOE_CHECK_PTR(in); MOE_CHECK_PTR(offsets); MOE_CHECK_PTR(offsets_pad); MOE_CHECK_PTR(qT); MOE_CHECK_PTR(sT);
  MOE_CHECK_ALIGN(in); MOE_CHECK_ALIGN(qT); MOE_CHECK_ALIGN(sT);
  MOE_REQUIRE((q == nullptr) == (s == nullptr), MOE_ERR_INVALID_ARG, "q and s come together");
  if (q) { MOE_CHECK_ALIGN(q); MOE_CHECK_ALIGN(s); }
  MOE_REQUIRE(E >= 1 && E <= 256, MOE_ERR_UNSUPPORTED, "E must be in [1, 256]");
  MOE_REQUIRE(n >= 1 && C >= 64 && C % 64 == 0, MOE_ERR_UNSUPPORTED, "need n >= 1 and C a multiple of 64");
  const int P = moe_mx_pad_cap(n, E);
  MOE_REQUIRE(P > 0, MOE_ERR_UNSUPPORTED, "padded token axis too long");
  const int ctiles = static_cast<int>(fp8b_blocks(C));
  const long long blocks = static_cast<long long>(P / kTile) * ctiles;
  MOE_REQUIRE(blocks <= 0x7fffffffLL, MOE_ERR_UNSUPPORTED, "too many tiles");
  hipStream_t st = as_stream(stream);
  auto run = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(blocks), kTileThreads, 0, st>>>(in, row_token, row_gate, offsets, offsets_pad, E, C, n, P,
                                                                   q, s, qT, sT, ctiles);
  };
  if (q) row_gate ? run(fp8b_grouped_kernel<true, true>) : run(fp8b_grouped_kernel<true, false>);
  else row_gate ? run(fp8b_grouped_kernel<false, true>) : run(fp8b_grouped_kernel<false, false>);
  return check_launch("fp8b_quantize_rows_grouped");
}

extern "C" int moe_fp8b_quantize_weights(const uint16_t* w, int E, int R, int C, uint8_t* q, float* s, uint8_t* qT,
                                         float* sT, void* stream) {
  MOE_CHECK_PTR(w); MOE_CHECK_PTR(q); MOE_CHECK_PTR(s);
  MOE_CHECK_ALIGN(w); MOE_CHECK_ALIGN(q); MOE_CHECK_ALIGN(s);
  MOE_REQUIRE((qT == nullptr) == (sT == nullptr), MOE_ERR_INVALID_ARG, "qT and sT come together");
  if (qT) { MOE_CHECK_ALIGN(qT); MOE_CHECK_ALIGN(sT); }
  MOE_REQUIRE(E >= 1, MOE_ERR_UNSUPPORTED, "E must be >= 1");
  MOE_REQUIRE(R >= 64 && R % 64 == 0 && C >= 64 && C % 64 == 0, MOE_ERR_UNSUPPORTED, "R and C must be multiples of 64");
  const int rblocks = static_cast<int>(fp8b_blocks(R)), cblocks = static_cast<int>(fp8b_blocks(C));
  const long long blocks = static_cast<long long>(E) * rblocks * cblocks;
  MOE_REQUIRE(blocks <= 0x7fffffffLL, MOE_ERR_UNSUPPORTED, "too many blocks");
  fp8b_weights_kernel<<<static_cast<unsigned>(blocks), kTileThreads, 0, as_stream(stream)>>>(w, R, C, rblocks, cblocks, q,
                                                                                            s, qT, sT);
  return check_launch("fp8b_quantize_weights");
}
