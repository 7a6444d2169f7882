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
// All are HBM-bound: 2 bytes read, 1 + 4/128 bytes written per element and layout.
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

// Transposes 8 x 8 codes in registers (row i: 8 columns' codes) and stages them as 8 column chunks.
__device__ __forceinline__ void stage_transposed(const uint2 (&o)[8], uint8_t* s_t, int cg, int pg) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a = j < 4 ? o[4 * h].x : o[4 * h].y, b = j < 4 ? o[4 * h + 1].x : o[4 * h + 1].y;
      const uint32_t c = j < 4 ? o[4 * h + 2].x : o[4 * h + 2].y, d = j < 4 ? o[4 * h + 3].x : o[4 * h + 3].y;
      const int sh = 8 * (j & 3);
      w[h] = ((a >> sh) & 0xffu) | (((b >> sh) & 0xffu) << 8) | (((c >> sh) & 0xffu) << 16) | (((d >> sh) & 0xffu) << 24);
    }
    *reinterpret_cast<uint2*>(s_t + tcode_off(8 * cg + j, pg)) = make_uint2(w[0], w[1]);
  }
}

// Column steps a grouped workgroup takes along its band of 128 positions.
constexpr int kBandSteps = 4;

// Grouped rows: padded position p of expert e holds grouped row r = offsets[e] + p - offsets_pad[e] while
// that is below offsets[e + 1]; its data is in[row_token ? row_token[r] : r], times row_gate[r] rounded
// to bf16 where given.  ROWS: also the real rows' row layout, q [n][C] and s [ceil(C/128)][n].
template <bool ROWS>
__global__ __launch_bounds__(kTileThreads) void fp8b_grouped_kernel(
    const uint16_t* __restrict__ in, const int32_t* __restrict__ row_token, const float* __restrict__ row_gate,
    const int32_t* __restrict__ offsets, const int32_t* __restrict__ offsets_pad, int E, int C, long long n, long long P,
    uint8_t* __restrict__ q, float* __restrict__ s, uint8_t* __restrict__ qT, float* __restrict__ sT, int cgroups) {
  __shared__ __attribute__((aligned(16))) uint8_t s_t[kTile * kTile];
  __shared__ uint32_t s_amax[16][kTile];
  __shared__ int s_row[kTile];
  const int tid = threadIdx.x, cg = tid & 15, pg = tid >> 4;
  const long long p0 = static_cast<long long>(blockIdx.x / cgroups) * kTile;
  int c0 = static_cast<int>(blockIdx.x % cgroups) * kTile * kBandSteps;
  if (tid < kTile) {
    const long long p = p0 + tid;
    int r = -1;
    if (p < offsets_pad[E]) {
      int lo = 0, hi = E - 1;                 // last e with offsets_pad[e] <= p
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (offsets_pad[mid] <= p) lo = mid; else hi = mid - 1;
      }
      const long long row = offsets[lo] + (p - offsets_pad[lo]);
      if (row < offsets[lo + 1] && row < n) r = static_cast<int>(row);
    }
    s_row[tid] = r;
  }
  __syncthreads();
  int row[8];
  long long src[8];
  float gate[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    row[i] = s_row[8 * pg + i];
    src[i] = row[i] < 0 ? -1 : (row_token != nullptr ? row_token[row[i]] : row[i]);
    gate[i] = row_gate != nullptr && row[i] >= 0 ? row_gate[row[i]] : 1.f;
  }
  for (int step = 0; step < kBandSteps && c0 < C; ++step, c0 += kTile) {
    const int col = c0 + 8 * cg;
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (src[i] >= 0 && col < C) v[i] = *reinterpret_cast<const uint4*>(in + src[i] * C + col);
    }
    uint32_t cmax[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[j] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      if (row_gate != nullptr) {
#pragma unroll
        for (int h = 0; h < 4; ++h) w[h] = pack_bf16x2(gate[i] * bf16_lo(w[h]), gate[i] * bf16_hi(w[h]));
        v[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        cmax[2 * h] = max(cmax[2 * h], w[h] & 0x7fffu);
        cmax[2 * h + 1] = max(cmax[2 * h + 1], (w[h] >> 16) & 0x7fffu);
      }
      if constexpr (ROWS) {
        const Fp8bScale f = fp8b_scale(max16(fp8b_amax8(w)));
        if (row[i] >= 0 && col < C) {
          *reinterpret_cast<uint2*>(q + static_cast<long long>(row[i]) * C + col) = fp8b_encode8(w, f.inv);
          if (cg == 0) s[(c0 / kTile) * n + row[i]] = f.scale;
        }
      }
    }
    __syncthreads();                 // the previous step's readers are done with the LDS
#pragma unroll
    for (int j = 0; j < 8; ++j) s_amax[pg][8 * cg + j] = cmax[j];
    __syncthreads();
    float inv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, s_amax[i][8 * cg + j]);
      const Fp8bScale f = fp8b_scale(m);
      inv[j] = f.inv;
      if (pg == 0 && col < C) sT[(p0 / kTile) * C + col + j] = f.scale;
    }
    uint2 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = make_uint2(fp8b_encode4(bf16_lo(v[i].x) * inv[0], bf16_hi(v[i].x) * inv[1], bf16_lo(v[i].y) * inv[2],
                                     bf16_hi(v[i].y) * inv[3]),
                        fp8b_encode4(bf16_lo(v[i].z) * inv[4], bf16_hi(v[i].z) * inv[5], bf16_lo(v[i].w) * inv[6],
                                     bf16_hi(v[i].w) * inv[7]));
    stage_transposed(o, s_t, cg, pg);
    __syncthreads();
    store_transposed(s_t, qT + c0 * P + p0, P, C - c0, kTile);
  }
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
  MOE_REQUIRE(blocks <= 0x7fffffffLL, MOE_ERR_UNSUPPORTED, "tensor too large");
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
  const int cgroups = static_cast<int>((fp8b_blocks(C) + kBandSteps - 1) / kBandSteps);
  const long long blocks = static_cast<long long>(P / kTile) * cgroups;
  MOE_REQUIRE(blocks <= 0x7fffffffLL, MOE_ERR_UNSUPPORTED, "too many tiles");
  hipStream_t st = as_stream(stream);
  if (q)
    fp8b_grouped_kernel<true><<<static_cast<unsigned>(blocks), kTileThreads, 0, st>>>(
        in, row_token, row_gate, offsets, offsets_pad, E, C, n, P, q, s, qT, sT, cgroups);
  else
    fp8b_grouped_kernel<false><<<static_cast<unsigned>(blocks), kTileThreads, 0, st>>>(
        in, row_token, row_gate, offsets, offsets_pad, E, C, n, P, q, s, qT, sT, cgroups);
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
