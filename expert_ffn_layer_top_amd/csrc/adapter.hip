// Low-rank adapters of many requests beside the experts' products: every routed row may have an adapter of
// its own (its token's), and of each adapter the matrices of its expert take part.
//
// [news] "Ai2 rebuilds Olmo's training stack for trillion-parameter MoEs", lead paragraphs: a router sends each
// token to a small selection of experts; "Routing work stays on the GPU": rows lie by expert in the expert
// buffers, and what is known about them stays on the device.
//
// Three products make up the forward and the backward.  With W [R][C] the matrix of one adapter and expert:
//   shrink   v[row][R]   = x[row][C] W^T       contracts over a long axis:  A x, and B^T dy, B^T dg in the backward
//   expand   y[row][C]  += s v[row][R] W       contracts over the rank:     B v, and A^T dv in the backward
//   wgrad    dW[R][C]    = v^T y               contracts over the rows of one adapter and expert
// B is stored by rank like A ([R][out]), so each of them serves A and B.  All three move far more bytes than
// the matrix cores need time for (R operations per byte of x or y), so they are built as streams for
// v_mfma_f32_16x16x32_bf16.  Shrink stages whole cache lines of x and W in LDS.  In expand and wgrad the long operands
// go straight from memory into fragments, and what those would have transposed is permuted in registers: a lane loads 16
// bytes of each of 8 rows along the contraction; the 8 columns that it holds become 8 column tiles, of which tile i takes
// column 8 c + i from lane c, so its accumulators hold 8 neighbouring columns and leave as 16-byte stores.
//
// Between its two products v is held in fp32, and goes into the second one as the sum of three bf16 values, each what those
// before it lack: 24 bits of mantissa, all that fp32 has.  With two of them (16 bits) 4 to 15 times as many results differ from the
// rounded 64-bit ones (4012 rows of d 2112, f 1344: 2.0e-3 of a' against 1.2e-4, 7.7e-3 of y' against 5.0e-4), for a
// percent or two: training forward of 131072 rows 1686 us against 1704, backward of 32768 359 and 368, of 131072 1940 and 1921.
//
// Rows are taken in tiles of up to 64 rows of one expert and adapter, from a list that adapter_plan makes on the
// device by a stable sort of each expert's rows by adapter, so sums run in a fixed order.  Where tiles are few or small,
// one kernel makes v and what is added; for few rows there is no list, and one kernel does both products of a row.
#include <hip/hip_runtime.h>

#include "common.h"
#include "dropout.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// Fragments are native vectors: kept across a loop as structs, they become four registers each that are copied at its
// head, which waits for their loads.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kTileRows = 64;      // rows of a tile
constexpr int kPlanBlock = 512;    // rows that a workgroup of the sort looks at together
constexpr int kSmallPlan = 4096;   // up to this many rows one workgroup makes the whole plan
constexpr int kMaxRank = 64;
constexpr int kMaxAdapters = 256;

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ u32x4 load16(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }
__device__ __forceinline__ void store16(uint16_t* p, u32x4 v) { *reinterpret_cast<u32x4*>(p) = v; }

// x = hi + mid + lo, three bf16 values (two rounded remainders of 24 bits leave at most 8); mid and lo are 0 where hi is not finite.
__device__ __forceinline__ float lack(float x, float hi) { return __builtin_isfinite(hi) ? x - hi : 0.f; }
constexpr int kSplit = 3;

// A wave's own LDS accesses keep their order; this keeps the compiler from changing it.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------- the plan

// Rows of one piece of a group's contraction in the weight gradients: pieces enough for the chip where few
// groups hold the rows.  A piece's fp32 sums are written and read, 8 R C bytes against the 2 C of each of its rows: with 2048 rows
// an eighth of the rows' own bytes for 64 ranks and less for fewer, with 256 (up to 8192 rows) as much as they for 64 ranks and
// twice that for A's 128 of gate/up.  A 32nd of the rows: the backward of 32768 rows of 64 experts took 363 us, 387 with a 64th (most experts
// then have two pieces), and that of 32768 rows of one expert, wider, 703 and 745.
__host__ __device__ inline int piece_rows(int n) {
  const int want = (n + 31) / 32;
  return want <= 256 ? 256 : want >= 2048 ? 2048 : (want + 31) / 32 * 32;
}

// The sort takes 5.6 + 6.1 + 6.3 us for 32768 rows of 64 experts and one adapter, 12 for the scan with 32 adapters.
// Rows of one expert that a workgroup of it takes: about 128 workgroups and one for each expert, so that the scan
// over an expert's chunks stays short.
__host__ __device__ inline int chunk_rows(int n) {
  return ((n + 127) / 128 + kPlanBlock - 1) / kPlanBlock * kPlanBlock;
}

struct Tile {
  int pos, count, e, l;   // rows [pos, pos + count) of the sorted list
};

// The plan's parts, as offsets in 4-byte words of its buffer.
struct PlanLayout {
  int chunks, pairs, tiles_cap, items_cap, multi_cap;
  long long rows, toks, goff, tile0, tiles, items, multi, hist, words;
};

constexpr int kHeadTiles = 0, kHeadItems = 1, kHeadMulti = 2, kHeadWords = 16;

__host__ __device__ inline PlanLayout plan_layout(int n, int E, int L) {
  PlanLayout p;
  p.chunks = n / chunk_rows(n) + E;
  p.pairs = E * (L + 1);
  const int groups = n < p.pairs ? n : p.pairs;
  p.tiles_cap = n / kTileRows + groups;
  p.items_cap = n / piece_rows(n) + E * L;
  p.multi_cap = n / piece_rows(n) + 1;
  long long at = kHeadWords;
  auto take = [&](long long words) {
    const long long here = at;
    at += (words + 3) / 4 * 4;
    return here;
  };
  p.rows = take(n);
  p.toks = take(n);
  p.goff = take(p.pairs + 1);
  p.tile0 = take(p.pairs);
  p.tiles = take(4LL * p.tiles_cap);
  p.items = take(4LL * p.items_cap);
  p.multi = take(p.multi_cap);
  p.hist = take(static_cast<long long>(p.chunks) * (L + 1));
  p.words = at;
  return p;
}

// The experts' first rows, begin[0 .. E], from the offsets: within [0, n] and never falling, whatever the offsets hold, so
// that the plan's parts hold whatever follows from them.  The first 256 threads of the workgroup do it, all call it.
__device__ __forceinline__ void load_begins(const int32_t* offsets, int E, int n, int (&begin)[257]) {
  __shared__ int most[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int v = tid < 256 && tid <= E ? min(max(offsets[tid], 0), n) : 0;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v = max(v, u);
  }
  if (lane == 63 && wave < 4) most[wave] = v;
  __syncthreads();
  for (int w = 0; w < min(wave, 4); ++w) v = max(v, most[w]);
  if (tid < 256 && tid <= E) begin[tid] = v;
  if (tid == 255 && E == 256) begin[256] = max(v, min(max(offsets[256], 0), n));
  __syncthreads();
}

// A row's token, within [0, T), and its adapter, L for none (also where the token is no token).
__device__ __forceinline__ int token_of(const int32_t* row_token, int row, int T) {
  return row_token != nullptr ? min(max(row_token[row], 0), T - 1) : row;
}
__device__ __forceinline__ int adapter_of(const int32_t* ids, const int32_t* row_token, int row, int T, int L) {
  const int t = row_token != nullptr ? row_token[row] : row;
  if (t < 0 || t >= T) return L;
  const int l = ids[t];
  return l >= 0 && l < L ? l : L;
}

struct Chunk {
  int e, begin, end, index;   // index < 0: there is none
};

// The rows that chunk `want` holds: chunks are counted expert by expert, each of up to chunk_rows(n) rows of one.
// All 256 threads call it (E <= 256: thread e looks at expert e).
__device__ __forceinline__ Chunk find_chunk(const int32_t* offsets, int E, int n, int want) {
  __shared__ int sums[4], found[3], begin[257];
  load_begins(offsets, E, n, begin);
  const int e = threadIdx.x, lane = e & 63, wave = e >> 6, size = chunk_rows(n);
  const int lo = e < E ? begin[e] : 0, hi = e < E ? begin[e + 1] : 0;
  const int mine = (hi - lo + size - 1) / size;
  int run = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(run, o, 64);
    if (lane >= o) run += v;
  }
  if (lane == 63) sums[wave] = run;
  if (e == 0) found[0] = -1;
  __syncthreads();
  int base = run - mine;
  for (int w = 0; w < wave; ++w) base += sums[w];
  if (want >= base && want < base + mine) {
    found[0] = e;
    found[1] = lo + (want - base) * size;
    found[2] = hi;
  }
  __syncthreads();
  Chunk c;
  c.e = found[0];
  c.index = c.e < 0 ? -1 : want;
  c.begin = found[1];
  c.end = min(found[2], found[1] + size);
  return c;
}

// Rows of each adapter in every chunk.
__global__ __launch_bounds__(256) void plan_count_kernel(const int32_t* __restrict__ ids, const int32_t* __restrict__ row_token,
                                                         const int32_t* __restrict__ offsets, int T, int n, int E, int L,
                                                         int32_t* __restrict__ plan) {
  __shared__ int count[kMaxAdapters + 1];
  const PlanLayout p = plan_layout(n, E, L);
  const Chunk c = find_chunk(offsets, E, n, blockIdx.x);
  if (c.index < 0) return;
  for (int l = threadIdx.x; l <= L; l += 256) count[l] = 0;
  __syncthreads();
  for (int r = c.begin + threadIdx.x; r < c.end; r += 256) atomicAdd(&count[adapter_of(ids, row_token, r, T, L)], 1);
  __syncthreads();
  int32_t* hist = plan + p.hist + static_cast<long long>(blockIdx.x) * (L + 1);
  for (int l = threadIdx.x; l <= L; l += 256) hist[l] = count[l];
}

// Exclusive sums over 1024 threads of four counts; `total` gets the sums over all.
__device__ __forceinline__ int4 scan4(int4 v, int4* total) {
  __shared__ int4 sums[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int4 run = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int4 u = make_int4(__shfl_up(run.x, o, 64), __shfl_up(run.y, o, 64), __shfl_up(run.z, o, 64), __shfl_up(run.w, o, 64));
    if (lane >= o) run = make_int4(run.x + u.x, run.y + u.y, run.z + u.z, run.w + u.w);
  }
  if (lane == 63) sums[wave] = run;
  __syncthreads();
  int4 base = make_int4(0, 0, 0, 0), all = base;
  for (int w = 0; w < 16; ++w) {
    const int4 s = sums[w];
    if (w < wave) base = make_int4(base.x + s.x, base.y + s.y, base.z + s.z, base.w + s.w);
    all = make_int4(all.x + s.x, all.y + s.y, all.z + s.z, all.w + s.w);
  }
  *total = all;
  return make_int4(base.x + run.x - v.x, base.y + run.y - v.y, base.z + run.z - v.z, base.w + run.w - v.w);
}

// Positions of every (expert, adapter) in the sorted list, of its tiles and of its pieces for the weight gradients.  1024
// threads, of which each takes consecutive pairs (their number is E (L + 1)); count(q): a pair's rows, start(q, pos): told
// where they begin.
template <class Count, class Start>
__device__ __forceinline__ void plan_positions(const PlanLayout& p, int n, int L, int32_t* plan, Count count, Start start) {
  int4 total;
  const int per = (p.pairs + 1023) / 1024, first = threadIdx.x * per, last = min(first + per, p.pairs);
  const int piece = piece_rows(n);
  int32_t* goff = plan + p.goff;
  int4 sum = make_int4(0, 0, 0, 0);   // rows, tiles, pieces, groups of several pieces
  for (int q = first; q < last; ++q) {
    const int rows = count(q);
    goff[q] = rows;
    sum.x += rows;
    sum.y += (rows + kTileRows - 1) / kTileRows;
    if (q % (L + 1) < L) {
      sum.z += rows > piece ? (rows + piece - 1) / piece : 1;
      sum.w += rows > piece;
    }
  }
  int4 at = scan4(sum, &total);
  Tile* items = reinterpret_cast<Tile*>(plan + p.items);
  for (int q = first; q < last; ++q) {
    const int e = q / (L + 1), l = q - e * (L + 1), rows = goff[q];
    goff[q] = at.x;
    plan[p.tile0 + q] = at.y;
    start(q, at.x);
    if (l < L) {
      const int pieces = rows > piece ? (rows + piece - 1) / piece : 1;
      for (int i = 0; i < pieces; ++i) items[at.z + i] = {at.x + i * piece, min(piece, rows - i * piece), e, l};
      if (rows > piece) plan[p.multi + at.w] = q;
      at.z += pieces;
      at.w += rows > piece;
    }
    at.x += rows;
    at.y += (rows + kTileRows - 1) / kTileRows;
  }
  if (threadIdx.x == 0) {
    goff[p.pairs] = total.x;
    plan[kHeadTiles] = total.y;
    plan[kHeadItems] = total.z;
    plan[kHeadMulti] = total.w;
  }
}

// The positions from the chunks' counts, which become the chunks' own positions.
__global__ __launch_bounds__(1024) void plan_scan_kernel(const int32_t* __restrict__ offsets, int n, int E, int L,
                                                         int32_t* __restrict__ plan) {
  __shared__ int chunk0[257], begin[257];
  const PlanLayout p = plan_layout(n, E, L);
  const int size = chunk_rows(n);
  load_begins(offsets, E, n, begin);
  int mine = 0;
  if (threadIdx.x < static_cast<unsigned>(E)) mine = (begin[threadIdx.x + 1] - begin[threadIdx.x] + size - 1) / size;
  int4 total;
  const int4 at = scan4(make_int4(mine, 0, 0, 0), &total);
  if (threadIdx.x < static_cast<unsigned>(E)) chunk0[threadIdx.x] = at.x;
  if (threadIdx.x == 0) chunk0[E] = total.x;
  __syncthreads();
  int32_t* hist = plan + p.hist;
  plan_positions(
      p, n, L, plan,
      [&](int q) {
        const int e = q / (L + 1), l = q - e * (L + 1);
        int rows = 0;
#pragma unroll 8
        for (int c = chunk0[e]; c < chunk0[e + 1]; ++c) rows += hist[static_cast<long long>(c) * (L + 1) + l];
        return rows;
      },
      [&](int q, int pos) {
        const int e = q / (L + 1), l = q - e * (L + 1);
#pragma unroll 8
        for (int c = chunk0[e]; c < chunk0[e + 1]; ++c) {
          int32_t* h = &hist[static_cast<long long>(c) * (L + 1) + l];
          const int here = *h;
          *h = pos;
          pos += here;
        }
      });
}

// Lanes of the wave whose `l` (9 bits) is this lane's, of those that are `live`.
__device__ __forceinline__ unsigned long long same_lanes(int l, bool live) {
  unsigned long long same = __ballot(live);
  for (int b = 0; b < 9; ++b) {
    const unsigned long long set = __ballot((l >> b) & 1);
    same &= ((l >> b) & 1) ? set : ~set;
  }
  return same;
}

// A row's place in the list, and where it is a tile's first, the tile.
__device__ __forceinline__ void place_row(int32_t* plan, const PlanLayout& p, const int32_t* row_token, int T, int L, int r,
                                          int e, int l, int pos) {
  const int q = e * (L + 1) + l, in = pos - plan[p.goff + q];
  plan[p.rows + pos] = r;
  plan[p.toks + pos] = token_of(row_token, r, T);
  if (in % kTileRows == 0)
    reinterpret_cast<Tile*>(plan + p.tiles)[plan[p.tile0 + q] + in / kTileRows] =
        Tile{pos, min(kTileRows, plan[p.goff + q + 1] - pos), e, l};
}

// The sorted list and the tiles.  A row's rank among those of its adapter is its position's count of equal
// adapters in the wave, plus those of the block's earlier groups of 64, plus the chunk's earlier blocks.
__global__ __launch_bounds__(256) void plan_place_kernel(const int32_t* __restrict__ ids, const int32_t* __restrict__ row_token,
                                                         const int32_t* __restrict__ offsets, int T, int n, int E, int L,
                                                         int32_t* __restrict__ plan) {
  constexpr int kGroups = kPlanBlock / 64;
  __shared__ int before[kGroups][kMaxAdapters + 1], run[kMaxAdapters + 1];
  const PlanLayout p = plan_layout(n, E, L);
  const Chunk c = find_chunk(offsets, E, n, blockIdx.x);
  if (c.index < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int a = threadIdx.x; a <= L; a += 256) run[a] = plan[p.hist + static_cast<long long>(blockIdx.x) * (L + 1) + a];
  for (int begin = c.begin; begin < c.end; begin += kPlanBlock) {
    __syncthreads();
    for (int i = threadIdx.x; i < kGroups * (kMaxAdapters + 1); i += 256) (&before[0][0])[i] = 0;
    __syncthreads();
    int l[kGroups / 4], rank[kGroups / 4];
#pragma unroll
    for (int i = 0; i < kGroups / 4; ++i) {
      const int g = i * 4 + wave, r = begin + g * 64 + lane;
      const bool live = r < c.end;
      l[i] = live ? adapter_of(ids, row_token, r, T, L) : -1;
      const unsigned long long same = same_lanes(l[i], live);
      rank[i] = __popcll(same & ((1ull << lane) - 1));
      if (live && rank[i] == 0) before[g][l[i]] = __popcll(same);
    }
    __syncthreads();
    for (int a = threadIdx.x; a <= L; a += 256) {
      int at = run[a];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int here = before[g][a];
        before[g][a] = at;
        at += here;
      }
      run[a] = at;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGroups / 4; ++i) {
      const int g = i * 4 + wave, r = begin + g * 64 + lane;
      if (r < c.end) place_row(plan, p, row_token, T, L, r, c.e, l[i], before[g][l[i]] + rank[i]);
    }
  }
}

// The whole plan of up to kSmallPlan rows in one workgroup: a wave walks the rows of one expert after another, 64 at a
// time, and keeps their adapters and ranks in LDS until the positions are known.  4012 rows take 12.7 us, a chain of
// about ten accesses to memory with a barrier after each (in the three kernels of more rows 14.5, and two launches more).
__global__ __launch_bounds__(1024) void plan_small_kernel(const int32_t* __restrict__ ids, const int32_t* __restrict__ row_token,
                                                          const int32_t* __restrict__ offsets, int T, int n, int E, int L,
                                                          int32_t* __restrict__ plan) {
  __shared__ int begin[257], run[16][kMaxAdapters + 1];
  __shared__ uint16_t adapter[kSmallPlan], rank[kSmallPlan];
  const PlanLayout p = plan_layout(n, E, L);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int kMine = kSmallPlan / 1024;
  int token[kMine], mine[kMine];       // all loads at once
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int r = min(tid + 1024 * i, n - 1);
    token[i] = row_token != nullptr ? row_token[r] : r;
  }
#pragma unroll
  for (int i = 0; i < kMine; ++i) mine[i] = ids[min(max(token[i], 0), T - 1)];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (token[i] < 0 || token[i] >= T || mine[i] < 0 || mine[i] >= L) mine[i] = L;
    if (tid + 1024 * i < n) adapter[tid + 1024 * i] = static_cast<uint16_t>(mine[i]);
  }
  load_begins(offsets, E, n, begin);
  __syncthreads();
  for (int e = wave; e < E; e += 16) {
    for (int a = lane; a <= L; a += 64) run[wave][a] = 0;
    wave_fence();
    for (int r0 = begin[e]; r0 < begin[e + 1]; r0 += 64) {
      const int r = r0 + lane;
      const bool live = r < begin[e + 1];
      const int l = live ? adapter[r] : -1;
      const unsigned long long same = same_lanes(l, live);
      const int in = __popcll(same & ((1ull << lane) - 1)), before = live ? run[wave][l] : 0;
      wave_fence();
      if (live) rank[r] = static_cast<uint16_t>(before + in);
      if (live && in == 0) run[wave][l] = before + __popcll(same);
      wave_fence();
    }
    for (int a = lane; a <= L; a += 64) plan[p.tile0 + e * (L + 1) + a] = run[wave][a];
    wave_fence();
  }
  __threadfence_block();
  __syncthreads();
  plan_positions(
      p, n, L, plan, [&](int q) { return plan[p.tile0 + q]; }, [](int, int) {});
  __threadfence_block();
  __syncthreads();
  // the rows' experts (the last that begins at or before each), their groups' positions, and what is written
  int e[kMine], first[kMine], past[kMine], tile0[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) e[i] = 0;
#pragma unroll
  for (int step = 128; step > 0; step /= 2)
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (e[i] + step < E && begin[e[i] + step] <= tid + 1024 * i) e[i] += step;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int q = e[i] * (L + 1) + mine[i];
    first[i] = plan[p.goff + q];
    past[i] = plan[p.goff + q + 1];
    tile0[i] = plan[p.tile0 + q];
  }
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int r = tid + 1024 * i;
    if (r >= n || r < begin[e[i]] || r >= begin[e[i] + 1]) continue;
    const int in = rank[r], pos = first[i] + in;
    plan[p.rows + pos] = r;
    plan[p.toks + pos] = min(max(token[i], 0), T - 1);
    if (in % kTileRows == 0)
      reinterpret_cast<Tile*>(plan + p.tiles)[tile0[i] + in / kTileRows] = Tile{pos, min(kTileRows, past[i] - pos), e[i], mine[i]};
  }
}

// ---------------------------------------------------------------- the rows of a call

struct Rows {
  const int32_t* plan;        // null in the kernel of few rows only
  const int32_t* ids;
  const int32_t* row_token;   // null: row r is token r
  const int32_t* offsets;
  int T, n, E, L;
};

// Tile `i`, the same in all lanes.
__device__ __forceinline__ Tile tile_at(const Rows& rows, const PlanLayout& p, int i) {
  const int4 t = reinterpret_cast<const int4*>(rows.plan + p.tiles)[i];
  return {__builtin_amdgcn_readfirstlane(t.x), __builtin_amdgcn_readfirstlane(t.y), __builtin_amdgcn_readfirstlane(t.z),
          __builtin_amdgcn_readfirstlane(t.w)};
}

__device__ __forceinline__ int n_tiles(const Rows& rows) { return rows.plan[kHeadTiles]; }

// Row at sorted position pos (clamped by the caller to the tile).
__device__ __forceinline__ int row_at(const Rows& rows, const PlanLayout& p, int pos) { return rows.plan[p.rows + pos]; }

// The shrink's items by workgroup: those of XCD x (workgroups x mod 8) are one contiguous run of the order, so that the
// tiles of one expert and adapter, which read the same matrix, share an L2 (131072 rows of 4096 by 32 ranks: 274 -> 263
// us).  gridDim.x is a multiple of 8.  Expand and the weight gradients take their items as they come: there, hot experts
// left whole XCDs with more to do (82 -> 109 us and 260 -> 365 us in runs).
struct Run {
  long long at, end, step;
};
__device__ __forceinline__ Run xcd_run(long long items) {
  const long long per = (items + 7) / 8, first = (blockIdx.x & 7) * per;
  return {first + (blockIdx.x >> 3), first + per < items ? first + per : items, gridDim.x >> 3};
}

// ---------------------------------------------------------------- shrink

struct ShrinkArgs {
  Rows rows;
  const uint16_t* x[2];    // up to two products in a launch (blockIdx.y): dg and du
  const uint16_t* w[2];
  int v0[2];               // their first columns in v
  int gather;              // x by token (through row_token)
  int K, R, ldv, S;        // slices of K
  int parts;               // a tile's rows are shared among this many workgroups (1, 2 or 4)
  const float* scale;      // null, or [L]: factor of v
  float* part;             // v [S][n][ldv], the sums of the slices
  uint16_t* v;             // [n][ldv], or null: v rounded, where there is one slice
  DropArgs drop;
};

// Staging of a wave: rows of 128 bytes (64 elements of K) of x and of W.  16-byte chunk k of row r is held at chunk
// k ^ (r / 2 % 8), so that both the 8 rows that a wave writes at once and the 16 that it reads lie in different banks.
// Within rows 8 i + r (writes) that depends on i by its lowest bit alone, within rows 16 b + r (reads) not on b.
__device__ __forceinline__ int staged(int row, int chunk) { return row * 8 + (chunk ^ ((row >> 1) & 7)); }

// One tile (NB blocks of 16 rows) times RT tiles of 16 ranks over K's units of 64 elements u0, u0 + STEP, ...  A load takes
// 8 rows of a whole cache line each; rows go through registers, where they wait for memory while the unit before them
// is multiplied, into the wave's staging, and come from there as operands.  Rows past the tile and ranks past R are copies
// of the last one, which nobody stores.
//
// What bounds it is memory: 131072 rows of 4096 (1.07 GB) by 32 ranks of 512 matrices take 250 to 263 us, and the L2s miss 1.33 GB
// in that time, 5.0 to 5.3 TB/s; a stream of the same rows alone reaches 5.5 to 6.  Loading fragments without the staging (16
// rows of 16 bytes in neighbouring lanes) with two units of loads in registers took 282: registers left two waves per
// SIMD, here there are three (four for 16 ranks without dropout, two for 64, one for 128).  With dropout 32 ranks do not fit
// three waves a SIMD and spill 18 registers (76 bytes of scratch a lane), 64 ranks 2.  A tile's K starting at a
// place of its own, so that fewer workgroups read the same columns at once, changed nothing.
template <int NB, int RT, bool DROP, int STEP = 4>
__device__ __forceinline__ void shrink_tile(const ShrinkArgs& a, const Tile& t, const PlanLayout& p, const uint16_t* x,
                                            const uint16_t* w, int u0, int u1, u32x4* lds, f32x4 (&acc)[NB][RT]) {
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4, lr = lane >> 3, lc = lane & 7;
  const uint16_t* xp[2 * NB];
  uint32_t row[2 * NB], wo[2 * RT];
#pragma unroll
  for (int i = 0; i < 2 * NB; ++i) {
    const int pos = t.pos + min(8 * i + lr, t.count - 1), r = row_at(a.rows, p, pos);
    int src = r;
    if (a.gather) src = a.rows.plan[p.toks + pos];
    row[i] = static_cast<uint32_t>(r);
    xp[i] = x + static_cast<long long>(src) * a.K + 8 * lc;
  }
#pragma unroll
  for (int i = 0; i < 2 * RT; ++i) wo[i] = static_cast<uint32_t>(min(8 * i + lr, a.R - 1)) * a.K + 8 * lc;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[b][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  DropKey key;
  if (DROP) key = drop_key(a.drop);
  const int w0 = staged(lr, lc), w1 = staged(8 + lr, lc) - 64, f0 = staged(c, q), f1 = staged(c, 4 + q);
  constexpr int kW = 16 * NB * 8;        // W's rows follow x's
  u32x4 xr[2 * NB], wr[2 * RT];
  auto load = [&](int u) {
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) xr[i] = load16(xp[i] + 64 * u);
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) wr[i] = load16(w + (wo[i] + 64u * u));
    __builtin_amdgcn_sched_barrier(0);
  };
  auto put = [&](int u) {
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
      if (DROP) xr[i] = drop_zero(key, row[i], 8 * u + lc, xr[i]);
      lds[(i & 1 ? w1 : w0) + 64 * i] = xr[i];
    }
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) lds[(i & 1 ? w1 : w0) + kW + 64 * i] = wr[i];
    wave_fence();
  };
  auto multiply = [&] {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 xf[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) xf[b] = lds[(h ? f1 : f0) + 128 * b];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const u32x4 wf = lds[(h ? f1 : f0) + kW + 128 * i];
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b][i] = mfma(xf[b], wf, acc[b][i]);
      }
    }
    wave_fence();
  };
  if (u0 >= u1) return;
  int u = u0;
  load(u);
  for (; u + STEP < u1; u += STEP) {
    put(u);
    load(u + STEP);
    multiply();
  }
  put(u);
  multiply();
}

// The four waves' sums joined through LDS, two tiles of ranks at a time, and stored.
template <int NB, int RT, bool DROP>
__device__ __forceinline__ void shrink_run(const ShrinkArgs& a, const Tile& t, const PlanLayout& p, int which, int slice,
                                           u32x4* stage) {
  f32x4* lds = reinterpret_cast<f32x4*>(stage);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int units = a.K / 64;
  const int s0 = static_cast<int>(static_cast<long long>(units) * slice / a.S);
  const int s1 = static_cast<int>(static_cast<long long>(units) * (slice + 1) / a.S);
  const uint16_t* w = a.w[which] + (static_cast<long long>(t.l) * a.rows.E + t.e) * a.R * a.K;
  f32x4 acc[NB][RT];
  __syncthreads();    // the last tile's sums have been read
  shrink_tile<NB, RT, DROP>(a, t, p, a.x[which], w, s0 + wave, s1, stage + wave * (4 + RT) * 128, acc);
  float f = a.scale != nullptr ? a.scale[t.l] : 1.f;
  if (DROP) f *= drop_scale(a.drop.drop);
  constexpr int G = RT < 2 ? RT : 2;
#pragma unroll
  for (int i0 = 0; i0 < RT; i0 += G) {
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < G; ++i) lds[((wave * NB + b) * G + i) * 64 + lane] = acc[b][i0 + i];
    __syncthreads();
    for (int at = threadIdx.x; at < NB * G * 64; at += 256) {
      f32x4 s = lds[at];
#pragma unroll
      for (int o = 1; o < 4; ++o) s += lds[o * NB * G * 64 + at];
      const int b = at / (G * 64), rank = 16 * (i0 + at / 64 % G) + (at & 15), m = 16 * b + 4 * (at >> 4 & 3);
      if (rank >= a.R) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (m + j >= t.count) break;
        const long long r = row_at(a.rows, p, t.pos + m + j);
        a.part[(static_cast<long long>(slice) * a.rows.n + r) * a.ldv + a.v0[which] + rank] = f * s[j];
        if (a.v != nullptr && a.S == 1) a.v[r * a.ldv + a.v0[which] + rank] = f32_to_bf16(f * s[j]);
      }
    }
  }
}

template <int RT, bool DROP>
__global__ __launch_bounds__(256, RT == 1 && !DROP ? 4 : RT <= 2 ? 3 : RT == 4 ? 2 : 1) void adapter_shrink_kernel(ShrinkArgs a) {
  __shared__ u32x4 lds[4 * (4 + RT) * 128];   // 2 KiB for 16 rows or ranks; the sums take at most two thirds of it
  const PlanLayout p = plan_layout(a.rows.n, a.rows.E, a.rows.L);
  const int each = a.S * a.parts, rows_each = kTileRows / a.parts;
  const long long items = static_cast<long long>(n_tiles(a.rows)) * each;
  const int which = blockIdx.y;
  const Run run = xcd_run(items);
  for (long long i = run.at; i < run.end; i += run.step) {
    Tile t = tile_at(a.rows, p, static_cast<int>(i / each));
    const int slice = static_cast<int>(i % a.S), first = static_cast<int>(i % each / a.S) * rows_each;
    t.pos += first;
    t.count = min(t.count - first, rows_each);
    if (t.count <= 0) continue;
    if (t.l >= a.rows.L) {   // no adapter: v is 0 (with slices, expand writes that), and nobody reads it here
      if (a.v != nullptr && a.S == 1)
        for (int at = threadIdx.x; at < t.count * a.R; at += 256)
          a.v[static_cast<long long>(row_at(a.rows, p, t.pos + at / a.R)) * a.ldv + a.v0[which] + at % a.R] = 0;
      continue;
    }
    const int nb = (t.count + 15) / 16;
    if (nb == 1) shrink_run<1, RT, DROP>(a, t, p, which, slice, lds);
    else if (nb == 2) shrink_run<2, RT, DROP>(a, t, p, which, slice, lds);
    else shrink_run<4, RT, DROP>(a, t, p, which, slice, lds);
  }
}

// ---------------------------------------------------------------- expand
//
// A wave takes 16 rows after another of a tile and 128 columns, for which it holds W's fragments.  It reads what it adds to
// and writes the sum, and that is what it costs: SwiGLU of 131072 x 2048 takes 491 us (2.7 GB, 5.5 TB/s), the addition to
// 131072 x 7168 685 us (3.8 GB, 5.5 TB/s); a copy runs at 4.9.  The loads of the first 16 rows are issued before W's, on
// whose arrival everything else waits; where a launch has few tiles their rows are shared among up to four waves (4012 rows
// of 1344: 27 -> 14 us, before one kernel did both products of such calls).

enum { kAdd = 0, kSwiglu = 1, kSwigluBwd = 2 };

struct ExpandArgs {
  Rows rows;
  const float* part;        // v [S][n][ldv], as shrink left it
  int ldv, S, R, N;         // R: ranks of one product
  int parts;                // a tile's rows are shared among this many waves (1, 2 or 4)
  const uint16_t* w[2];     // kSwiglu: gate and up (v's columns [0, R) and [R, 2 R))
  const float* scale;       // null, or [L]
  const uint16_t* in[4];    // kAdd: y; kSwiglu: g, u, a; kSwigluBwd: g, u, dg, du
  uint16_t* out[3];         // kAdd: y; kSwiglu: g, u (or null), a; kSwigluBwd: dg, du
  uint16_t* v_out;          // with slices: v rounded, and in fp32, where they are wanted
  float* sum_out;
  DropArgs drop;
};

// Logistic function with the hardware reciprocal (about 1 ulp), as the experts' products have it.
__device__ __forceinline__ float logistic(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

__device__ __forceinline__ void unpack8(const u32x4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

// 8 rows (the contraction) of 8 columns -> for each column its 8 rows: tile i's fragment is o[i].
__device__ __forceinline__ void transpose8(const u32x4 (&r)[8], u32x4 (&o)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)        // rows 2 j, 2 j + 1
#pragma unroll
    for (int h = 0; h < 4; ++h) {    // columns 2 h, 2 h + 1
      const uint32_t lo = r[2 * j][h], hi = r[2 * j + 1][h];
      o[2 * h][j] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
      o[2 * h + 1][j] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
    }
}

// w's fragments for 128 columns: ranks 32 k + 8 q .. + 7 of the columns that the lane holds, 0 past R.
template <int KS>
__device__ __forceinline__ void load_w(const uint16_t* w, int R, int N, int col, u32x4 (&f)[KS][8]) {
  const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    u32x4 r[8];
    const bool live = 32 * k + 8 * q < R;
    const uint16_t* at = w + static_cast<long long>(live ? 32 * k + 8 * q : 0) * N + col;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r[j] = load16(at + static_cast<long long>(j) * N);
      if (!live) r[j] = u32x4{0, 0, 0, 0};
    }
    transpose8(r, f[k]);
  }
}

// 8 ranks of one row of v: the slices' sums in their order.
__device__ __forceinline__ void load_v(const ExpandArgs& a, long long row, int col, float (&f)[8]) {
  const float* at = a.part + row * a.ldv + col;
  if (a.S == 1) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(at), y = *reinterpret_cast<const f32x4*>(at + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = x[i];
      f[4 + i] = y[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 0.f;
  const long long step = static_cast<long long>(a.rows.n) * a.ldv;
  for (int s = 0; s < a.S; s += 4) {       // four slices' loads in flight; past the last one it is read again and not added
    f32x4 x[4], y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float* from = at + min(s + j, a.S - 1) * step;
      x[j] = *reinterpret_cast<const f32x4*>(from);
      y[j] = *reinterpret_cast<const f32x4*>(from + 4);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (s + j >= a.S) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] += x[j][i];
        f[4 + i] += y[j][i];
      }
    }
  }
}

// The three bf16 values of 8 ranks, the smallest last.
__device__ __forceinline__ void split8(float (&f)[8], u32x4 (&v)[kSplit]) {
#pragma unroll
  for (int h = 0; h < kSplit; ++h) {
    float g[8];
    v[h] = pack8(f);
    unpack8(v[h], g);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = lack(f[i], g[i]);
  }
}

// The four rows of a lane: what was read (`in`) and the products' sums -> what is written.  `left`: rows that there are.
template <int MODE, bool DROP, int NI, int NW>
__device__ __forceinline__ void expand_store(const ExpandArgs& a, const u32x4 (&in)[4][NI], const f32x4 (&acc)[NW][8],
                                             const int (&row)[4], int left, bool live, int col, float f, const DropKey& key) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= left || !live) continue;
    const long long at = static_cast<long long>(row[j]) * a.N + col;
    float x0[8], x1[8];
    unpack8(in[j][0], x0);
    if constexpr (MODE == kAdd) {
      float delta[8];
#pragma unroll
      for (int o = 0; o < 8; ++o) delta[o] = acc[0][o][j];
      if (DROP) drop_apply(key, row[j], col >> 3, 1.f, delta);
#pragma unroll
      for (int o = 0; o < 8; ++o) x0[o] = fmaf(f, delta[o], x0[o]);
      store16(a.out[0] + at, pack8(x0));
    } else if constexpr (MODE == kSwiglu) {
      float y[8];
      unpack8(in[j][1], x1);
#pragma unroll
      for (int o = 0; o < 8; ++o) {
        x0[o] = fmaf(f, acc[0][o][j], x0[o]);
        x1[o] = fmaf(f, acc[NW - 1][o][j], x1[o]);
        y[o] = x0[o] * logistic(x0[o]) * x1[o];
      }
      if (a.out[0] != nullptr) {
        store16(a.out[0] + at, pack8(x0));
        store16(a.out[1] + at, pack8(x1));
      }
      store16(a.out[2] + at, pack8(y));
    } else {
      float dg[8], du[8], delta[8];
      unpack8(in[j][1], x1);
      unpack8(in[j][2], dg);
      unpack8(in[j][3], du);
#pragma unroll
      for (int o = 0; o < 8; ++o) delta[o] = acc[0][o][j];
      if (DROP) drop_apply(key, row[j], col >> 3, 1.f, delta);
#pragma unroll
      for (int o = 0; o < 8; ++o) {
        const float s = logistic(x0[o]), da = f * delta[o];
        dg[o] = fmaf(da * x1[o], s * fmaf(x0[o], 1.f - s, 1.f), dg[o]);
        du[o] = fmaf(da, x0[o] * s, du[o]);
      }
      store16(a.out[0] + at, pack8(dg));
      store16(a.out[1] + at, pack8(du));
    }
  }
}

template <int KS, int MODE, bool DROP>
__global__ __launch_bounds__(256, KS == 1 || (KS == 2 && MODE != kSwiglu) ? 2 : 1) void adapter_expand_kernel(ExpandArgs a) {
  constexpr int NW = MODE == kSwiglu ? 2 : 1;
  constexpr int NOUT = MODE == kAdd ? 1 : MODE == kSwiglu ? 3 : 2;
  const PlanLayout p = plan_layout(a.rows.n, a.rows.E, a.rows.L);
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  const int stripes = (a.N + 127) / 128;
  const int each = stripes * a.parts, rows_each = kTileRows / a.parts;
  const long long items = static_cast<long long>(n_tiles(a.rows)) * each, step = gridDim.x * 4LL;
  DropKey key;
  if (DROP) key = drop_key(a.drop);
  for (long long i = blockIdx.x * 4LL + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); i < items; i += step) {
    Tile t = tile_at(a.rows, p, static_cast<int>(i / each));
    const int stripe = static_cast<int>(i % stripes), first = static_cast<int>(i % each / stripes) * rows_each;
    t.pos += first;
    t.count = min(t.count - first, rows_each);
    if (t.count <= 0) continue;
    const int col = 128 * stripe + 8 * c;
    const bool live = col < a.N;        // the last stripe may be half
    const int cc = live ? col : 0;
    if (t.l >= a.rows.L) {              // no adapter: copies
      if (a.v_out != nullptr && stripe == 0)
        for (int at = lane; at < t.count * a.ldv; at += 64)
          a.v_out[static_cast<long long>(row_at(a.rows, p, t.pos + at / a.ldv)) * a.ldv + at % a.ldv] = 0;
      for (int m = q; m < t.count; m += 4) {
        const long long at = static_cast<long long>(row_at(a.rows, p, t.pos + m)) * a.N + cc;
#pragma unroll
        for (int o = 0; o < NOUT; ++o)
          if (live && a.out[o] != nullptr)
            store16(a.out[o] + at, load16(a.in[MODE == kSwigluBwd ? o + 2 : o] + at));
      }
      continue;
    }
    // the first 16 rows' loads before the matrices', on whose arrival everything else waits
    constexpr int NI = MODE == kAdd ? 1 : MODE == kSwiglu ? 2 : 4;
    const int all = row_at(a.rows, p, t.pos + min(lane, t.count - 1));    // the tile's rows, one a lane
    u32x4 in[4][NI];
    auto load_rows = [&](int b) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long at = static_cast<long long>(__shfl(all, 16 * b + 4 * q + j, 64)) * a.N + cc;
#pragma unroll
        for (int o = 0; o < NI; ++o) in[j][o] = load16(a.in[o] + at);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    load_rows(0);
    u32x4 wf[NW][KS][8];
    const long long g = (static_cast<long long>(t.l) * a.rows.E + t.e) * a.R * a.N;
#pragma unroll
    for (int m = 0; m < NW; ++m) load_w<KS>(a.w[m] + g, a.R, a.N, cc, wf[m]);
    float f = a.scale != nullptr ? a.scale[t.l] : 1.f;
    if (DROP) f *= drop_scale(a.drop.drop);
    const int nb = (t.count + 15) / 16;
    for (int b = 0; b < nb; ++b) {
      if (b > 0) load_rows(b);
      const int mine = __shfl(all, 16 * b + c, 64);
      int row[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) row[j] = __shfl(all, 16 * b + 4 * q + j, 64);
      f32x4 acc[NW][8];
#pragma unroll
      for (int m = 0; m < NW; ++m) {
#pragma unroll
        for (int o = 0; o < 8; ++o) acc[m][o] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int rank = 32 * k + 8 * q;
          float x[8] = {};
          if (rank < a.R) {
            load_v(a, mine, m * a.R + rank, x);
            if (stripe == 0 && 16 * b + c < t.count) {
              const long long to = static_cast<long long>(mine) * a.ldv + m * a.R + rank;
              if (a.v_out != nullptr) store16(a.v_out + to, pack8(x));
              if (a.sum_out != nullptr) {
                *reinterpret_cast<f32x4*>(a.sum_out + to) = f32x4{x[0], x[1], x[2], x[3]};
                *reinterpret_cast<f32x4*>(a.sum_out + to + 4) = f32x4{x[4], x[5], x[6], x[7]};
              }
            }
          }
          u32x4 v[kSplit];
          split8(x, v);
#pragma unroll
          for (int h = kSplit - 1; h >= 0; --h)
#pragma unroll
            for (int o = 0; o < 8; ++o) acc[m][o] = mfma(v[h], wf[m][k][o], acc[m][o]);
        }
      }
      expand_store<MODE, DROP>(a, in, acc, row, t.count - 16 * b - 4 * q, live, col, f, key);
    }
  }
}

// ---------------------------------------------------------------- both products of a tile's rows

// A workgroup makes v of up to ROWS rows of a tile, which stays in LDS (as three bf16 values), and then what is added to them: its waves take
// K's units in turn, then the columns' stripes.  Where few tiles leave the chip idle, what shrink and expand cost is their two
// launches and the chain of loads in each (4012 rows of 16 experts and 5 adapters, d 2112, f 1344: 17 and 15 us against 8 + 14
// and 8 + 11).  Loading a wave's first stripe before v is made, so that it is there by then, took 37 us a call where this takes 35.
// Calls with dropout, which are training's and of more rows, keep to the two kernels.
constexpr int kBothWaves = 8;

// v = x A^T of a unit's rows, NB blocks of 16, into vs.  The waves' sums meet in LDS, each wave's in its own staging.
template <int NB, int RT, int ROWS>
__device__ __forceinline__ void both_shrink(const ShrinkArgs& s, const ExpandArgs& a, const Tile& t, const PlanLayout& p,
                                            const uint16_t* w, u32x4* lds, uint16_t (&vs)[kSplit][ROWS][16 * RT + 8]) {
  constexpr int kStage = (ROWS / 16 + RT) * 128;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  u32x4* stage = lds + wave * kStage;
  f32x4 acc[NB][RT];
  shrink_tile<NB, RT, false, kBothWaves>(s, t, p, s.x[0], w, wave, s.K / 64, stage, acc);
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < RT; ++r) reinterpret_cast<f32x4*>(stage)[64 * (b * RT + r) + lane] = acc[b][r];
  __syncthreads();
  for (int at = tid; at < 64 * NB * RT; at += 64 * kBothWaves) {
    f32x4 sum = reinterpret_cast<f32x4*>(lds)[at];
#pragma unroll
    for (int o = 1; o < kBothWaves; ++o) sum += reinterpret_cast<f32x4*>(lds + o * kStage)[at];
    const int rank = at / 64 % RT * 16 + (at & 15), m = at / (64 * RT) * 16 + 4 * (at >> 4 & 3);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x = rank < s.R ? sum[j] : 0.f;
#pragma unroll
      for (int h = 0; h < kSplit; ++h) {
        const uint16_t here = f32_to_bf16(x);
        vs[h][m + j][rank] = here;
        x = lack(x, bf16_to_f32(here));
      }
      if (a.v_out != nullptr && rank < s.R && m + j < t.count)
        a.v_out[static_cast<long long>(row_at(a.rows, p, t.pos + m + j)) * a.ldv + rank] = vs[0][m + j][rank];
    }
  }
  __syncthreads();
}

template <int RT, int MODE, int ROWS>
__global__ __launch_bounds__(64 * kBothWaves) void adapter_both_kernel(ShrinkArgs s, ExpandArgs a) {
  constexpr int NW = MODE == kSwiglu ? 2 : 1, NOUT = MODE == kSwiglu ? 3 : 1, KS = (16 * RT / NW + 31) / 32, NI = NW;
  __shared__ u32x4 lds[kBothWaves * (ROWS / 16 + RT) * 128];
  __shared__ alignas(16) uint16_t vs[kSplit][ROWS][16 * RT + 8];     // (rows in different banks)
  const PlanLayout p = plan_layout(a.rows.n, a.rows.E, a.rows.L);
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int stripes = (a.N + 127) / 128;
  constexpr int kParts = kTileRows / ROWS;
  const long long items = static_cast<long long>(n_tiles(a.rows)) * kParts;
  for (long long i = blockIdx.x; i < items; i += gridDim.x) {
    Tile t = tile_at(a.rows, p, static_cast<int>(i / kParts));
    const int first = static_cast<int>(i % kParts) * ROWS;
    t.pos += first;
    t.count = min(t.count - first, ROWS);
    if (t.count <= 0) continue;
    if (t.l >= a.rows.L) {              // no adapter: copies
      const int chunks = a.N / 8;
      for (int at = tid; at < t.count * chunks; at += 64 * kBothWaves) {
        const long long to = static_cast<long long>(row_at(a.rows, p, t.pos + at / chunks)) * a.N + at % chunks * 8;
#pragma unroll
        for (int o = 0; o < NOUT; ++o)
          if (a.out[o] != nullptr) store16(a.out[o] + to, load16(a.in[o] + to));
      }
      if (a.v_out != nullptr)
        for (int at = tid; at < t.count * a.ldv; at += 64 * kBothWaves)
          a.v_out[static_cast<long long>(row_at(a.rows, p, t.pos + at / a.ldv)) * a.ldv + at % a.ldv] = 0;
      continue;
    }
    const long long group = static_cast<long long>(t.l) * a.rows.E + t.e;
    const int nb = (t.count + 15) / 16, all = row_at(a.rows, p, t.pos + min(lane, t.count - 1));
    const uint16_t* w = s.w[0] + group * s.R * s.K;
    if (ROWS == 16 || nb == 1) both_shrink<1, RT, ROWS>(s, a, t, p, w, lds, vs);
    else if (ROWS == 32 || nb == 2) both_shrink<2, RT, ROWS>(s, a, t, p, w, lds, vs);
    else both_shrink<ROWS / 16, RT, ROWS>(s, a, t, p, w, lds, vs);
    const float f = a.scale[t.l];
    for (int stripe = wave; stripe < stripes; stripe += kBothWaves) {
      const int col = 128 * stripe + 8 * c;
      const bool live = col < a.N;        // the last stripe may be half
      const int cc = live ? col : 0;
      u32x4 in[4][NI], wf[NW][KS][8];
      int row[4];
      auto load_rows = [&](int b) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          row[j] = __shfl(all, 16 * b + 4 * q + j, 64);
#pragma unroll
          for (int o = 0; o < NI; ++o) in[j][o] = load16(a.in[o] + static_cast<long long>(row[j]) * a.N + cc);
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      load_rows(0);
#pragma unroll
      for (int m = 0; m < NW; ++m) load_w<KS>(a.w[m] + group * a.R * a.N, a.R, a.N, cc, wf[m]);
      for (int b = 0; b < nb; ++b) {
        if (b > 0) load_rows(b);
        f32x4 acc[NW][8];
#pragma unroll
        for (int m = 0; m < NW; ++m) {
#pragma unroll
          for (int o = 0; o < 8; ++o) acc[m][o] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int rank = 32 * k + 8 * q;
#pragma unroll
            for (int h = kSplit - 1; h >= 0; --h) {
              const u32x4 v = rank < a.R ? *reinterpret_cast<const u32x4*>(&vs[h][16 * b + c][m * a.R + rank]) : u32x4{0, 0, 0, 0};
#pragma unroll
              for (int o = 0; o < 8; ++o) acc[m][o] = mfma(v, wf[m][k][o], acc[m][o]);
            }
          }
        }
        expand_store<MODE, false>(a, in, acc, row, t.count - 16 * b - 4 * q, live, col, f, DropKey{});
      }
    }
  }
}

// ---------------------------------------------------------------- few rows

// Both products of one row in a workgroup, without a plan: what few rows cost is the chain of loads that hang on each
// other (token, adapter, matrices) and the launches, not bytes.  One token's 8 rows (d 4096, f 768, rank 16) take 10 us and
// 6 us (down), and a whole call 11 us of the host's time; as shrink and expand they took 14, 10 and 18 us.  A wave takes RW
// ranks of A along whole cache lines, v meets in LDS as fp32, and then a lane takes 8 columns of B for all ranks; the first
// 8 ranks of B, and the row's own values, are on their way while A is read.  Products and sums are fp32 FMAs.
struct RowArgs {
  Rows rows;
  const uint16_t* x;
  int gather, K, R;         // R: rows of A
  const uint16_t* a;
  int N, r;                 // r: ranks of one product
  const uint16_t* b[2];     // kSwiglu: gate and up
  const float* scale;
  const uint16_t* in[3];    // kAdd: y; kSwiglu: g, u, a
  uint16_t* out[3];
  uint16_t* v_out;          // [n][R] or null
  DropArgs drop;
};

constexpr int kRowThreads = 512;

template <int RW, int MODE, bool DROP>
__global__ __launch_bounds__(kRowThreads) void adapter_row_kernel(RowArgs a) {
  constexpr int NW = MODE == kSwiglu ? 2 : 1, NOUT = MODE == kSwiglu ? 3 : 1;
  __shared__ float v[2 * kMaxRank];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i = blockIdx.x;
  // the row's token first: its adapter's number hangs on it
  const int l = __builtin_amdgcn_readfirstlane(adapter_of(a.rows.ids, a.rows.row_token, i, a.rows.T, a.rows.L));
  // its expert: the first one whose rows end behind it (of offsets that fall too, what their running maximum says, as in a plan)
  int end[4], e = a.rows.E;
#pragma unroll
  for (int b = 0; b < 4; ++b) end[b] = a.rows.offsets[min(64 * b + lane, a.rows.E - 1) + 1];
#pragma unroll
  for (int b = 3; b >= 0; --b) {
    const unsigned long long behind = __ballot(64 * b + lane < a.rows.E && end[b] > i);
    if (behind) e = 64 * b + __builtin_ctzll(behind);
  }
  if (e >= a.rows.E || i < a.rows.offsets[0]) return;      // behind the last expert's rows, or before the first's
  const long long row = static_cast<long long>(i) * a.N;
  const int chunks = a.N / 8;
  if (l >= a.rows.L) {                                     // no adapter: copies
    for (int c = tid; c < chunks; c += kRowThreads)
#pragma unroll
      for (int o = 0; o < NOUT; ++o)
        if (a.out[o] != nullptr) store16(a.out[o] + row + 8 * c, load16(a.in[o] + row + 8 * c));
    if (a.v_out != nullptr && tid < a.R) a.v_out[static_cast<long long>(i) * a.R + tid] = 0;
    return;
  }
  const long long g = static_cast<long long>(l) * a.rows.E + e;
  const int mine = min(tid, chunks - 1);
  u32x4 in[NW], bf[NW][8];
#pragma unroll
  for (int m = 0; m < NW; ++m) {
    in[m] = load16(a.in[m] + row + 8 * mine);
#pragma unroll
    for (int k = 0; k < 8; ++k) bf[m][k] = load16(a.b[m] + (g * a.r + k) * a.N + 8 * mine);
  }
  __builtin_amdgcn_sched_barrier(0);
  {
    const int src = a.gather ? token_of(a.rows.row_token, i, a.rows.T) : i;
    const uint16_t* x = a.x + static_cast<long long>(src) * a.K;
    const uint16_t* w[RW];
    float sum[RW];
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      w[k] = a.a + (g * a.R + min(wave * RW + k, a.R - 1)) * a.K;
      sum[k] = 0.f;
    }
    DropKey key;
    if (DROP) key = drop_key(a.drop);
    constexpr int U = RW <= 2 ? 4 : RW <= 4 ? 2 : 1;       // chunks of the row at a time
    for (int c0 = lane; c0 < a.K / 8; c0 += 64 * U) {
      u32x4 xf[U], wf[U][RW];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = min(c0 + 64 * u, a.K / 8 - 1);
        xf[u] = load16(x + 8 * c);
#pragma unroll
        for (int k = 0; k < RW; ++k) wf[u][k] = load16(w[k] + 8 * c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c0 + 64 * u >= a.K / 8) break;
        if (DROP) xf[u] = drop_zero(key, i, c0 + 64 * u, xf[u]);
        float xs[8];
        unpack8(xf[u], xs);
#pragma unroll
        for (int k = 0; k < RW; ++k) {
          float ws[8];
          unpack8(wf[u][k], ws);
#pragma unroll
          for (int o = 0; o < 8; ++o) sum[k] = fmaf(xs[o], ws[o], sum[k]);
        }
      }
    }
    const float f = DROP ? drop_scale(a.drop.drop) : 1.f;
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      const float t = wave_sum(sum[k]);
      if (lane == 0 && wave * RW + k < a.R) v[wave * RW + k] = f * t;
    }
  }
  __syncthreads();
  if (a.v_out != nullptr && tid < a.R) a.v_out[static_cast<long long>(i) * a.R + tid] = f32_to_bf16(v[tid]);
  const float s = a.scale[l];
  for (int c = tid; c < chunks; c += kRowThreads) {
    if (c != tid) {
#pragma unroll
      for (int m = 0; m < NW; ++m) {
        in[m] = load16(a.in[m] + row + 8 * c);
#pragma unroll
        for (int k = 0; k < 8; ++k) bf[m][k] = load16(a.b[m] + (g * a.r + k) * a.N + 8 * c);
      }
    }
    float acc[NW][8];
#pragma unroll
    for (int m = 0; m < NW; ++m)
#pragma unroll
      for (int o = 0; o < 8; ++o) acc[m][o] = 0.f;
    for (int k0 = 0; k0 < a.r; k0 += 8) {
      u32x4 cur[NW][8];
#pragma unroll
      for (int m = 0; m < NW; ++m)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          cur[m][k] = bf[m][k];
          if (k0 + 8 < a.r) bf[m][k] = load16(a.b[m] + (g * a.r + k0 + 8 + k) * a.N + 8 * c);
        }
#pragma unroll
      for (int m = 0; m < NW; ++m)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float ws[8];
          unpack8(cur[m][k], ws);
          const float vk = v[m * a.r + k0 + k];
#pragma unroll
          for (int o = 0; o < 8; ++o) acc[m][o] = fmaf(vk, ws[o], acc[m][o]);
        }
    }
    float x0[8];
    unpack8(in[0], x0);
    if constexpr (MODE == kAdd) {
#pragma unroll
      for (int o = 0; o < 8; ++o) x0[o] = fmaf(s, acc[0][o], x0[o]);
      store16(a.out[0] + row + 8 * c, pack8(x0));
    } else {
      float x1[8], y[8];
      unpack8(in[NW - 1], x1);
#pragma unroll
      for (int o = 0; o < 8; ++o) {
        x0[o] = fmaf(s, acc[0][o], x0[o]);
        x1[o] = fmaf(s, acc[NW - 1][o], x1[o]);
        y[o] = x0[o] * logistic(x0[o]) * x1[o];
      }
      if (a.out[0] != nullptr) {
        store16(a.out[0] + row + 8 * c, pack8(x0));
        store16(a.out[1] + row + 8 * c, pack8(x1));
      }
      store16(a.out[2] + row + 8 * c, pack8(y));
    }
  }
}

// ---------------------------------------------------------------- wgrad

struct WgradArgs {
  Rows rows;
  const uint16_t* v;        // [n][ldv]
  const float* vf;          // F32: the same in fp32 instead
  int v0[2];                // first columns of up to two products (blockIdx.y): gate and up
  const uint16_t* y[2];
  int gather;               // y by token
  int ldv, R, C;
  const float* scale;       // null, or [L]
  uint16_t* out[2];         // [L][E][R][C]
  float* part;              // [2 products][2 (n / piece + 1)][R][C]: sums of pieces of groups that have several
  DropArgs drop;
};

// Slot of a piece that starts at `pos`: pieces of one group start `piece` apart, and a group's first one never lies in the same
// `piece` positions as another group's first, nor a later one as another's later one (groups of several
// pieces are longer than that), so a bit for the first keeps all apart.
__device__ __forceinline__ long long piece_slot(int pos, int piece, bool first) { return 2LL * (pos / piece) + first; }

// RT tiles of 16 ranks (from rank r0) x 128 columns a wave over the rows of one piece, 64 rows a step.  The workgroup's waves take
// neighbouring columns of the same rows, so v's 64 rows are staged once for all of them, transposed: pairs of rows [rank][32] in
// LDS (padded to 36: the 16 ranks of a fragment's 16-byte reads lie in different banks).  y's rows go from memory into
// registers half a step (32 rows) ahead, v's and the row numbers a whole one; loads past the piece read its last row.
//
// Bound by memory and its latency: 131072 rows of 4096 by 32 ranks take 243 us (1.28 GB through the L2s' misses, 5.3 TB/s).
// More than 32 ranks are a workgroup for each 32, whose second reading of y comes from the L2: 64 ranks of fp32 take 338 us.  With v in two
// bf16 values they took 320, where a wave with all 64 (one wave per SIMD then) took 412, and a workgroup of eight waves, four for each half, 441.
template <int RT, bool DROP, bool F32>
__global__ __launch_bounds__(256, 2) void adapter_wgrad_kernel(WgradArgs a) {
  // a thread stages a pair of rows and VR ranks: 16 bytes of each row
  constexpr int NV = F32 ? kSplit : 1, VR = F32 ? 4 : 8, kItems = 32 * 16 * RT / VR, kPad = 36;
  static_assert(kItems <= 256);
  __shared__ uint32_t vt[2][NV][16 * RT][kPad];
  // row and row of y, of steps s (read until its last product) and s + 1 while those of s + 2 come
  __shared__ int ids[4][2][64];
  const PlanLayout p = plan_layout(a.rows.n, a.rows.E, a.rows.L);
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int stripes = (a.C + 127) / 128, groups = (stripes + 3) / 4, per = (stripes + groups - 1) / groups;
  const int parts = (a.R + 16 * RT - 1) / (16 * RT), which = blockIdx.y;
  const int piece = piece_rows(a.rows.n);
  const long long items = static_cast<long long>(a.rows.plan[kHeadItems]) * parts * groups;
  const uint16_t* y = a.y[which];
  DropKey key;
  if (DROP) key = drop_key(a.drop);
  for (long long i = blockIdx.x; i < items; i += gridDim.x) {
    const Tile t = reinterpret_cast<const Tile*>(a.rows.plan + p.items)[i / (parts * groups)];
    const int stripe = static_cast<int>(i % groups) * per + wave, r0 = static_cast<int>(i / groups % parts) * 16 * RT;
    const bool busy = wave < per && stripe < stripes;
    const int col = 128 * stripe + 8 * c, cc = busy && col < a.C ? col : 0;
    const int32_t* list = a.rows.plan + p.rows + t.pos;
    const int32_t* srcs = a.gather ? a.rows.plan + p.toks + t.pos : list;
    f32x4 acc[RT][8];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int o = 0; o < 8; ++o) acc[m][o] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (t.count > 0) {
      auto row_of = [&](int at) { return list[min(at, t.count - 1)]; };
      auto src_of = [&](int at) { return srcs[min(at, t.count - 1)]; };
      const int pair = tid & 31, vrank = r0 + VR * ((tid >> 5) % (16 * RT / VR)), vcol = a.v0[which] + (vrank < a.R ? vrank : 0);
      u32x4 vr[2];
      auto load_v = [&](int s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const long long at = static_cast<long long>(ids[s & 3][0][2 * pair + h]) * a.ldv + vcol;
          vr[h] = F32 ? *reinterpret_cast<const u32x4*>(a.vf + at) : load16(a.v + at);
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      auto put_v = [&](int buf, int left) {
        if (tid >= kItems) return;
        const uint32_t m0 = 2 * pair < left ? ~0u : 0u, m1 = 2 * pair + 1 < left ? ~0u : 0u;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint32_t lo = vr[0][h] & m0, hi = vr[1][h] & m1;
          if constexpr (F32) {
            float x = __builtin_bit_cast(float, lo), y = __builtin_bit_cast(float, hi);
#pragma unroll
            for (int n = 0; n < NV; ++n) {
              const uint32_t both = pack_bf16x2(x, y);
              vt[buf][n][vrank - r0 + h][pair] = both;
              x = lack(x, bf16_lo(both));
              y = lack(y, bf16_hi(both));
            }
          } else {
            vt[buf][0][vrank - r0 + 2 * h][pair] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
            vt[buf][0][vrank - r0 + 2 * h + 1][pair] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
          }
        }
      };
      auto load_y = [&](u32x4 (&yr)[8], int s, int sub) {
#pragma unroll
        for (int j = 0; j < 8; ++j) yr[j] = load16(y + static_cast<long long>(ids[s & 3][1][32 * sub + 8 * q + j]) * a.C + cc);
        __builtin_amdgcn_sched_barrier(0);
      };
      auto multiply = [&](u32x4 (&yr)[8], int s, int sub, int left) {
        const int buf = s & 1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = 32 * sub + 8 * q + j;
          if (DROP) yr[j] = drop_zero(key, ids[s & 3][0][at], cc >> 3, yr[j]);
          const uint32_t keep = at < left ? ~0u : 0u;
          yr[j] &= u32x4{keep, keep, keep, keep};
        }
        u32x4 yf[8];
        transpose8(yr, yf);
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int n = NV - 1; n >= 0; --n) {
            const u32x4 vf = *reinterpret_cast<const u32x4*>(&vt[buf][n][16 * m + c][16 * sub + 4 * q]);
#pragma unroll
            for (int o = 0; o < 8; ++o) acc[m][o] = mfma(vf, yf[o], acc[m][o]);
          }
        __builtin_amdgcn_sched_barrier(0);
      };
      __syncthreads();                   // the last item's reads are over
      if (tid < 64) {
        ids[0][0][tid] = row_of(tid);
        ids[0][1][tid] = src_of(tid);
      }
      int next = row_of(64 + lane), next_src = src_of(64 + lane);
      __syncthreads();
      u32x4 ya[8], yb[8];
      load_v(0);
      load_y(ya, 0, 0);
      const int steps = (t.count + 63) / 64;
      for (int s = 0; s < steps; ++s) {
        const int left = t.count - 64 * s;
        put_v(s & 1, left);
        if (tid < 64) {
          ids[(s + 1) & 3][0][tid] = next;
          ids[(s + 1) & 3][1][tid] = next_src;
        }
        __syncthreads();
        next = row_of(64 * (s + 2) + lane);
        next_src = src_of(64 * (s + 2) + lane);
        load_v(s + 1);
        load_y(yb, s, 1);
        multiply(ya, s, 0, left);
        load_y(ya, s + 1, 0);
        multiply(yb, s, 1, left);
      }
    }
    if (!busy) continue;
    float f = a.scale != nullptr ? a.scale[t.l] : 1.f;
    if (DROP) f *= drop_scale(a.drop.drop);
    const int32_t* goff = a.rows.plan + p.goff + t.e * (a.rows.L + 1) + t.l;
    const bool several = goff[1] - goff[0] > piece;
    uint16_t* out = a.out[which] + (static_cast<long long>(t.l) * a.rows.E + t.e) * a.R * a.C;
    float* part = a.part + ((which * 2LL * (a.rows.n / piece + 1)) + piece_slot(t.pos, piece, t.pos == goff[0])) * a.R * a.C;
#pragma unroll
    for (int m = 0; m < RT; ++m) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int rank = r0 + 16 * m + 4 * q + j;      // accumulator row 4 q + j of tile m
        if (rank >= a.R || col >= a.C) continue;
        const long long at = static_cast<long long>(rank) * a.C + col;
        float x[8];
#pragma unroll
        for (int o = 0; o < 8; ++o) x[o] = f * acc[m][o][j];
        if (several) {
          *reinterpret_cast<float4*>(part + at) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4*>(part + at + 4) = make_float4(x[4], x[5], x[6], x[7]);
        } else {
          store16(out + at, pack8(x));
        }
      }
    }
  }
}

// Groups of several pieces: their sums in the order of the pieces.  gridDim.x workgroups to a group, blockIdx.z one of up to
// three products.
struct JoinArgs {
  Rows rows;
  const float* part[3];
  uint16_t* out[3];
  int R[3], C[3];
};

__global__ __launch_bounds__(256) void adapter_join_kernel(JoinArgs a) {
  if (static_cast<int>(blockIdx.y) >= a.rows.plan[kHeadMulti]) return;
  const PlanLayout p = plan_layout(a.rows.n, a.rows.E, a.rows.L);
  const int which = blockIdx.z, piece = piece_rows(a.rows.n);
  const int pair = a.rows.plan[p.multi + blockIdx.y], e = pair / (a.rows.L + 1), l = pair - e * (a.rows.L + 1);
  const int begin = a.rows.plan[p.goff + pair], end = a.rows.plan[p.goff + pair + 1];
  const long long size = static_cast<long long>(a.R[which]) * a.C[which];
  const float* part = a.part[which];
  uint16_t* out = a.out[which] + (static_cast<long long>(l) * a.rows.E + e) * size;
  for (long long i = (blockIdx.x * 256LL + threadIdx.x) * 8; i < size; i += gridDim.x * 2048LL) {
    float x[8];
#pragma unroll
    for (int o = 0; o < 8; ++o) x[o] = 0.f;
    for (int pos = begin; pos < end; pos += piece) {
      const float4* at = reinterpret_cast<const float4*>(part + piece_slot(pos, piece, pos == begin) * size + i);
      const float4 lo = at[0], hi = at[1];
      x[0] += lo.x; x[1] += lo.y; x[2] += lo.z; x[3] += lo.w;
      x[4] += hi.x; x[5] += hi.y; x[6] += hi.z; x[7] += hi.w;
    }
    store16(out + i, pack8(x));
  }
}

// ---------------------------------------------------------------- host side

constexpr int kGridCap = 8192;   // workgroups of a launch; more tiles are taken in turn

int tiles_cap(const Rows& r) { return plan_layout(r.n, r.E, r.L).tiles_cap; }

// Tiles that a call is likely to have (their number is on the device): those of whole tiles, and one more for half of the
// experts' adapters that can have rows.  Of many adapters loaded and few in use it is too high, and such calls are cut into fewer pieces
// than the chip could take: 4096 rows of 64 experts and 256 adapters count 2112, also where one adapter has them all and there are about 64.
long long likely_tiles(int n, int E, int L) {
  const long long groups = static_cast<long long>(E) * L;
  return n / kTileRows + ((groups < n ? groups : n) + 1) / 2;
}

// Pieces of 16 rows or more that a tile is cut into, to have `want` of them where there are few tiles.
int row_parts(int n, long long tiles, long long want) {
  const long long rows = n / tiles;
  return tiles >= want || rows < 32 ? 1 : 2 * tiles >= want || rows < 64 ? 2 : 4;
}

// How the shrink's work is cut beyond tiles, to have workgroups enough for the chip: rows first (the matrices are read
// again, from the second-level cache), then K into slices, each with a unit for every wave.  Two products in a launch are twice
// the workgroups (32768 rows of 64 experts, dG and dU of 1024: 31 us in whole tiles, 36 in halves).
int shrink_parts(int n, int E, int L, int products) { return row_parts(n, likely_tiles(n, E, L), 1024 / products); }
int slices(int n, int E, int L, int K) {
  const int most = (K / 64 + 3) / 4;
  const long long want = 512 / (likely_tiles(n, E, L) * shrink_parts(n, E, L, 1));
  const int s = want < 1 ? 1 : want > 8 ? 8 : static_cast<int>(want);
  return s > most ? most : s;
}

unsigned grid_of(long long workgroups) {
  return static_cast<unsigned>(workgroups < kGridCap ? (workgroups + 7) / 8 * 8 : kGridCap);
}

template <bool DROP>
void launch_shrink(ShrinkArgs a, int products, hipStream_t st) {
  a.parts = shrink_parts(a.rows.n, a.rows.E, a.rows.L, products);
  const dim3 grid(grid_of(static_cast<long long>(tiles_cap(a.rows)) * a.S * a.parts), products);
  if (a.R <= 16) adapter_shrink_kernel<1, DROP><<<grid, 256, 0, st>>>(a);
  else if (a.R <= 32) adapter_shrink_kernel<2, DROP><<<grid, 256, 0, st>>>(a);
  else if (a.R <= 64) adapter_shrink_kernel<4, DROP><<<grid, 256, 0, st>>>(a);
  else adapter_shrink_kernel<8, DROP><<<grid, 256, 0, st>>>(a);
}

template <int MODE, bool DROP>
void launch_expand(ExpandArgs a, hipStream_t st) {
  const long long stripes = (a.N + 127) / 128, waves = tiles_cap(a.rows) * stripes;
  // A wave walks its rows 16 at a time, each time waiting for memory: where a launch has few waves they take fewer rows.
  a.parts = row_parts(a.rows.n, likely_tiles(a.rows.n, a.rows.E, a.rows.L), (4096 + stripes - 1) / stripes);
  const unsigned grid = grid_of((waves * a.parts + 3) / 4);
  if (a.R <= 32) adapter_expand_kernel<1, MODE, DROP><<<grid, 256, 0, st>>>(a);
  else if (a.R <= 64) adapter_expand_kernel<2, MODE, DROP><<<grid, 256, 0, st>>>(a);
  else if constexpr (MODE == kAdd) adapter_expand_kernel<4, MODE, DROP><<<grid, 256, 0, st>>>(a);
}

// Rows of a workgroup's unit where one kernel makes v and what is added (adapter_both_kernel), 0 where two kernels do.  It
// pays where the units fit the chip at once, a workgroup to a compute unit, parts of tiles without rows included; units are as small as
// that allows.  Past that, only where tiles have few rows: there its matrices are its time, and two kernels wait for them
// twice.  Gate/up, down and the plan, two kernels -> one, us: 16 experts x 5 adapters of 8 ranks (d 2112, f 1344), 1024 rows 50 ->
// 32 (with 32 or 64 rows 37 and 41), 4096 52 -> 46 (16 rows 53, 64 rows 61), 8192 71 -> 69, 16384 113 -> 141; 64 x 8 of 16 (d 2048, f
// 1024), 4096 rows 73 -> 66, 16384 143 -> 128, 65536 (46 rows a tile) 325 -> 336; 64 x 32 of 32, 1024 rows 121 -> 109, 16384 283 ->
// 270, 65536 478 -> 475; 128 x 16 of 32 (d 4096, f 768), 1024 rows 126 -> 117, 16384 (exactly at the limit of 1280, on the wrong side by two
// percent) 330 -> 336, 65536 612 -> 636.
int both_rows(const Rows& r, int R) {
  if (R > 64) return 0;
  const long long tiles = likely_tiles(r.n, r.E, r.L), rows = r.n / tiles, groups = tiles - r.n / kTileRows;
  if (rows > 8 && 4 * tiles <= 288 && r.n / 16 + groups <= 256) return 16;
  if (rows > 32 && 2 * tiles <= 288 && r.n / 32 + groups <= 256) return 32;
  return tiles <= 256 || (rows <= 32 && tiles <= 1280) ? 64 : 0;
}

template <int MODE, int ROWS>
void launch_both_of(const ShrinkArgs& s, const ExpandArgs& e, hipStream_t st) {
  const unsigned grid = grid_of(static_cast<long long>(kTileRows / ROWS) * tiles_cap(e.rows));
  if (s.R <= 16) adapter_both_kernel<1, MODE, ROWS><<<grid, 64 * kBothWaves, 0, st>>>(s, e);
  else if (s.R <= 32) adapter_both_kernel<2, MODE, ROWS><<<grid, 64 * kBothWaves, 0, st>>>(s, e);
  else adapter_both_kernel<4, MODE, ROWS><<<grid, 64 * kBothWaves, 0, st>>>(s, e);
}
template <int MODE>
void launch_both(int rows, const ShrinkArgs& s, const ExpandArgs& e, hipStream_t st) {
  if (rows == 16) launch_both_of<MODE, 16>(s, e, st);
  else if (rows == 32) launch_both_of<MODE, 32>(s, e, st);
  else launch_both_of<MODE, 64>(s, e, st);
}

template <int MODE, bool DROP>
void launch_rows(const RowArgs& a, hipStream_t st) {
  constexpr int W = kRowThreads / 64;       // (8: gate/up has 16 ranks at the least, down 64 at the most)
  if constexpr (MODE == kAdd) {
    if (a.R <= W) return adapter_row_kernel<1, MODE, DROP><<<a.rows.n, kRowThreads, 0, st>>>(a);
  }
  if (a.R <= 2 * W) adapter_row_kernel<2, MODE, DROP><<<a.rows.n, kRowThreads, 0, st>>>(a);
  else if (a.R <= 4 * W) adapter_row_kernel<4, MODE, DROP><<<a.rows.n, kRowThreads, 0, st>>>(a);
  else if (a.R <= 8 * W) adapter_row_kernel<8, MODE, DROP><<<a.rows.n, kRowThreads, 0, st>>>(a);
  else if constexpr (MODE == kSwiglu) adapter_row_kernel<16, MODE, DROP><<<a.rows.n, kRowThreads, 0, st>>>(a);
}

template <bool DROP, bool F32>
void launch_wgrad(const WgradArgs& a, int products, hipStream_t st) {
  const PlanLayout p = plan_layout(a.rows.n, a.rows.E, a.rows.L);
  const int rt = a.R <= 16 ? 1 : 2;
  const int stripes = (a.C + 127) / 128;
  const long long wgs = static_cast<long long>(p.items_cap) * ((a.R + 16 * rt - 1) / (16 * rt)) * ((stripes + 3) / 4);
  const dim3 grid(grid_of(wgs), products);
  if (rt == 1) adapter_wgrad_kernel<1, DROP, F32><<<grid, 256, 0, st>>>(a);
  else adapter_wgrad_kernel<2, DROP, F32><<<grid, 256, 0, st>>>(a);
}

// Joins the pieces of up to three products in one launch, where there can be groups of several.
void launch_join(const JoinArgs& a, int products, hipStream_t st) {
  const int piece = piece_rows(a.rows.n);
  if (a.rows.n <= piece) return;
  long long blocks = 0;
  for (int i = 0; i < products; ++i) blocks = max(blocks, (static_cast<long long>(a.R[i]) * a.C[i] + 2047) / 2048);
  adapter_join_kernel<<<dim3(static_cast<unsigned>(blocks < 64 ? blocks : 64), a.rows.n / piece + 1, products), 256, 0, st>>>(a);
}

int check_sizes(int T, int n, int E, int L) {
  MOE_REQUIRE(T >= 1 && n >= 1, MOE_ERR_UNSUPPORTED, "T and n must be >= 1 (got %d, %d)", T, n);
  MOE_REQUIRE(E >= 1 && E <= 256, MOE_ERR_UNSUPPORTED, "E must be in [1, 256] (got %d)", E);
  MOE_REQUIRE(L >= 1 && L <= kMaxAdapters, MOE_ERR_UNSUPPORTED, "adapters must be 1 to %d in number (got %d)", kMaxAdapters, L);
  MOE_REQUIRE(n <= 1 << 26, MOE_ERR_UNSUPPORTED, "n must be at most 2^26 (got %d)", n);
  return MOE_OK;
}

int check_rows(const Rows& r) {
  if (int st = check_sizes(r.T, r.n, r.E, r.L)) return st;
  MOE_CHECK_PTR(r.ids); MOE_CHECK_PTR(r.offsets);
  MOE_REQUIRE(r.row_token != nullptr || r.T == r.n, MOE_ERR_INVALID_ARG, "without row_token n = %d must be T = %d", r.n, r.T);
  if (r.plan) MOE_CHECK_ALIGN(r.plan);
  return MOE_OK;
}

// Without a plan every row is a workgroup.
int check_few(const Rows& r) {
  MOE_REQUIRE(r.plan != nullptr || r.n <= 1 << 22, MOE_ERR_UNSUPPORTED, "more than 2^22 rows need a plan (got %d)", r.n);
  return MOE_OK;
}

int check_dims(int d, int f, int r) {
  // (a matrix of 128 ranks is addressed by 32 bits)
  MOE_REQUIRE(d >= 64 && d % 64 == 0 && d <= 1 << 24, MOE_ERR_UNSUPPORTED, "d must be a multiple of 64 in [64, 2^24] (got %d)", d);
  MOE_REQUIRE(f >= 64 && f % 64 == 0 && f <= 1 << 24, MOE_ERR_UNSUPPORTED, "f must be a multiple of 64 in [64, 2^24] (got %d)", f);
  MOE_REQUIRE(r >= 8 && r <= kMaxRank && r % 8 == 0, MOE_ERR_UNSUPPORTED, "r must be a multiple of 8 in [8, %d] (got %d)",
              kMaxRank, r);
  return MOE_OK;
}

long long align256(long long b) { return (b + 255) / 256 * 256; }

// Bytes of v's slices (fp32 [S][n][R]) and of the weight gradients' pieces for a product pair of widths K -> R.
long long part_bytes(int n, int E, int L, int R, int K) { return align256(4LL * slices(n, E, L, K) * n * R); }
long long piece_bytes(int n, int products, int R, int C) {
  const int piece = piece_rows(n);
  return n > piece ? align256(4LL * products * 2 * (n / piece + 1) * R * C) : 0;
}

// The workspace of a backward call: v's slices, their sum [n][R] (the slice itself where there is one), the pieces of the B's
// gradients (1 or 2 products of C1 columns and r ranks) and of A's (R ranks, C2 columns).
struct BwdSpace {
  long long part, sum, pieces_b, pieces_a, bytes;
};
BwdSpace bwd_space(int n, int E, int L, int r, int products, int C1, int R, int C2) {
  const bool sliced = slices(n, E, L, C1) > 1;
  BwdSpace w;
  w.part = 0;
  w.sum = sliced ? part_bytes(n, E, L, R, C1) : 0;
  w.pieces_b = w.sum + align256(4LL * n * R);
  w.pieces_a = w.pieces_b + piece_bytes(n, products, r, C1);
  w.bytes = w.pieces_a + piece_bytes(n, 1, R, C2);
  return w;
}
BwdSpace down_bwd_space(int n, int E, int L, int d, int f, int r) { return bwd_space(n, E, L, r, 1, d, r, f); }
BwdSpace gate_up_bwd_space(int n, int E, int L, int d, int f, int r) { return bwd_space(n, E, L, r, 2, f, 2 * r, d); }

#define MOE_CHECK_WS(need)                                                                                     \
  do {                                                                                                         \
    MOE_REQUIRE(ws != nullptr && ws_bytes >= static_cast<size_t>(need), MOE_ERR_WORKSPACE,                     \
                "workspace of %lld bytes needed", static_cast<long long>(need));                               \
    MOE_CHECK_ALIGN(ws);                                                                                       \
  } while (0)

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_adapter_plan_bytes(int n, int E, int L) {
  if (check_sizes(1, n, E, L)) return 0;
  return static_cast<size_t>(plan_layout(n, E, L).words) * 4;
}

extern "C" int moe_adapter_plan(const int32_t* ids, const int32_t* row_token, const int32_t* offsets, int T, int n,
                                int E, int L, void* plan, size_t plan_bytes, void* stream) {
  const Rows rows = {nullptr, ids, row_token, offsets, T, n, E, L};
  if (int st = check_rows(rows)) return st;
  const PlanLayout p = plan_layout(n, E, L);
  MOE_REQUIRE(plan != nullptr && plan_bytes >= static_cast<size_t>(p.words) * 4, MOE_ERR_WORKSPACE,
              "plan buffer of %lld bytes needed", p.words * 4);
  MOE_CHECK_ALIGN(plan);
  hipStream_t st = as_stream(stream);
  int32_t* buf = static_cast<int32_t*>(plan);
  if (n <= kSmallPlan) {
    plan_small_kernel<<<1, 1024, 0, st>>>(ids, row_token, offsets, T, n, E, L, buf);
    return check_launch("adapter_plan");
  }
  plan_count_kernel<<<p.chunks, 256, 0, st>>>(ids, row_token, offsets, T, n, E, L, buf);
  plan_scan_kernel<<<1, 1024, 0, st>>>(offsets, n, E, L, buf);
  plan_place_kernel<<<p.chunks, 256, 0, st>>>(ids, row_token, offsets, T, n, E, L, buf);
  return check_launch("adapter_plan");
}

extern "C" size_t moe_adapter_workspace_bytes(int n, int E, int L, int d, int f, int r, int planned, int backward) {
  if (check_sizes(1, n, E, L) || check_dims(d, f, r)) return 0;
  if (backward) return static_cast<size_t>(max(down_bwd_space(n, E, L, d, f, r).bytes, gate_up_bwd_space(n, E, L, d, f, r).bytes));
  if (!planned) return 0;      // one kernel, which keeps v to itself
  return static_cast<size_t>(max(part_bytes(n, E, L, 2 * r, d), part_bytes(n, E, L, r, f)));
}

extern "C" int moe_adapter_gate_up(const uint16_t* x, const int32_t* ids, const int32_t* row_token, const int32_t* offsets,
                                   const void* plan, int T, int n, int E, int L, int d, int f, int r,
                                   const uint16_t* a_gu, const uint16_t* b_gate, const uint16_t* b_up, const float* scale,
                                   const int64_t* rng, float p, int site, const uint16_t* g, const uint16_t* u,
                                   const uint16_t* a, uint16_t* v, uint16_t* g_out, uint16_t* u_out, uint16_t* a_out,
                                   void* ws, size_t ws_bytes, void* stream) {
  const Rows rows = {static_cast<const int32_t*>(plan), ids, row_token, offsets, T, n, E, L};
  if (int st = check_rows(rows)) return st;
  if (int st = check_few(rows)) return st;
  if (int st = check_dims(d, f, r)) return st;
  MOE_CHECK_PTR(x); MOE_CHECK_PTR(a_gu); MOE_CHECK_PTR(b_gate); MOE_CHECK_PTR(b_up); MOE_CHECK_PTR(scale);
  MOE_CHECK_PTR(g); MOE_CHECK_PTR(u); MOE_CHECK_PTR(a); MOE_CHECK_PTR(a_out);
  MOE_CHECK_ALIGN(x); MOE_CHECK_ALIGN(a_gu); MOE_CHECK_ALIGN(b_gate); MOE_CHECK_ALIGN(b_up);
  MOE_CHECK_ALIGN(g); MOE_CHECK_ALIGN(u); MOE_CHECK_ALIGN(a); MOE_CHECK_ALIGN(v);
  MOE_CHECK_ALIGN(g_out); MOE_CHECK_ALIGN(u_out); MOE_CHECK_ALIGN(a_out);
  MOE_REQUIRE((g_out == nullptr) == (u_out == nullptr), MOE_ERR_INVALID_ARG, "g_out and u_out are wanted both or neither");
  DropArgs drop;
  if (int st = make_drop(rng, p, site, &drop)) return st;
  hipStream_t st = as_stream(stream);
  if (plan == nullptr) {
    const RowArgs k = {rows, x, 1, d, 2 * r, a_gu, f, r, {b_gate, b_up}, scale, {g, u, a}, {g_out, u_out, a_out}, v, drop};
    if (drop.drop) launch_rows<kSwiglu, true>(k, st);
    else launch_rows<kSwiglu, false>(k, st);
    return check_launch("adapter_gate_up");
  }
  MOE_CHECK_WS(part_bytes(n, E, L, 2 * r, d));
  float* part = static_cast<float*>(ws);
  const int S = slices(n, E, L, d);
  ShrinkArgs s = {rows, {x, nullptr}, {a_gu, nullptr}, {0, 0}, 1, d, 2 * r, 2 * r, S, 1, nullptr, part, v, drop};
  ExpandArgs e = {rows, part, 2 * r, S, r, f, 1, {b_gate, b_up}, scale, {g, u, a, nullptr}, {g_out, u_out, a_out},
                  S > 1 ? v : nullptr, nullptr, DropArgs{}};
  const int both = drop.drop == 0 ? both_rows(rows, 2 * r) : 0;
  if (both) {
    e.v_out = v;
    launch_both<kSwiglu>(both, s, e, st);
    return check_launch("adapter_gate_up");
  }
  if (drop.drop) launch_shrink<true>(s, 1, st);
  else launch_shrink<false>(s, 1, st);
  launch_expand<kSwiglu, false>(e, st);
  return check_launch("adapter_gate_up");
}

extern "C" int moe_adapter_down(const uint16_t* a, const int32_t* ids, const int32_t* row_token, const int32_t* offsets,
                                const void* plan, int T, int n, int E, int L, int d, int f, int r, const uint16_t* a_down,
                                const uint16_t* b_down, const float* scale, const int64_t* rng, float p, int site,
                                const uint16_t* yexp, uint16_t* v, uint16_t* y_out, void* ws, size_t ws_bytes, void* stream) {
  const Rows rows = {static_cast<const int32_t*>(plan), ids, row_token, offsets, T, n, E, L};
  if (int st = check_rows(rows)) return st;
  if (int st = check_few(rows)) return st;
  if (int st = check_dims(d, f, r)) return st;
  MOE_CHECK_PTR(a); MOE_CHECK_PTR(a_down); MOE_CHECK_PTR(b_down); MOE_CHECK_PTR(scale); MOE_CHECK_PTR(yexp);
  MOE_CHECK_PTR(y_out);
  MOE_CHECK_ALIGN(a); MOE_CHECK_ALIGN(a_down); MOE_CHECK_ALIGN(b_down); MOE_CHECK_ALIGN(yexp); MOE_CHECK_ALIGN(v);
  MOE_CHECK_ALIGN(y_out);
  DropArgs drop;
  if (int st = make_drop(rng, p, site, &drop)) return st;
  hipStream_t st = as_stream(stream);
  if (plan == nullptr) {
    const RowArgs k = {rows, a, 0, f, r, a_down, d, r, {b_down, nullptr}, scale, {yexp, nullptr, nullptr},
                       {y_out, nullptr, nullptr}, v, drop};
    if (drop.drop) launch_rows<kAdd, true>(k, st);
    else launch_rows<kAdd, false>(k, st);
    return check_launch("adapter_down");
  }
  MOE_CHECK_WS(part_bytes(n, E, L, r, f));
  float* part = static_cast<float*>(ws);
  const int S = slices(n, E, L, f);
  ShrinkArgs s = {rows, {a, nullptr}, {a_down, nullptr}, {0, 0}, 0, f, r, r, S, 1, nullptr, part, v, drop};
  ExpandArgs e = {rows, part, r, S, r, d, 1, {b_down, nullptr}, scale, {yexp, nullptr, nullptr, nullptr},
                  {y_out, nullptr, nullptr}, S > 1 ? v : nullptr, nullptr, DropArgs{}};
  const int both = drop.drop == 0 ? both_rows(rows, r) : 0;
  if (both) {
    e.v_out = v;
    launch_both<kAdd>(both, s, e, st);
    return check_launch("adapter_down");
  }
  if (drop.drop) launch_shrink<true>(s, 1, st);
  else launch_shrink<false>(s, 1, st);
  launch_expand<kAdd, false>(e, st);
  return check_launch("adapter_down");
}

extern "C" int moe_adapter_down_bwd(const uint16_t* dyexp, const uint16_t* a, const uint16_t* v, const int32_t* ids,
                                    const int32_t* row_token, const int32_t* offsets, const void* plan, int T, int n, int E,
                                    int L, int d, int f, int r, const uint16_t* a_down, const uint16_t* b_down,
                                    const float* scale, const int64_t* rng, float p, int site, const uint16_t* g,
                                    const uint16_t* u, const uint16_t* dg, const uint16_t* du, uint16_t* dg_out,
                                    uint16_t* du_out, uint16_t* d_a_down, uint16_t* d_b_down, void* ws, size_t ws_bytes,
                                    void* stream) {
  const Rows rows = {static_cast<const int32_t*>(plan), ids, row_token, offsets, T, n, E, L};
  if (int st = check_rows(rows)) return st;
  if (int st = check_dims(d, f, r)) return st;
  MOE_CHECK_PTR(plan);
  MOE_CHECK_PTR(dyexp); MOE_CHECK_PTR(a); MOE_CHECK_PTR(v); MOE_CHECK_PTR(a_down); MOE_CHECK_PTR(b_down);
  MOE_CHECK_PTR(scale); MOE_CHECK_PTR(g); MOE_CHECK_PTR(u); MOE_CHECK_PTR(dg); MOE_CHECK_PTR(du);
  MOE_CHECK_PTR(dg_out); MOE_CHECK_PTR(du_out); MOE_CHECK_PTR(d_a_down); MOE_CHECK_PTR(d_b_down);
  MOE_CHECK_ALIGN(dyexp); MOE_CHECK_ALIGN(a); MOE_CHECK_ALIGN(v); MOE_CHECK_ALIGN(a_down); MOE_CHECK_ALIGN(b_down);
  MOE_CHECK_ALIGN(g); MOE_CHECK_ALIGN(u); MOE_CHECK_ALIGN(dg); MOE_CHECK_ALIGN(du); MOE_CHECK_ALIGN(dg_out);
  MOE_CHECK_ALIGN(du_out); MOE_CHECK_ALIGN(d_a_down); MOE_CHECK_ALIGN(d_b_down);
  DropArgs drop;
  if (int st = make_drop(rng, p, site, &drop)) return st;
  const BwdSpace space = down_bwd_space(n, E, L, d, f, r);
  MOE_CHECK_WS(space.bytes);
  char* base = static_cast<char*>(ws);
  float* part = reinterpret_cast<float*>(base + space.part);
  float* dv = reinterpret_cast<float*>(base + space.sum);
  float* pieces_b = reinterpret_cast<float*>(base + space.pieces_b);
  float* pieces_a = reinterpret_cast<float*>(base + space.pieces_a);
  const int S = slices(n, E, L, d);
  hipStream_t st = as_stream(stream);
  // dyexp's second reader follows its first, so that what the last-level cache still holds of it is found there
  const ShrinkArgs s = {rows, {dyexp, nullptr}, {b_down, nullptr}, {0, 0}, 0, d, r, r, S, 1, scale, part, nullptr, DropArgs{}};
  launch_shrink<false>(s, 1, st);
  const WgradArgs wb = {rows, v, nullptr, {0, 0}, {dyexp, nullptr}, 0, r, r, d, scale, {d_b_down, nullptr}, pieces_b, DropArgs{}};
  launch_wgrad<false, false>(wb, 1, st);
  const ExpandArgs e = {rows, part, r, S, r, f, 1, {a_down, nullptr}, nullptr, {g, u, dg, du}, {dg_out, du_out, nullptr},
                        nullptr, S > 1 ? dv : nullptr, drop};
  if (drop.drop) launch_expand<kSwigluBwd, true>(e, st);
  else launch_expand<kSwigluBwd, false>(e, st);
  const WgradArgs wa = {rows, nullptr, dv, {0, 0}, {a, nullptr}, 0, r, r, f, nullptr, {d_a_down, nullptr}, pieces_a, drop};
  if (drop.drop) launch_wgrad<true, true>(wa, 1, st);
  else launch_wgrad<false, true>(wa, 1, st);
  launch_join({rows, {pieces_b, pieces_a, nullptr}, {d_b_down, d_a_down, nullptr}, {r, r, 0}, {d, f, 0}}, 2, st);
  return check_launch("adapter_down_bwd");
}

extern "C" int moe_adapter_gate_up_bwd(const uint16_t* dg, const uint16_t* du, const uint16_t* x, const uint16_t* v,
                                       const int32_t* ids, const int32_t* row_token, const int32_t* offsets,
                                       const void* plan, int T, int n, int E, int L, int d, int f, int r,
                                       const uint16_t* a_gu, const uint16_t* b_gate, const uint16_t* b_up,
                                       const float* scale, const int64_t* rng, float p, int site, const uint16_t* dxp,
                                       uint16_t* dxp_out, uint16_t* d_a_gu, uint16_t* d_b_gate, uint16_t* d_b_up, void* ws,
                                       size_t ws_bytes, void* stream) {
  const Rows rows = {static_cast<const int32_t*>(plan), ids, row_token, offsets, T, n, E, L};
  if (int st = check_rows(rows)) return st;
  if (int st = check_dims(d, f, r)) return st;
  MOE_CHECK_PTR(plan);
  MOE_CHECK_PTR(dg); MOE_CHECK_PTR(du); MOE_CHECK_PTR(x); MOE_CHECK_PTR(v); MOE_CHECK_PTR(a_gu); MOE_CHECK_PTR(b_gate);
  MOE_CHECK_PTR(b_up); MOE_CHECK_PTR(scale); MOE_CHECK_PTR(dxp); MOE_CHECK_PTR(dxp_out); MOE_CHECK_PTR(d_a_gu);
  MOE_CHECK_PTR(d_b_gate); MOE_CHECK_PTR(d_b_up);
  MOE_CHECK_ALIGN(dg); MOE_CHECK_ALIGN(du); MOE_CHECK_ALIGN(x); MOE_CHECK_ALIGN(v); MOE_CHECK_ALIGN(a_gu);
  MOE_CHECK_ALIGN(b_gate); MOE_CHECK_ALIGN(b_up); MOE_CHECK_ALIGN(dxp); MOE_CHECK_ALIGN(dxp_out);
  MOE_CHECK_ALIGN(d_a_gu); MOE_CHECK_ALIGN(d_b_gate); MOE_CHECK_ALIGN(d_b_up);
  DropArgs drop;
  if (int st = make_drop(rng, p, site, &drop)) return st;
  const BwdSpace space = gate_up_bwd_space(n, E, L, d, f, r);
  MOE_CHECK_WS(space.bytes);
  char* base = static_cast<char*>(ws);
  float* part = reinterpret_cast<float*>(base + space.part);
  float* dv = reinterpret_cast<float*>(base + space.sum);
  float* pieces_b = reinterpret_cast<float*>(base + space.pieces_b);
  float* pieces_a = reinterpret_cast<float*>(base + space.pieces_a);
  const int S = slices(n, E, L, f);
  hipStream_t st = as_stream(stream);
  const ShrinkArgs s = {rows, {dg, du}, {b_gate, b_up}, {0, r}, 0, f, r, 2 * r, S, 1, scale, part, nullptr, DropArgs{}};
  launch_shrink<false>(s, 2, st);
  const WgradArgs wb = {rows, v, nullptr, {0, r}, {dg, du}, 0, 2 * r, r, f, scale, {d_b_gate, d_b_up}, pieces_b, DropArgs{}};
  launch_wgrad<false, false>(wb, 2, st);
  const ExpandArgs e = {rows, part, 2 * r, S, 2 * r, d, 1, {a_gu, nullptr}, nullptr, {dxp, nullptr, nullptr, nullptr},
                        {dxp_out, nullptr, nullptr}, nullptr, S > 1 ? dv : nullptr, drop};
  if (drop.drop) launch_expand<kAdd, true>(e, st);
  else launch_expand<kAdd, false>(e, st);
  const WgradArgs wa = {rows, nullptr, dv, {0, 0}, {x, nullptr}, 1, 2 * r, 2 * r, d, nullptr, {d_a_gu, nullptr}, pieces_a, drop};
  if (drop.drop) launch_wgrad<true, true>(wa, 1, st);
  else launch_wgrad<false, true>(wa, 1, st);
  const float* second = pieces_b + 2LL * (n / piece_rows(n) + 1) * r * f;
  launch_join({rows, {pieces_b, second, pieces_a}, {d_b_gate, d_b_up, d_a_gu}, {r, r, 2 * r}, {f, f, d}}, 3, st);
  return check_launch("adapter_gate_up_bwd");
}
