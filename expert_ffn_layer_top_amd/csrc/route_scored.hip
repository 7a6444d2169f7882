// The scored router: a score for every expert (the sigmoid of its logit, or the softmax over all of
// them), a bias for balance that is added for the choice alone, the best groups of experts, the k
// best experts of those, and gates from the unbiased scores; its gradient.
//
//   s[e] = sigmoid(l[e]) or exp(l[e] - max) / sum
//   c[e] = s[e] + bias[e]                                         (-inf where l[e] is -inf or NaN)
//   v[g] = sum of the group_top largest c of group g              (E / n_group experts each)
//   choice: the topk_group groups of largest v, of their experts the k of largest c (of largest l
//   where there is no bias), ties to the lower index; gate = scale * s / (sum of the chosen s)
//
// The choice is the one that 64-bit scores make: with 256 experts a batch of 32768 tokens has a handful
// whose k-th and next value differ by less than one fp32 rounding, and a choice that depends on how fp32
// rounds an exponential would differ between implementations and move every later row of two experts.
// Computing it all in 64 bits is what the first version did, and it was bound by those exponentials (130
// us for 32768 tokens of 256 experts).  So a token is chosen from fp32 scores with a bound on their error,
// and the few tokens (about 1 in 700 there) where two values that the choice separates are closer than the
// bound are chosen again from 64-bit ones, as every token is whose scores are asked for.  Gates are computed from their
// logits in 64 bits, all of a block's together; only the sum over all experts, by which a softmax's are divided that are
// not renormalised, is the choice's own, of fp32 exponentials.  Measured for that batch, us: choice 21, gates and ranks 18, scan 5, rows 6; one token in
// one launch 7.5; the gradient of 16384 tokens of 128 experts (softmax, not renormalised) 10.
#include <algorithm>
#include <cmath>

#include "common.h"

namespace moe {
namespace {

constexpr int kRouteBlock = 64;                // tokens per block (one bit each in a 64-bit mask)
constexpr int kLocalThreads = 512;             // 8 waves of some 110 registers: two blocks per compute unit
constexpr int kMaxK = 16;
constexpr int kMaxE = 256;
constexpr int kQ = kMaxE / 64;                 // experts of a lane: kQ lane .. kQ lane + kQ - 1
constexpr int kOut = INT32_MIN;                // key of an expert that cannot be chosen (any more)

// A logit as the router reads it: NaN counts as -inf (an absent expert), +inf as the largest float.
__device__ __forceinline__ float clean_logit(float l) {
  return l != l ? -INFINITY : fminf(l, 3.4028234663852886e38f);
}

// Order-preserving map of a float to int (-0 as +0; never kOut), and back.
__device__ __forceinline__ int float_key(float v) {
  const int b = __float_as_int(v + 0.0f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_float(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

// The same for a double, to uint64 (never 0).
__device__ __forceinline__ unsigned long long double_key(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return b < 0 ? ~static_cast<unsigned long long>(b) : static_cast<unsigned long long>(b) | 0x8000000000000000ull;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Largest key over the wave, as a scalar: row shifts within 16 lanes, then broadcasts across rows.
template <int CTRL>
__device__ __forceinline__ int dpp_max(int v) {
  return max(v, __builtin_amdgcn_update_dpp(kOut, v, CTRL, 0xf, 0xf, false));   // folds into one v_max
}
__device__ __forceinline__ int wave_max_key(int v) {
  v = dpp_max<0x111>(v);
  v = dpp_max<0x112>(v);
  v = dpp_max<0x114>(v);
  v = dpp_max<0x118>(v);
  v = dpp_max<0x142>(v);
  v = dpp_max<0x143>(v);
  return __builtin_amdgcn_readlane(v, 63);
}

// Orders the wave's LDS accesses before and after (lanes of one wave exchange values through LDS).
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

struct ScoredArgs {
  const float* logits;
  const float* bias;
  int T, E, k, score, n_group, topk_group, group_top, renormalize;
  float scale;
};

// The k chosen experts of one token in lanes 0 .. k-1, from 64-bit scores; one wave per token.
// `scores`: this token's row of the score output, or null.  Rarely taken, so it keeps its values in LDS and
// its loops rolled: unrolled, its exponentials set the kernel's registers and halved the waves in flight.
__device__ __forceinline__ int choose_exact(const ScoredArgs& a, const float (&l)[kQ], int lane, double* s_c,
                                            float* __restrict__ scores) {
  const int e0 = kQ * lane;
  const double ninf = -INFINITY;
  const bool sigmoid = a.score == MOE_SCORE_SIGMOID;
  const float m = sigmoid ? 0.f : wave_max(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])));
  const double md = m == -INFINITY ? 0.0 : static_cast<double>(m);
  double sum = 0.0;
#pragma unroll
  for (int q = 0; q < kQ; ++q) s_c[e0 + q] = static_cast<double>(l[q]);
#pragma unroll 1
  for (int q = 0; q < kQ; ++q) {
    const double x = s_c[e0 + q], y = exp(sigmoid ? -x : x - md);
    s_c[e0 + q] = y;
    sum += y;
  }
  if (!sigmoid) sum = wave_sum_f64(sum);
#pragma unroll 1
  for (int q = 0; q < kQ; ++q) {
    const int e = e0 + q;
    const double y = s_c[e], p = sigmoid ? 1.0 / (1.0 + y) : (sum > 0.0 ? y / sum : 0.0);
    const float lq = q == 0 ? l[0] : (q == 1 ? l[1] : (q == 2 ? l[2] : l[3]));
    double c = p;
    if (e < a.E) {
      if (scores != nullptr) scores[e] = static_cast<float>(p);
      if (a.bias != nullptr) c += static_cast<double>(a.bias[e]);
    }
    s_c[e] = lq == -INFINITY || c != c ? ninf : c;
  }
  wave_lds_sync();
  unsigned long long kept[kQ] = {~0ull, ~0ull, ~0ull, ~0ull};     // kept groups, 64 to a word
  const int per = a.E / a.n_group;
  if (a.topk_group < a.n_group) {
#pragma unroll
    for (int q = 0; q < kQ; ++q) kept[q] = 0ull;
    unsigned long long gkey[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const int g = lane + 64 * q;
      gkey[q] = 0ull;
      if (g < a.n_group) {
        double b0 = ninf, b1 = ninf;
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
          const double v = s_c[g * per + i];
          b1 = v > b0 ? b0 : (v > b1 ? v : b1);
          b0 = v > b0 ? v : b0;
        }
        gkey[q] = double_key(a.group_top == 1 || b1 == ninf ? b0 : b0 + b1);
      }
    }
#pragma unroll 1
    for (int r = 0; r < a.topk_group; ++r) {
      unsigned long long best = gkey[0];
#pragma unroll
      for (int q = 1; q < kQ; ++q) best = gkey[q] > best ? gkey[q] : best;
      best = wave_max_u64(best);
      int g = -1;
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const unsigned long long hit = __ballot(gkey[q] == best);
        if (g < 0 && hit) g = 64 * q + __ffsll(static_cast<long long>(hit)) - 1;
      }
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        if (lane + 64 * q == g) gkey[q] = 0ull;
        if (g >> 6 == q) kept[q] |= 1ull << (g & 63);
      }
    }
  }
  unsigned long long key[kQ];
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const int e = e0 + q, g = e / per;
    unsigned long long word = kept[0];
#pragma unroll
    for (int i = 1; i < kQ; ++i) word = g >> 6 == i ? kept[i] : word;
    const double v = a.bias != nullptr ? s_c[e] : static_cast<double>(l[q]);
    key[q] = e < a.E && (word >> (g & 63) & 1ull) ? double_key(v) : 0ull;
  }
  int my_e = 0;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    unsigned long long best = key[0];
    int bq = 0;
#pragma unroll
    for (int q = 1; q < kQ; ++q)
      if (key[q] > best) { best = key[q]; bq = q; }
    const unsigned long long top = wave_max_u64(best);
    const int src = __ffsll(static_cast<long long>(__ballot(best == top))) - 1;   // lower lanes hold lower experts
    const int e = kQ * src + __shfl(bq, src, 64);
    if (lane == j) my_e = e;
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      if (e0 + q == e) key[q] = 0ull;
  }
  wave_lds_sync();
  return my_e;
}

// How far apart two values of fp32 scores have to be (beside 2^-22 of the value: adding a bias rounds to 2^-24 of the
// result) to be in the same order in 64 bits.  With u = 2^-24, an exponential of x is off by 2.3 u |x| (x, log2 e and
// their product are rounded) + 2 u (a unit of the instruction) of itself.
//   sigmoid  x = -l is exact, which leaves s (1 - s) (1.3 u |l| + 2 u) < 0.8 u; rounding 1 + exp(-l) adds u, the
//            reciprocal 2 u: less than 2^-22 each, 2^-21 for two.
//   softmax  p = e^x / sum: 2.3 u |x| + 2 u of its own, and the mean of that over all experts for the sum, with 9 u
//            for at most 9 levels of additions, and u each for 1 / sum and the product; together
//            p (15 u + 2.3 u (|x| + mean |x|)).  The p add up to 1, and where one is near it the mean of |x| is small (256
//            experts: 15.2 u at p = 0.95 is the most that one or two can be off), so the difference of two experts'
//            scores is off by less than 15.2 u, that of two groups' sums by less than 17 u.
// Twice that is taken.
__device__ __forceinline__ float score_margin(const ScoredArgs& a) {
  return a.score == MOE_SCORE_SIGMOID ? 0x1p-20f : 0x1p-19f;
}

// Where a group's value lies in 64 bits, from the fp32 values b0 >= b1 of its best two experts (-inf: absent).
// Each of them is off by its score's error and by 2^-24 of itself, to which adding
// the bias rounds it; their sum by 2^-24 of the sum, and the bounds by as much again.  The two may cancel (biases of
// either sign), so the margin counts their magnitudes, not the sum's.  Not `known` where those leave fp32.
struct GroupRange {
  float lo, hi;
  bool known;
};
__device__ __forceinline__ GroupRange group_range(const ScoredArgs& a, float b0, float b1) {
  const bool two = a.group_top == 2 && b1 != -INFINITY;
  const float v = two ? b0 + b1 : b0, size = two ? fabsf(b0) + fabsf(b1) : fabsf(b0);
  const bool absent = b0 == -INFINITY;
  const float tol = absent ? 0.f : score_margin(a) + 0x1p-22f * size;
  return {v - tol, v + tol, absent || size < INFINITY};
}

// The same choice from fp32 scores, with my_e valid where the result is true: whether every comparison
// that the choice rests on is wider than the scores' error (score_margin, group_range).  Logits compare exactly.
// m_out, sum_out: the softmax's maximum and sum.
__device__ __forceinline__ bool choose_fast(const ScoredArgs& a, const float (&l)[kQ], const float (&bias)[kQ], int lane,
                                            float* s_choice, int& my_e, float& m_out, float& sum_out) {
  const int e0 = kQ * lane;
  const bool grouped = a.topk_group < a.n_group;
  float c[kQ];
  m_out = 0.f;
  sum_out = 1.f;
  if (a.score == MOE_SCORE_SOFTMAX) {
    float m = fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3]));
    m = key_float(wave_max_key(float_key(m)));
    m_out = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      c[q] = __expf(l[q] - m_out);
      sum += c[q];
    }
    sum_out = wave_sum(sum);
    const float inv = sum_out > 0.f ? 1.f / sum_out : 0.f;
#pragma unroll
    for (int q = 0; q < kQ; ++q) c[q] *= inv;
  } else if (a.bias != nullptr || grouped) {
#pragma unroll
    for (int q = 0; q < kQ; ++q) c[q] = __builtin_amdgcn_rcpf(1.f + __expf(-l[q]));
  }
  if (a.bias != nullptr || grouped) {
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      c[q] += bias[q];
      if (l[q] == -INFINITY || c[q] != c[q]) c[q] = -INFINITY;
    }
  }
  bool sure = true;
  int key[kQ];
#pragma unroll
  for (int q = 0; q < kQ; ++q) key[q] = e0 + q < a.E ? float_key(a.bias != nullptr ? c[q] : l[q]) : kOut;
  if (grouped) {
    if (a.n_group > 64) return false;
    const int per = a.E / a.n_group, lanes = per / kQ;
    // v: the value of the lane's group, groups `stride` lanes apart.  Groups of whole aligned runs of 4, 8, ..
    // experts merge the best two of each lane, others (20 or 40 experts, say) are walked in LDS, a lane each.
    const bool aligned = per % kQ == 0 && (lanes & (lanes - 1)) == 0;
    const int stride = aligned ? lanes : 1;
    float b0, b1;
    if (aligned) {
      b0 = fmaxf(c[0], c[1]);
      b1 = fminf(c[0], c[1]);
#pragma unroll
      for (int q = 2; q < kQ; ++q) {
        b1 = fmaxf(b1, fminf(b0, c[q]));
        b0 = fmaxf(b0, c[q]);
      }
      for (int o = 1; o < lanes; o <<= 1) {
        const float p0 = __shfl_xor(b0, o, 64), p1 = __shfl_xor(b1, o, 64);
        b1 = fmaxf(fminf(b0, p0), fmaxf(b1, p1));
        b0 = fmaxf(b0, p0);
      }
    } else {
#pragma unroll
      for (int q = 0; q < kQ; ++q) s_choice[e0 + q] = c[q];
      wave_lds_sync();
      b0 = b1 = -INFINITY;
      if (lane < a.n_group) {
        for (int i = 0; i < per; ++i) {
          const float x = s_choice[lane * per + i];
          b1 = fmaxf(b1, fminf(b0, x));
          b0 = fmaxf(b0, x);
        }
      }
      wave_lds_sync();
    }
    const GroupRange v = group_range(a, b0, b1);
    // kept: at most topk_group groups (itself among them) may be as large; dropped: at least that many are
    // larger for certain; neither: not sure
    int maybe = 0, above = 0;
    for (int i = 0; i < a.n_group; ++i) {
      const float lo = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v.lo), i * stride));
      const float hi = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v.hi), i * stride));
      maybe += hi >= v.lo ? 1 : 0;
      above += lo > v.hi ? 1 : 0;
    }
    const bool in = maybe <= a.topk_group;
    const bool counts = lane < a.n_group * stride;       // lanes that hold a group
    if (__ballot(counts && ((!in && above < a.topk_group) || !v.known)) != 0ull) return false;
    const unsigned long long kept = __ballot(counts && in);
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const int g = aligned ? lane : (e0 + q) / per;
      if (!(kept >> (g & 63) & 1ull)) key[q] = kOut;
    }
  }
  // each lane's experts in descending order (stable: adjacent swaps of strictly larger keys), their
  // positions in the bytes of `order`
  int pos[kQ] = {0, 1, 2, 3};
  auto swap = [&](int i) {
    const bool up = key[i + 1] > key[i];
    const int x = key[i], y = pos[i];
    key[i] = up ? key[i + 1] : x;
    key[i + 1] = up ? x : key[i + 1];
    pos[i] = up ? pos[i + 1] : y;
    pos[i + 1] = up ? y : pos[i + 1];
  };
  swap(0); swap(1); swap(2);
  swap(0); swap(1);
  swap(0);
  unsigned order = pos[0] | pos[1] << 8 | pos[2] << 16 | pos[3] << 24;
  my_e = 0;
  float last = 0.f;
  const int rounds = a.k + (a.bias != nullptr ? 1 : 0);
  const float margin = score_margin(a);
  for (int j = 0; j < rounds; ++j) {
    const int m = wave_max_key(key[0]);
    if (a.bias != nullptr) {
      const float v = key_float(m);
      if (j > 0 && m != kOut) sure = sure && last - v > margin + 0x1p-22f * fabsf(last);
      if (j > 0 && m == kOut) sure = sure && last > -INFINITY;
      last = v;
    }
    if (j == a.k) break;
    const int src = __ffsll(static_cast<long long>(__ballot(key[0] == m))) - 1;
    const int e = kQ * src + (__builtin_amdgcn_readlane(order, src) & 0xff);
    my_e = lane == j ? e : my_e;
    const bool pop = lane == src;
    key[0] = pop ? key[1] : key[0];
    key[1] = pop ? key[2] : key[1];
    key[2] = pop ? key[3] : key[2];
    key[3] = pop ? kOut : key[3];
    order = pop ? order >> 8 : order;
  }
  return sure;
}

// Inclusive scan over the 256 first threads of two values at once (every thread of the block calls it).
__device__ __forceinline__ void scan256(int& x, int& y, int (*s_part)[2]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int p = __shfl_up(x, o, 64), q = __shfl_up(y, o, 64);
    if (lane >= o) { x += p; y += q; }
  }
  if (lane == 63 && wave < 4) { s_part[wave][0] = x; s_part[wave][1] = y; }
  __syncthreads();
  for (int w = 0; w < wave && w < 3; ++w) { x += s_part[w][0]; y += s_part[w][1]; }
}

struct MetaOut {
  int32_t* counts;
  int32_t* offsets;
  int32_t* offsets_pad;
  int pad;
  int32_t* dest;
  int32_t* row_token;
};

// Offsets of the experts from their counts: thread e < 256 gives its count, and afterwards holds in
// s_off[e] its first row; `lead` also writes offsets and offsets_pad.
__device__ __forceinline__ void expert_offsets(int count, int E, const MetaOut& m, bool lead, int* s_off,
                                               int (*s_part)[2]) {
  const int e = threadIdx.x;
  const int padded = m.offsets_pad != nullptr ? (count + m.pad - 1) / m.pad * m.pad : 0;
  int x = count, y = padded;
  scan256(x, y, s_part);
  if (e < kMaxE) s_off[e] = x - count;
  if (lead && e < E) {
    m.offsets[e + 1] = x;
    if (e == 0) m.offsets[0] = 0;
    if (m.offsets_pad != nullptr) {
      m.offsets_pad[e + 1] = y;
      if (e == 0) m.offsets_pad[0] = 0;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ float group_sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ float group_max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

// One token's logits, 4 per lane (-inf past the experts and past the tokens).
__device__ __forceinline__ void load_logits(const ScoredArgs& a, long long t, int lane, float (&l)[kQ]) {
  if ((a.E & 3) == 0) {
    const bool in = t < a.T && kQ * lane < a.E;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) v = *reinterpret_cast<const float4*>(a.logits + t * a.E + kQ * lane);
    l[0] = in ? v.x : -INFINITY; l[1] = in ? v.y : -INFINITY;
    l[2] = in ? v.z : -INFINITY; l[3] = in ? v.w : -INFINITY;
  } else {
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      l[q] = t < a.T && kQ * lane + q < a.E ? a.logits[t * a.E + kQ * lane + q] : -INFINITY;
  }
}

__device__ __forceinline__ void load_bias(const ScoredArgs& a, int lane, float (&bias)[kQ]) {
#pragma unroll
  for (int q = 0; q < kQ; ++q)
    bias[q] = a.bias != nullptr && kQ * lane + q < a.E ? a.bias[kQ * lane + q] : 0.f;
}

// The fp32 choice of more than 64 tokens, a wave per token, -1 in the token's first slot where
// that does not decide it.  Apart from the 64-bit code, whose registers (96 instead of 56) would halve the
// waves in flight: this kernel is bound by the latency of its chains of reductions.
constexpr int kChooseWaves = 4, kChooseTokens = 4;
__global__ __launch_bounds__(64 * kChooseWaves, 8) void route_scored_choose(ScoredArgs a, int32_t* __restrict__ topk_idx,
                                                                           float2* __restrict__ softmax_sums) {
  __shared__ float s_choice[kChooseWaves][kMaxE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long long t0 = (static_cast<long long>(blockIdx.x) * kChooseWaves + wave) * kChooseTokens;
  float bias[kQ], next[kQ];
  load_bias(a, lane, bias);
  load_logits(a, t0, lane, next);
#pragma unroll 1
  for (int i = 0; i < kChooseTokens; ++i) {
    const long long t = t0 + i;
    if (t >= a.T) break;
    float l[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) l[q] = clean_logit(next[q]);
    if (i + 1 < kChooseTokens) load_logits(a, t + 1, lane, next);
    int e;
    float m, sum;
    const bool sure = choose_fast(a, l, bias, lane, s_choice[wave], e, m, sum);
    if (__ballot(!sure) != 0ull) e = -1;
    if (lane < a.k) topk_idx[t * a.k + lane] = e;
    if (softmax_sums != nullptr && lane == 0) softmax_sums[t] = make_float2(m, sum);
  }
}

// The fp32 choice of four tokens per wave, 16 lanes each and PL consecutive experts per lane: the form for
// batches.  A value and its expert are one double, the fp32 value's with the expert's number in mantissa bits
// that a float leaves zero (ties to the lower expert), so values sort and are maximised with their experts by
// v_max_f64 and v_min_f64 alone; each lane sorts its own, and a round takes the largest head of the 16 lanes.
// Same comparisons and bounds as choose_fast.  Both are bound by the instructions that they issue, and a wave
// per token spends all its lanes on the k rounds of one: some 700 per token against 350 here, 39 against 21 us
// for 32768 tokens of 256 experts, best 8 of the best 4 of 8 groups.  choose_fast stays for groups that are not
// whole lanes here and for the few tokens of a single launch, where lanes are plenty.
constexpr double kHuge = 0x1p129;              // stands for an infinity, whose mantissa has no room for a number
constexpr double kGone = -0x1p200;             // an expert that cannot be chosen

template <int CTRL>
__device__ __forceinline__ double row_max_step(double v) {
  const unsigned long long b = __double_as_longlong(v);
  const int lo = __builtin_amdgcn_mov_dpp(static_cast<int>(b), CTRL, 0xf, 0xf, true);
  const int hi = __builtin_amdgcn_mov_dpp(static_cast<int>(b >> 32), CTRL, 0xf, 0xf, true);
  const unsigned long long p = static_cast<unsigned>(lo) | static_cast<unsigned long long>(static_cast<unsigned>(hi)) << 32;
  return fmax(v, __longlong_as_double(p));
}
// Largest of each row of 16 lanes, in all of them (rotations by 8, 4, 2 and 1 lanes).
__device__ __forceinline__ double row_max(double v) {
  v = row_max_step<0x128>(v);
  v = row_max_step<0x124>(v);
  v = row_max_step<0x122>(v);
  return row_max_step<0x121>(v);
}

__device__ __forceinline__ double pack_expert(float v, int e) {
  const double d = fmax(fmin(static_cast<double>(v + 0.f), kHuge), -kHuge);
  const unsigned long long b = __double_as_longlong(d);
  const unsigned sign = static_cast<unsigned>(static_cast<int>(b >> 32) >> 31);
  return __longlong_as_double(b | ((255u - e) ^ (sign & 255u)));   // larger for the lower expert, whatever the sign
}
__device__ __forceinline__ int packed_expert(double d) {
  const unsigned long long b = __double_as_longlong(d);
  const unsigned sign = static_cast<unsigned>(static_cast<int>(b >> 32) >> 31);
  return static_cast<int>((static_cast<unsigned>(b) & 255u) ^ (~sign & 255u));
}

// PL consecutive values from p[e0] on; past `E` -inf.
template <int PL>
__device__ __forceinline__ void load_row(const float* p, int e0, int E, float (&v)[PL]) {
  if ((E & 3) == 0) {
#pragma unroll
    for (int q = 0; q < PL; q += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + min(e0 + q, E - 4));
      v[q] = x.x; v[q + 1] = x.y; v[q + 2] = x.z; v[q + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < PL; ++q) v[q] = p[min(e0 + q, E - 1)];
  }
#pragma unroll
  for (int q = 0; q < PL; ++q) v[q] = e0 + q < E ? v[q] : -INFINITY;
}

// Batcher's merge exchange, descending.
template <int N>
__device__ __forceinline__ void sort_descending(double (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const double x = v[i + j], y = v[i + j + q];
            v[i + j] = fmax(x, y);
            v[i + j + q] = fmin(x, y);
          }
}

constexpr int kQuadWaves = 4;
template <int PL>
__global__ __launch_bounds__(64 * kQuadWaves) void route_scored_choose_quad(ScoredArgs a, int32_t* __restrict__ topk_idx,
                                                                           float2* __restrict__ softmax_sums) {
  extern __shared__ double s_list[];       // [waves][rows][64]: a lane's experts after its best, best first
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane & 15, row = lane & 48;
  const long long t = (static_cast<long long>(blockIdx.x) * kQuadWaves + wave) * 4 + (lane >> 4);
  const int e0 = PL * j;
  const bool live = t < a.T, grouped = a.topk_group < a.n_group, biased = a.bias != nullptr;
  float l[PL], c[PL];
  load_row<PL>(a.logits + (live ? t : 0) * a.E, e0, a.E, l);
#pragma unroll
  for (int q = 0; q < PL; ++q) l[q] = clean_logit(l[q]);
  if (a.score == MOE_SCORE_SOFTMAX) {
    float m = l[0];
#pragma unroll
    for (int q = 1; q < PL; ++q) m = fmaxf(m, l[q]);
    m = group_max16(m);
    m = m == -INFINITY ? 0.f : m;
    float part[PL];
#pragma unroll
    for (int q = 0; q < PL; ++q) part[q] = c[q] = __expf(l[q] - m);
#pragma unroll
    for (int w = PL / 2; w > 0; w /= 2)
#pragma unroll
      for (int q = 0; q < w; ++q) part[q] += part[q + w];
    const float sum = group_sum16(part[0]);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int q = 0; q < PL; ++q) c[q] *= inv;
    if (softmax_sums != nullptr && live && j == 0) softmax_sums[t] = make_float2(m, sum);
  } else if (biased || grouped) {
#pragma unroll
    for (int q = 0; q < PL; ++q) c[q] = __builtin_amdgcn_rcpf(1.f + __expf(-l[q]));
  }
  if (biased || grouped) {
#pragma unroll
    for (int q = 0; q < PL; ++q) c[q] = l[q] == -INFINITY ? -INFINITY : c[q];
  }
  if (biased) {
    float bias[PL];
    load_row<PL>(a.bias, e0, a.E, bias);
#pragma unroll
    for (int q = 0; q < PL; ++q) {
      c[q] += bias[q];
      c[q] = c[q] != c[q] ? -INFINITY : c[q];
      l[q] = c[q];                                // what the experts are compared by
    }
  }
  bool sure = true, in = true;
  if (grouped) {
    const int lanes = a.E / a.n_group / PL;
    float b0 = fmaxf(c[0], c[1]), b1 = fminf(c[0], c[1]);
#pragma unroll
    for (int q = 2; q < PL; ++q) {
      b1 = fmaxf(b1, fminf(b0, c[q]));
      b0 = fmaxf(b0, c[q]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const float p0 = __shfl_xor(b0, o, 64), p1 = __shfl_xor(b1, o, 64);
      b1 = fmaxf(fminf(b0, p0), fmaxf(b1, p1));
      b0 = fmaxf(b0, p0);
    }
    const GroupRange v = group_range(a, b0, b1);
    int maybe = 0, above = 0;
    for (int i = 0; i < a.n_group; ++i) {
      const float lo = __shfl(v.lo, row + i * lanes, 64), hi = __shfl(v.hi, row + i * lanes, 64);
      maybe += hi >= v.lo ? 1 : 0;
      above += lo > v.hi ? 1 : 0;
    }
    in = maybe <= a.topk_group;
    if (e0 < a.E) sure = (in || above >= a.topk_group) && v.known;
  }
  double key[PL];
#pragma unroll
  for (int q = 0; q < PL; ++q) {
    const double v = pack_expert(l[q], e0 + q);
    key[q] = in && e0 + q < a.E ? v : kGone;
  }
  sort_descending(key);
  const int rows = min(PL, a.k);                  // no round needs a lane's later ones
  double* list = s_list + wave * rows * 64 + lane;
#pragma unroll
  for (int q = 1; q <= PL; ++q)
    if (q <= rows) list[64 * (q - 1)] = q < PL ? key[q < PL ? q : 0] : kGone;
  double head = key[0];
  int at = 0;
  float last = 3.4028234663852886e38f;
  double mine = kGone;
  const int rounds = a.k + (biased ? 1 : 0);
  const float margin = score_margin(a);
  for (int i = 0; i < rounds; ++i) {              // (the last round of a biased choice only compares)
    const double m = row_max(head);
    const float v = static_cast<float>(m);        // -inf for kGone
    sure = sure & (!biased | (last - v > margin + 0x1p-22f * fabsf(last)));
    last = v;
    mine = j == i ? m : mine;
    const bool pop = head == m;
    const double next = list[64 * at];
    head = pop ? next : head;
    at = min(at + (pop ? 1 : 0), rows - 1);       // past a lane's last, its head stays kGone
  }
  const int my_e = packed_expert(mine);
  const unsigned long long doubt = __ballot(!sure);
  if (live && j < a.k) topk_idx[t * a.k + j] = (doubt >> row & 0xffffull) != 0ull ? -1 : my_e;
}

// 64 tokens per block: the choices that are not made yet, every gate (16 lanes per token, from
// the chosen logits in 64 bits) and the block's part of the row metadata.  Each (token, slot) sets its
// token's bit in its expert's 64-bit mask, so a row's rank among the block's rows of its expert is a
// popcount of the lower bits.  SINGLE: one block has all tokens, makes the whole choice and finishes the
// metadata; else it leaves the ranks in dest and its counts in hist [E][blocks].
template <bool SINGLE>
__global__ __launch_bounds__(SINGLE ? 1024 : kLocalThreads) void route_scored_local(ScoredArgs a, int32_t* __restrict__ topk_idx,
                                                               float* __restrict__ topk_gate,
                                                               float* __restrict__ scores,
                                                               const float2* __restrict__ softmax_sums,
                                                               int32_t* __restrict__ hist, MetaOut out) {
  constexpr int kThreads = SINGLE ? 1024 : kLocalThreads, kWaves = kThreads / 64, kWaveTokens = kRouteBlock / kWaves;
  constexpr int kHalf = kThreads / 16;           // tokens that the threads take at a time, 16 lanes each
  __shared__ unsigned long long s_mask[kMaxE];
  __shared__ int s_e[kRouteBlock][kMaxK];
  __shared__ float s_max[kRouteBlock], s_sum[kRouteBlock];
  __shared__ double s_choice[kWaves][kMaxE];
  __shared__ int s_off[kMaxE];
  __shared__ int s_part[4][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int j = tid & 15;
  const long long t0 = static_cast<long long>(blockIdx.x) * kRouteBlock;
  if (tid < kMaxE) s_mask[tid] = 0ull;
  if constexpr (SINGLE) {
    // the tokens dealt over the waves, so that a few tokens are a wave each
    float bias[kQ];
    load_bias(a, lane, bias);
#pragma unroll 1
    for (int i = wave; i < a.T; i += kWaves) {
      float l[kQ];
      load_logits(a, i, lane, l);
#pragma unroll
      for (int q = 0; q < kQ; ++q) l[q] = clean_logit(l[q]);
      int e;
      float m, sum;
      const bool sure = choose_fast(a, l, bias, lane, reinterpret_cast<float*>(s_choice[wave]), e, m, sum);
      if (__ballot(!sure) != 0ull || scores != nullptr)
        e = choose_exact(a, l, lane, s_choice[wave], scores != nullptr ? scores + static_cast<long long>(i) * a.E : nullptr);
      if (lane < a.k) s_e[i][lane] = e;
      if (lane == 0) { s_max[i] = m; s_sum[i] = sum; }
    }
  } else {
#pragma unroll
    for (int tl = tid >> 4; tl < kRouteBlock; tl += kHalf) {
      const long long t = t0 + tl;
      if (t < a.T && j < a.k) s_e[tl][j] = topk_idx[t * a.k + j];
      if (softmax_sums != nullptr && j == 0 && t < a.T) {
        const float2 v = softmax_sums[t];
        s_max[tl] = v.x;
        s_sum[tl] = v.y;
      }
    }
    wave_lds_sync();                             // a wave reads back its own tokens
#pragma unroll 1
    for (int i = 0; i < kWaveTokens; ++i) {
      const int it = 4 * wave + (i & 3) + (i >> 2) * kHalf;
      if (t0 + it >= a.T) continue;
      if (scores == nullptr && s_e[it][0] >= 0) continue;
      float l[kQ];
      load_logits(a, t0 + it, lane, l);
#pragma unroll
      for (int q = 0; q < kQ; ++q) l[q] = clean_logit(l[q]);
      const int e = choose_exact(a, l, lane, s_choice[wave], scores != nullptr ? scores + (t0 + it) * a.E : nullptr);
      if (lane < a.k) s_e[it][lane] = e;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int tl = tid >> 4; tl < kRouteBlock; tl += kHalf) {
    const long long t = t0 + tl;
    const bool live = t < a.T && j < a.k;
    const int e = live ? s_e[tl][j] : 0;
    if (live) atomicOr(&s_mask[e], 1ull << tl);
    float lj = live ? clean_logit(a.logits[t * a.E + e]) : -INFINITY;
    const bool sigmoid = a.score == MOE_SCORE_SIGMOID;
    // renormalised, the row's maximum cancels and the chosen logits' own serves
    float m = sigmoid ? 0.f : group_max16(lj);
    if (!sigmoid && !a.renormalize) m = t < a.T ? s_max[tl] : 0.f;
    const double x = static_cast<double>(lj);
    double p = lj == -INFINITY ? (sigmoid ? INFINITY : 0.0) : exp(sigmoid ? -x : x - static_cast<double>(m));
    if (sigmoid) p = 1.0 / (1.0 + p);
    double sum = 1.0;
    if (a.renormalize) {
      sum = p;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    } else if (!sigmoid) {
      sum = live ? static_cast<double>(s_sum[tl]) : 0.0;
    }
    const double gate = sum > 0.0 ? p / sum : 0.0;
    if (live) {
      topk_idx[t * a.k + j] = e;
      topk_gate[t * a.k + j] = static_cast<float>(gate * static_cast<double>(a.scale));
    }
  }
  __syncthreads();
  if constexpr (SINGLE) {
    const int count = tid < a.E ? __popcll(s_mask[tid]) : 0;
    if (tid < a.E) out.counts[tid] = count;
    expert_offsets(count, a.E, out, true, s_off, s_part);
  }
#pragma unroll
  for (int tl = tid >> 4; tl < kRouteBlock; tl += kHalf) {
    const long long t = t0 + tl;
    if (t >= a.T || j >= a.k) continue;
    const int e = s_e[tl][j], rank = __popcll(s_mask[e] & ((1ull << tl) - 1ull));
    if constexpr (SINGLE) {
      const int r = s_off[e] + rank;
      out.dest[t * a.k + j] = r;
      if (out.row_token != nullptr) out.row_token[r] = static_cast<int32_t>(t);
    } else {
      out.dest[t * a.k + j] = rank;
    }
  }
  if constexpr (!SINGLE)
    for (int i = tid; i < a.E; i += kThreads)
      hist[static_cast<long long>(i) * gridDim.x + blockIdx.x] = __popcll(s_mask[i]);
}

// One wave per expert: its block counts become exclusive prefixes, their sum counts[e].
__global__ __launch_bounds__(256) void route_scored_scan(int32_t* __restrict__ hist, int nb, int E,
                                                         int32_t* __restrict__ counts) {
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (e >= E) return;
  int32_t* h = hist + static_cast<long long>(e) * nb;
  int carry = 0;
  for (int b0 = 0; b0 < nb; b0 += 256) {          // 4 consecutive entries per lane
    int v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = b0 + 4 * lane + i < nb ? h[b0 + 4 * lane + i] : 0;
    const int own = v[0] + v[1] + v[2] + v[3];
    int incl = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int p = __shfl_up(incl, o, 64);
      if (lane >= o) incl += p;
    }
    int run = carry + incl - own;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (b0 + 4 * lane + i < nb) h[b0 + 4 * lane + i] = run;
      run += v[i];
    }
    carry += __shfl(incl, 63, 64);
  }
  if (lane == 0) counts[e] = carry;
}

// Rows: the expert's first row + its rows in earlier blocks + the rank in the block.  Every workgroup
// scans the 256 counts itself.
constexpr int kFinalThreads = 256, kFinalItems = 4;
__global__ __launch_bounds__(kFinalThreads) void route_scored_finalize(const int32_t* __restrict__ topk_idx,
                                                                       const int32_t* __restrict__ hist, int nb,
                                                                       long long n, int k, int E, MetaOut out) {
  __shared__ int s_off[kMaxE];
  __shared__ int s_part[4][2];
  const int e_t = threadIdx.x;
  const int count = e_t < E ? out.counts[e_t] : 0;
  const long long i0 = static_cast<long long>(blockIdx.x) * kFinalThreads * kFinalItems + threadIdx.x;
  int e[kFinalItems], rank[kFinalItems];
#pragma unroll
  for (int i = 0; i < kFinalItems; ++i) {
    const long long at = i0 + i * kFinalThreads;
    e[i] = at < n ? topk_idx[at] : 0;
    rank[i] = at < n ? out.dest[at] : 0;
  }
#pragma unroll
  for (int i = 0; i < kFinalItems; ++i) {
    const long long at = i0 + i * kFinalThreads;
    if (at < n) rank[i] += hist[static_cast<long long>(e[i]) * nb + at / k / kRouteBlock];
  }
  expert_offsets(count, E, out, blockIdx.x == 0, s_off, s_part);
#pragma unroll
  for (int i = 0; i < kFinalItems; ++i) {
    const long long at = i0 + i * kFinalThreads;
    if (at < n) {
      const int r = s_off[e[i]] + rank[i];
      out.dest[at] = r;
      if (out.row_token != nullptr) out.row_token[r] = static_cast<int32_t>(at / k);
    }
  }
}

// ---- gradient, with the choice held fixed:
//   sigmoid  dl = s (1 - s) ds,  softmax  dl[e] = s[e] (ds[e] - sum s ds),  ds of the chosen experts from
//   the gates (renormalised: ds_j = (dg_j - sum g dg) / sum s), 0 elsewhere.
// Renormalised gates come from the chosen logits alone, in the log domain, so scores that underflow still
// give finite ratios; only the plain softmax needs (and has) a gradient at every expert.
// Bound by its bytes (the gradient written, and the logits read by the plain softmax).  A wave takes four
// tokens, 16 lanes each, and forms their rows in LDS, so rows come and go as whole 16-byte runs.
constexpr int kBwdTokens = 4, kBwdWaves = 4;

template <bool DENSE>
__global__ __launch_bounds__(64 * kBwdWaves) void route_scored_bwd_kernel(const float* __restrict__ logits,
                                                                         const int32_t* __restrict__ idx,
                                                                         const float* __restrict__ dgate, int T, int E,
                                                                         int k, int score, int renormalize, float scale,
                                                                         float* __restrict__ dlogits) {
  // rows 16 floats past a multiple of 64 apart, so the four tokens' lanes use different banks
  __shared__ __attribute__((aligned(16))) float s_row[kBwdWaves][kBwdTokens][kMaxE + 16];
  __shared__ int s_e[kBwdWaves][kBwdTokens][kMaxK];
  __shared__ float s_v[kBwdWaves][kBwdTokens][kMaxK];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tok = lane >> 4, j = lane & 15;
  const long long t0 = (static_cast<long long>(blockIdx.x) * kBwdWaves + wave) * kBwdTokens;
  if (t0 >= T) return;
  const long long t = t0 + tok;
  const bool vec = (E & 3) == 0;
  float(*row)[kMaxE + 16] = s_row[wave];
  const bool live = t < T && j < k;
  int e = live ? idx[t * k + j] : -1;
  if (e >= E) e = -1;                              // no expert of this layer: no gradient
  const float l = e >= 0 ? clean_logit(logits[t * E + e]) : -INFINITY;
  const float dg = e >= 0 ? dgate[t * k + j] * scale : 0.f;
  float val, inner = 0.f;
  float pe[kMaxE / 16];                            // DENSE: scores of experts j + 16 i
  if constexpr (DENSE) {
#pragma unroll
    for (int i = 0; i < kBwdTokens; ++i) {
      if (t0 + i >= T) break;
      if (vec) {
        if (4 * lane < E) *reinterpret_cast<float4*>(&row[i][4 * lane]) = *reinterpret_cast<const float4*>(logits + (t0 + i) * E + 4 * lane);
      } else {
        for (int c = lane; c < E; c += 64) row[i][c] = logits[(t0 + i) * E + c];
      }
    }
    wave_lds_sync();
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMaxE / 16; ++i) {
      pe[i] = t < T && j + 16 * i < E ? clean_logit(row[tok][j + 16 * i]) : -INFINITY;
      m = fmaxf(m, pe[i]);
    }
    m = group_max16(m);
    m = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxE / 16; ++i) {
      pe[i] = j + 16 * i < E ? expf(pe[i] - m) : 0.f;
      sum += pe[i];
    }
    sum = group_sum16(sum);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < kMaxE / 16; ++i) pe[i] *= inv;
    val = expf(l - m) * inv * dg;
    inner = group_sum16(val);
  } else if (renormalize) {
    // log sigmoid(l) = min(l, 0) - log(1 + exp(-|l|))
    const float w = score == MOE_SCORE_SIGMOID ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : l;
    float m = group_max16(w);
    m = m == -INFINITY ? 0.f : m;
    const float ex = l == -INFINITY ? 0.f : expf(w - m);
    const float sum = group_sum16(ex);
    const float g = sum > 0.f ? ex / sum : 0.f;
    val = g * (dg - group_sum16(g * dg));
    if (score == MOE_SCORE_SIGMOID) val *= 1.f / (1.f + expf(l));
  } else {
    const float ex = expf(-fabsf(l));              // s (1 - s) = x / (1 + x)^2 with x = exp(-|l|)
    val = ex / ((1.f + ex) * (1.f + ex)) * dg;
  }
  // a repeated expert gets the sum of its slots, in slot order
  s_e[wave][tok][j] = e;
  s_v[wave][tok][j] = val;
  wave_lds_sync();
  float total = 0.f;
  for (int i = 0; i < k; ++i) total += s_e[wave][tok][i] == e ? s_v[wave][tok][i] : 0.f;
#pragma unroll
  for (int i = 0; i < kMaxE / 16; ++i)
    if (j + 16 * i < E) row[tok][j + 16 * i] = DENSE ? -pe[i] * inner : 0.f;
  wave_lds_sync();
  const float base = e >= 0 ? row[tok][e] : 0.f;
  wave_lds_sync();
  if (e >= 0) row[tok][e] = base + total;
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < kBwdTokens; ++i) {
    if (t0 + i >= T) break;
    if (vec) {
      if (4 * lane < E) *reinterpret_cast<float4*>(dlogits + (t0 + i) * E + 4 * lane) = *reinterpret_cast<const float4*>(&row[i][4 * lane]);
    } else {
      for (int c = lane; c < E; c += 64) dlogits[(t0 + i) * E + c] = row[i][c];
    }
  }
}

// Bytes of the block counts, and with the softmax's maximum and sum of every token behind them.
size_t hist_bytes(int T, int E) {
  return (static_cast<size_t>(T) + kRouteBlock - 1) / kRouteBlock * E * sizeof(int32_t) / 16 * 16 + 16;
}

int check_scored(int T, int E, int k, int score, float scale) {
  if (int st = check_layer_shape(T, E, k)) return st;
  // 16 lanes per token, in launches of fewer than 2^32 threads
  MOE_REQUIRE(T <= (1 << 28) - 64, MOE_ERR_UNSUPPORTED, "T must be at most 2^28 - 64 (got %d)", T);
  MOE_REQUIRE(score == MOE_SCORE_SIGMOID || score == MOE_SCORE_SOFTMAX, MOE_ERR_INVALID_ARG,
              "score must be MOE_SCORE_SIGMOID or MOE_SCORE_SOFTMAX (got %d)", score);
  MOE_REQUIRE(std::isfinite(scale), MOE_ERR_INVALID_ARG, "the gates' scale must be finite");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_route_scored_workspace_bytes(int T, int E, int k) {
  (void)k;
  if (T <= kRouteBlock || E < 1) return 0;
  return hist_bytes(T, E) + static_cast<size_t>(T) * sizeof(float2);
}

extern "C" int moe_route_scored(const float* logits, const float* bias, int T, int E, int k, int score, int n_group,
                                int topk_group, int group_top, int renormalize, float scale, int32_t* topk_idx,
                                float* topk_gate, float* scores, int32_t* counts, int32_t* offsets,
                                int32_t* offsets_pad, int pad, int32_t* dest, int32_t* row_token, void* ws,
                                size_t ws_bytes, void* stream) {
  if (int st = check_scored(T, E, k, score, scale)) return st;
  MOE_REQUIRE(n_group >= 1 && E % n_group == 0, MOE_ERR_UNSUPPORTED, "n_group must divide E (got %d, E = %d)", n_group, E);
  MOE_REQUIRE(topk_group >= 1 && topk_group <= n_group, MOE_ERR_UNSUPPORTED,
              "topk_group must be in [1, n_group] (got %d of %d)", topk_group, n_group);
  MOE_REQUIRE(group_top == 1 || group_top == 2, MOE_ERR_UNSUPPORTED, "group_top must be 1 or 2 (got %d)", group_top);
  MOE_REQUIRE(k <= topk_group * (E / n_group), MOE_ERR_UNSUPPORTED,
              "k = %d exceeds the %d experts of the chosen groups", k, topk_group * (E / n_group));
  MOE_CHECK_PTR(logits); MOE_CHECK_PTR(topk_idx); MOE_CHECK_PTR(topk_gate);
  MOE_CHECK_PTR(counts); MOE_CHECK_PTR(offsets); MOE_CHECK_PTR(dest);
  MOE_CHECK_ALIGN(logits); MOE_CHECK_ALIGN(topk_idx); MOE_CHECK_ALIGN(topk_gate);
  MOE_CHECK_ALIGN(counts); MOE_CHECK_ALIGN(offsets); MOE_CHECK_ALIGN(dest);
  if (bias) MOE_CHECK_ALIGN(bias);
  if (scores) MOE_CHECK_ALIGN(scores);
  if (offsets_pad) { MOE_CHECK_ALIGN(offsets_pad); MOE_REQUIRE(pad >= 1, MOE_ERR_INVALID_ARG, "pad must be >= 1"); }
  if (row_token) MOE_CHECK_ALIGN(row_token);
  const size_t need = moe_route_scored_workspace_bytes(T, E, k);
  MOE_REQUIRE(need == 0 || (ws != nullptr && ws_bytes >= need), MOE_ERR_WORKSPACE, "route workspace: need %zu bytes", need);
  MOE_CHECK_ALIGN(ws);
  const ScoredArgs a{logits, bias, T, E, k, score, n_group, topk_group, group_top, renormalize, scale};
  const MetaOut out{counts, offsets, offsets_pad, pad, dest, row_token};
  int32_t* hist = static_cast<int32_t*>(ws);
  hipStream_t s = as_stream(stream);
  if (T <= kRouteBlock) {
    route_scored_local<true><<<1, 1024, 0, s>>>(a, topk_idx, topk_gate, scores, nullptr, hist, out);
    return check_launch("route_scored_local");
  }
  const int nb = (T + kRouteBlock - 1) / kRouteBlock;
  const long long n = static_cast<long long>(T) * k;
  float2* sums = score == MOE_SCORE_SOFTMAX && !renormalize
                     ? reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + hist_bytes(T, E))
                     : nullptr;
  // four tokens per wave where every group of experts is 1, 2, 4 .. whole lanes of it, else one
  const int pl = E > 128 ? 16 : E > 64 ? 8 : 4, per_group = E / n_group;
  const bool quad = topk_group == n_group || (per_group % pl == 0 && (per_group / pl & (per_group / pl - 1)) == 0);
  const int chosen = quad ? 4 * kQuadWaves : kChooseWaves * kChooseTokens;
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(T) + chosen - 1) / chosen);
  const size_t lds = static_cast<size_t>(kQuadWaves) * std::min(pl, k) * 64 * sizeof(double);
  if (!quad) route_scored_choose<<<grid, 64 * kChooseWaves, 0, s>>>(a, topk_idx, sums);
  else if (pl == 16) route_scored_choose_quad<16><<<grid, 64 * kQuadWaves, lds, s>>>(a, topk_idx, sums);
  else if (pl == 8) route_scored_choose_quad<8><<<grid, 64 * kQuadWaves, lds, s>>>(a, topk_idx, sums);
  else route_scored_choose_quad<4><<<grid, 64 * kQuadWaves, lds, s>>>(a, topk_idx, sums);
  if (int st = check_launch("route_scored_choose")) return st;
  route_scored_local<false><<<nb, kLocalThreads, 0, s>>>(a, topk_idx, topk_gate, scores, sums, hist, out);
  if (int st = check_launch("route_scored_local")) return st;
  route_scored_scan<<<(E + 3) / 4, 256, 0, s>>>(hist, nb, E, counts);
  if (int st = check_launch("route_scored_scan")) return st;
  constexpr int per = kFinalThreads * kFinalItems;
  route_scored_finalize<<<static_cast<unsigned>((n + per - 1) / per), kFinalThreads, 0, s>>>(topk_idx, hist, nb, n, k, E,
                                                                                          out);
  return check_launch("route_scored_finalize");
}

extern "C" int moe_route_scored_bwd(const float* logits, const int32_t* topk_idx, const float* d_gate, int T, int E,
                                    int k, int score, int renormalize, float scale, float* d_logits, void* stream) {
  if (int st = check_scored(T, E, k, score, scale)) return st;
  MOE_CHECK_PTR(logits); MOE_CHECK_PTR(topk_idx); MOE_CHECK_PTR(d_gate); MOE_CHECK_PTR(d_logits);
  MOE_CHECK_ALIGN(logits); MOE_CHECK_ALIGN(d_logits);
  constexpr int per = kBwdWaves * kBwdTokens;
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(T) + per - 1) / per);
  hipStream_t s = as_stream(stream);
  if (score == MOE_SCORE_SOFTMAX && !renormalize)
    route_scored_bwd_kernel<true><<<blocks, 64 * kBwdWaves, 0, s>>>(logits, topk_idx, d_gate, T, E, k, score, renormalize,
                                                                   scale, d_logits);
  else
    route_scored_bwd_kernel<false><<<blocks, 64 * kBwdWaves, 0, s>>>(logits, topk_idx, d_gate, T, E, k, score, renormalize,
                                                                    scale, d_logits);
  return check_launch("route_scored_bwd");
}
