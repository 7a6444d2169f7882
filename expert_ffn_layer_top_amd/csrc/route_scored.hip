// The scored router: a score for every expert (the sigmoid of its logit, or the softmax over all of
// them), a bias for balance that is added for the choice alone, the best groups of experts, the k
// best experts of those, and gates from the unbiased scores; its gradient.
//
//   s[e] = sigmoid(l[e]) or exp(l[e] - max) / sum                 (64 bits)
//   c[e] = s[e] + bias[e]                                         (64 bits; -inf where l[e] is -inf or NaN)
//   v[g] = sum of the group_top largest c of group g              (E / n_group experts each)
//   choice: the topk_group groups of largest v, of their experts the k of largest c (of largest l
//   where there is no bias), ties to the lower index; gate = scale * s / (sum of the chosen s)
//
// The choice is made in 64 bits: with 256 experts a batch of 32768 tokens has a handful whose k-th and
// next value differ by less than one fp32 rounding, and a choice that depends on how fp32 rounds an
// exponential would differ between implementations and moves every later row of two experts.
#include <cmath>

#include "common.h"
#include "route_meta.h"

namespace moe {
namespace {

constexpr int kWaveTokens = 4;                 // tokens of a wave, one after the other
constexpr int kBlockWaves = kRouteBlock / kWaveTokens;
constexpr int kQ = kMaxE / 64;                 // experts of a lane: lane + 64 q

// A logit as the router reads it: NaN counts as -inf (an absent expert), +inf as the largest float.
__device__ __forceinline__ float clean_logit(float l) {
  return l != l ? -INFINITY : fminf(l, 3.4028234663852886e38f);
}

// Order-preserving map of a double to uint64 (larger value -> larger key, -0 as +0, never 0).
__device__ __forceinline__ unsigned long long double_key(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return b < 0 ? ~static_cast<unsigned long long>(b) : static_cast<unsigned long long>(b) | 0x8000000000000000ull;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
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

// One wave per token.  Returns, in lane j < k, the j-th chosen expert and its gate.
__device__ __forceinline__ void route_token(const ScoredArgs& a, long long t, int lane, double* s_choice,
                                            float* __restrict__ scores, int& my_e, float& my_gate) {
  const float* row = a.logits + t * a.E;
  float l[kQ];
  double p[kQ];
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const int e = lane + 64 * q;
    l[q] = e < a.E ? clean_logit(row[e]) : -INFINITY;
    m = fmaxf(m, l[q]);
  }
  if (a.score == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int q = 0; q < kQ; ++q) p[q] = 1.0 / (1.0 + exp(-static_cast<double>(l[q])));
  } else {
    m = wave_max(m);
    const double md = m == -INFINITY ? 0.0 : static_cast<double>(m);
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      p[q] = exp(static_cast<double>(l[q]) - md);
      sum += p[q];
    }
    sum = wave_sum_f64(sum);
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int q = 0; q < kQ; ++q) p[q] *= inv;
  }
  if (scores != nullptr) {
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      if (lane + 64 * q < a.E) scores[t * a.E + lane + 64 * q] = static_cast<float>(p[q]);
  }
  double c[kQ];
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const int e = lane + 64 * q;
    c[q] = a.bias != nullptr && e < a.E ? p[q] + static_cast<double>(a.bias[e]) : p[q];
    if (l[q] == -INFINITY || c[q] != c[q]) c[q] = -INFINITY;
  }
  // which of this lane's experts lie in a chosen group
  unsigned inside = (1u << kQ) - 1u;
  if (a.topk_group < a.n_group) {
    const int per = a.E / a.n_group;
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      if (lane + 64 * q < a.E) s_choice[lane + 64 * q] = c[q];
    wave_lds_sync();
    unsigned long long gkey[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const int g = lane + 64 * q;
      gkey[q] = 0ull;
      if (g < a.n_group) {
        double b0 = -INFINITY, b1 = -INFINITY;
        for (int i = 0; i < per; ++i) {
          const double v = s_choice[g * per + i];
          b1 = v > b0 ? b0 : (v > b1 ? v : b1);
          b0 = v > b0 ? v : b0;
        }
        const double v = a.group_top == 1 || b1 == -INFINITY ? b0 : b0 + b1;
        gkey[q] = double_key(v);
      }
    }
    inside = 0u;
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
        if (lane + 64 * q >= g * per && lane + 64 * q < (g + 1) * per) inside |= 1u << q;
      }
    }
    wave_lds_sync();
  }
  unsigned long long key[kQ];
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const int e = lane + 64 * q;
    const double v = a.bias != nullptr ? c[q] : static_cast<double>(l[q]);
    key[q] = e < a.E && (inside >> q & 1u) ? double_key(v) : 0ull;
  }
  my_e = 0;
  double my_p = 0.0;
  for (int j = 0; j < a.k; ++j) {
    unsigned long long best = key[0];
#pragma unroll
    for (int q = 1; q < kQ; ++q) best = key[q] > best ? key[q] : best;
    best = wave_max_u64(best);
    int e = -1;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const unsigned long long hit = __ballot(key[q] == best);
      if (e < 0 && hit) e = 64 * q + __ffsll(static_cast<long long>(hit)) - 1;
    }
    e = __builtin_amdgcn_readfirstlane(e);
    double pe = p[0];
#pragma unroll
    for (int q = 1; q < kQ; ++q) pe = (e >> 6) == q ? p[q] : pe;
    pe = __shfl(pe, e & 63, 64);
    if (lane == j) { my_e = e; my_p = pe; }
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      if (lane + 64 * q == e) key[q] = 0ull;
  }
  double gate = my_p;
  if (a.renormalize) {
    const double sum = wave_sum_f64(my_p);
    gate = sum > 0.0 ? my_p / sum : 0.0;
  }
  my_gate = static_cast<float>(gate * static_cast<double>(a.scale));
}

// 64 tokens per block of 16 waves; the row metadata as the other router's first kernel leaves it.
__global__ __launch_bounds__(1024) void route_scored_local(ScoredArgs a, int32_t* __restrict__ topk_idx,
                                                           float* __restrict__ topk_gate, float* __restrict__ scores,
                                                           int32_t* __restrict__ local_rank,
                                                           int32_t* __restrict__ hist) {
  __shared__ unsigned long long s_mask[kMaxE];
  __shared__ int s_e[kRouteBlock][kMaxK];
  __shared__ double s_choice[kBlockWaves][kMaxE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const long long t0 = static_cast<long long>(blockIdx.x) * kRouteBlock;
  for (int e = tid; e < a.E; e += 1024) s_mask[e] = 0ull;
  __syncthreads();
  for (int i = 0; i < kWaveTokens; ++i) {
    const int tl = wave * kWaveTokens + i;
    const long long t = t0 + tl;
    if (t >= a.T) break;
    int e;
    float gate;
    route_token(a, t, lane, s_choice[wave], scores, e, gate);
    if (lane < a.k) {
      topk_idx[t * a.k + lane] = e;
      topk_gate[t * a.k + lane] = gate;
      s_e[tl][lane] = e;
      atomicOr(&s_mask[e], 1ull << tl);
    }
  }
  __syncthreads();
  for (int i = tid; i < kRouteBlock * a.k; i += 1024) {
    const int tl = i / a.k, j = i - tl * a.k;
    const long long t = t0 + tl;
    if (t < a.T) local_rank[t * a.k + j] = __popcll(s_mask[s_e[tl][j]] & ((1ull << tl) - 1ull));
  }
  for (int e = tid; e < a.E; e += 1024) hist[static_cast<long long>(blockIdx.x) * a.E + e] = __popcll(s_mask[e]);
}

// Gradient with the choice held fixed, one wave per token:
//   sigmoid  dl = s (1 - s) ds,  softmax  dl[e] = s[e] (ds[e] - sum s ds),  ds of the chosen experts from
//   the gates (renormalised: ds_j = (dg_j - sum g dg) / sum s), 0 elsewhere.
// Renormalised gates come from the chosen logits alone, in the log domain, so scores that underflow
// still give finite ratios; only the plain softmax needs (and has) a gradient at every expert.
__global__ __launch_bounds__(256) void route_scored_bwd_kernel(const float* __restrict__ logits,
                                                               const int32_t* __restrict__ idx,
                                                               const float* __restrict__ dgate, int T, int E, int k,
                                                               int score, int renormalize, float scale,
                                                               float* __restrict__ dlogits) {
  const long long t = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= T) return;
  int e_l = lane < k ? idx[t * k + lane] : -1;
  if (e_l >= E) e_l = -1;                          // no expert of this layer: no gradient
  const float l_l = e_l >= 0 ? clean_logit(logits[t * E + e_l]) : -INFINITY;
  const float dg = e_l >= 0 ? dgate[t * k + lane] * scale : 0.f;
  float val;                        // lane j: the gradient at the j-th chosen expert (plain softmax: p dg)
  float pe[kQ];                     // plain softmax: scores of experts lane + 64 q
  float inner = 0.f;
  const bool dense = score == MOE_SCORE_SOFTMAX && !renormalize;
  if (dense) {
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      pe[q] = lane + 64 * q < E ? clean_logit(logits[t * E + lane + 64 * q]) : -INFINITY;
      m = fmaxf(m, pe[q]);
    }
    m = wave_max(m);
    m = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      pe[q] = expf(pe[q] - m);
      sum += pe[q];
    }
    sum = wave_sum(sum);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int q = 0; q < kQ; ++q) pe[q] *= inv;
    val = expf(l_l - m) * inv * dg;
    inner = wave_sum(val);
  } else if (renormalize) {
    // log sigmoid(l) = min(l, 0) - log(1 + exp(-|l|))
    const float w = score == MOE_SCORE_SIGMOID ? fminf(l_l, 0.f) - log1pf(expf(-fabsf(l_l))) : l_l;
    float m = wave_max(w);
    m = m == -INFINITY ? 0.f : m;
    const float ex = l_l == -INFINITY ? 0.f : expf(w - m);
    const float sum = wave_sum(ex);
    const float g = sum > 0.f ? ex / sum : 0.f;
    val = g * (dg - wave_sum(g * dg));
    if (score == MOE_SCORE_SIGMOID) val *= 1.f / (1.f + expf(l_l));
  } else {
    const float ex = expf(-fabsf(l_l));            // s (1 - s) = e / (1 + e)^2 with e = exp(-|l|)
    val = ex / ((1.f + ex) * (1.f + ex)) * dg;
  }
  int ej[kMaxK];
  float vj[kMaxK];
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    ej[j] = __shfl(e_l, j, 64);
    vj[j] = __shfl(val, j, 64);
  }
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const int e = lane + 64 * q;
    if (e >= E) break;
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (j < k && ej[j] == e) v += vj[j];
    if (dense) v -= pe[q] * inner;
    dlogits[t * E + e] = v;
  }
}

int check_scored(int T, int E, int k, int score, float scale) {
  if (int st = check_layer_shape(T, E, k)) return st;
  MOE_REQUIRE(score == MOE_SCORE_SIGMOID || score == MOE_SCORE_SOFTMAX, MOE_ERR_INVALID_ARG,
              "score must be MOE_SCORE_SIGMOID or MOE_SCORE_SOFTMAX (got %d)", score);
  MOE_REQUIRE(std::isfinite(scale), MOE_ERR_INVALID_ARG, "the gates' scale must be finite");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

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
  const size_t need = moe_route_workspace_bytes(T, E, k);
  MOE_REQUIRE(ws != nullptr && ws_bytes >= need, MOE_ERR_WORKSPACE, "route workspace: need %zu bytes", need);
  MOE_CHECK_ALIGN(ws);
  const ScoredArgs a{logits, bias, T, E, k, score, n_group, topk_group, group_top, renormalize, scale};
  int32_t* hist = static_cast<int32_t*>(ws);
  hipStream_t s = as_stream(stream);
  route_scored_local<<<(T + kRouteBlock - 1) / kRouteBlock, 1024, 0, s>>>(a, topk_idx, topk_gate, scores, dest, hist);
  if (int st = check_launch("route_scored_local")) return st;
  return enqueue_route_metadata(topk_idx, T, E, k, counts, offsets, offsets_pad, pad, dest, row_token, hist, s);
}

extern "C" int moe_route_scored_bwd(const float* logits, const int32_t* topk_idx, const float* d_gate, int T, int E,
                                    int k, int score, int renormalize, float scale, float* d_logits, void* stream) {
  if (int st = check_scored(T, E, k, score, scale)) return st;
  MOE_CHECK_PTR(logits); MOE_CHECK_PTR(topk_idx); MOE_CHECK_PTR(d_gate); MOE_CHECK_PTR(d_logits);
  route_scored_bwd_kernel<<<static_cast<unsigned>((static_cast<long long>(T) + 3) / 4), 256, 0, as_stream(stream)>>>(
      logits, topk_idx, d_gate, T, E, k, score, renormalize, scale, d_logits);
  return check_launch("route_scored_bwd");
}
