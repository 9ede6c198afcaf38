// fg_route.hip -- the router of a mixture-of-experts layer: each token's k best
// experts from its router logits, their weights, and the logits' gradient.
//
// With l the token's logits and an expert eligible where l > -inf (a masked
// expert is -inf or NaN), the scores are
//
//     softmax   s_e = exp(l_e - max l) / sum_eligible exp(l_j - max l)
//     sigmoid   s_e = 1 / (1 + exp(-l_e))
//
// The experts are ranked by l_e, or by s_e + bias_e where a selection bias is
// given (both scores increase with l, so without one the logits themselves
// give the order, free of rounding in exp). Equal ranks go to the lower index.
// The weights are scale * s, or scale * s / (sum of the chosen s) when they
// are renormalised. The bias takes no part in the weights or the gradient.
//
// Gradient, for g_i = scale * dw_i on the chosen experts, 0 elsewhere:
//
//     softmax                  dl = s (g - <g, s>)
//     softmax, renormalised    dl = p (g - <g, p>),  p = s / sum of the chosen s, chosen only
//     sigmoid                  dl = g s (1 - s)
//     sigmoid, renormalised    dl = (g - <g, p>) / (sum of the chosen s) * s (1 - s), chosen only
//
// 1 - s of a sigmoid is worked out from the logit, 1 / (1 + exp(l)): as a difference it
// keeps u / (1 - s) of relative error (u = 2^-24), 1% at a logit of 12, and is 0 from 17 on.
//
// A group of L = 64 or 16 lanes holds a token: lane i of it has experts
// [i * V, (i + 1) * V). Each of the k rounds is a maximum over the group's 32-bit
// order keys on the DPP path, a ballot that finds the lowest lane holding it, and
// that lane clearing its lowest such key and noting the choice in LDS; no
// barrier, since a group lies within one wave. All sums are fp32 in a fixed order.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fg.h"
#include "fg_device.hpp"
#include "fg_wave.hpp"

namespace {

using namespace fg;

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr int kThreads = 256;
// Tokens from which on four share a wave: with few tokens the wave's longer chain
// shows, with many its fewer instructions. One token / four a wave, k 8, fp32 softmax
// in a graph: E 64, T 1024 3.3 / 3.8, 4096 3.9 / 3.9, 16384 7.8 / 5.6 us, its gradient
// 5.7 / 5.0. E 128, T 4096 4.5 / 4.5, 16384 9.5 / 7.2; sigmoid with a bias 9.4 / 9.2 there
// but 6.0 / 6.8 at 8192, so twice the tokens. Above 128 experts one token a wave always:
// with E 256 and T 16384 softmax would gain (12.9 / 11.0) but sigmoid with a bias (13.6 /
// 15.0) and the gradient (12.3 / 15.0) lose.
constexpr int kPackTokens = 8192;        // E <= 64
constexpr int kPackTokensWide = 16384;   // E <= 128

// V consecutive elements of a row move in pieces of up to 16 bytes where V
// divides E (a lane then has V experts or none, and pieces are aligned).
template <class R, int V>
struct Pieces {
  static constexpr int kBytes = V * R::kBytes < 16 ? V * R::kBytes : 16;
  static constexpr int kEach = kBytes / R::kBytes, kCount = V / kEach;
  struct alignas(kBytes) Piece {
    uint8_t b[kBytes];
  };
};

// V consecutive logits from expert e0 of a row; experts past E and NaN as -inf.
template <class R, int V>
__device__ __forceinline__ void load_logits(const void* logits, long row, int E, int e0, float* l) {
  using P = Pieces<R, V>;
  if (E % V == 0) {
    const int at = e0 < E ? e0 : E - V;
    const char* src = (const char*)logits + (row * E + at) * R::kBytes;
    if constexpr (P::kBytes == 16) {
      u32x4 raw[P::kCount];
#pragma unroll
      for (int c = 0; c < P::kCount; ++c) raw[c] = ((const u32x4*)src)[c];
#pragma unroll
      for (int c = 0; c < P::kCount; ++c) R::unpack(raw[c], l + c * R::kPer16);
    } else {
      const typename P::Piece raw = *(const typename P::Piece*)src;
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = R::load1(&raw, i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // loads are not predicated: past the row's end its last logit is read and dropped
      const int e = e0 + i < E ? e0 + i : E - 1;
      l[i] = R::load1(logits, row * E + e);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = e0 + i < E && l[i] > -INFINITY ? l[i] : -INFINITY;
}

template <class R, int V>
__device__ __forceinline__ void store_row(void* out, long row, int E, int e0, const float* v) {
  using P = Pieces<R, V>;
  if (E % V == 0) {
    char* dst = (char*)out + (row * E + e0) * R::kBytes;
    if (e0 >= E) return;
    if constexpr (P::kBytes == 16) {
#pragma unroll
      for (int c = 0; c < P::kCount; ++c) ((u32x4*)dst)[c] = R::pack(v + c * R::kPer16);
    } else {
      typename P::Piece raw;
#pragma unroll
      for (int i = 0; i < V; ++i) R::store1(&raw, i, v[i]);
      *(typename P::Piece*)dst = raw;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < E) R::store1(out, row * E + e0 + i, v[i]);
  }
}

// The largest of the group's logits (-inf if nothing is eligible).
template <int L, int V>
__device__ __forceinline__ float top_logit(const float* l) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
  const uint32_t u = group_max_u32<L>(order_key(m));
  return __uint_as_float((u >> 31) ? (u & 0x7fffffffu) : ~u);
}

// A score before its division: exp(l - top) or the whole sigmoid; 0 for l = -inf.
__device__ __forceinline__ float raw_score(float l, float top, int softmax) {
  if (!(l > -INFINITY)) return 0.0f;
  return softmax ? expf(l - top) : 1.0f / (1.0f + expf(-l));
}

// 1 - 1 / (1 + exp(-l)), to a few u of itself for either sign of l.
__device__ __forceinline__ float sigmoid_complement(float l) { return 1.0f / (1.0f + expf(l)); }

// Scores of the lane's V logits.
template <int L, int V>
__device__ __forceinline__ void scores(const float* l, int softmax, float* s) {
  const float top = softmax ? top_logit<L, V>(l) : 0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    s[i] = raw_score(l[i], top, softmax);
    sum += s[i];
  }
  if (softmax) {
    sum = group_sum<L>(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = s[i] == 0.0f ? 0.0f : s[i] / sum;   // a row with nothing eligible has sum 0
  }
}

// BIAS: the ranks are scores + bias, so every expert's score is worked out first.
// Without one the logits are ranked, and only the chosen are divided (softmax) or
// have a score at all (sigmoid).
template <class R, int L, int V, bool BIAS>
__global__ __launch_bounds__(kThreads) void route_topk(const void* __restrict__ logits,
                                                       const float* __restrict__ bias, int32_t* __restrict__ ids,
                                                       float* __restrict__ w, int T, int E, int k, int softmax,
                                                       int renorm, float scale) {
  __shared__ int32_t best_id[kThreads / L][kMaxTopK];
  __shared__ float best_v[kThreads / L][kMaxTopK];   // the choice's score (BIAS) or logit
  const int group = threadIdx.x / L, lane = threadIdx.x % L;
  const long t = (long)blockIdx.x * (kThreads / L) + group;
  const long row = t < T ? t : T - 1L;   // groups past the last token repeat it and store nothing
  float l[V], s[V];
  uint32_t key[V];
  load_logits<R, V>(logits, row, E, lane * V, l);
  float top = 0.0f, total = 1.0f;
  if (BIAS) {
    float b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = bias[lane * V + i < E ? lane * V + i : E - 1];
    scores<L, V>(l, softmax, s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float rank = l[i] > -INFINITY ? s[i] + b[i] : l[i];
      key[i] = rank > -INFINITY ? order_key(rank) : 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = l[i];
      key[i] = l[i] > -INFINITY ? order_key(l[i]) : 0u;
    }
    if (softmax) {
      top = top_logit<L, V>(l);
      if (!renorm) {   // renormalised, the sum over all experts cancels
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum += raw_score(l[i], top, 1);
        total = group_sum<L>(sum);
      }
    }
  }
  for (int j = lane; j < k; j += L) {
    best_id[group][j] = -1;
    best_v[group][j] = BIAS ? 0.0f : -INFINITY;
  }
  for (int j = 0; j < k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = umax(m, key[i]);
    const uint32_t best = group_max_u32<L>(m);
    // the group's lowest lane with the best key; its lowest expert among equals
    unsigned long long same = __ballot(m == best);
    if (L == 16) same = (same >> (threadIdx.x & 48)) & 0xffffu;
    if (__builtin_ctzll(same | (1ull << 63)) == lane && best != 0u) {
      int at = 0;
      float v = 0.0f;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) {
        at = key[i] == best ? i : at;
        v = key[i] == best ? s[i] : v;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = i == at ? 0u : key[i];
      best_id[group][j] = lane * V + at;
      best_v[group][j] = v;
    }
  }
  // the group's own LDS writes, in order within its wave
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  constexpr int kEach = (kMaxTopK + L - 1) / L;   // choices per lane
  float c[kEach], sum = 0.0f;
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int j = lane + u * L;
    c[u] = 0.0f;
    if (j < k) {
      const float v = best_v[group][j];
      c[u] = BIAS ? v : raw_score(v, top, softmax);
      if (!BIAS && softmax && !renorm) c[u] = c[u] == 0.0f ? 0.0f : c[u] / total;
    }
    sum += c[u];
  }
  if (renorm) sum = group_sum<L>(sum);
  if (t >= T) return;
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int j = lane + u * L;
    if (j < k) {
      ids[t * k + j] = best_id[group][j];
      w[t * k + j] = (renorm ? (sum > 0.0f ? c[u] / sum : 0.0f) : c[u]) * scale;
    }
  }
}

template <class R, int L, int V>
__global__ __launch_bounds__(kThreads) void route_topk_grad(const void* __restrict__ logits,
                                                            const int32_t* __restrict__ ids,
                                                            const float* __restrict__ dw,
                                                            void* __restrict__ dlogits, int T, int E, int k,
                                                            int softmax, int renorm, float scale) {
  const int group = threadIdx.x / L, lane = threadIdx.x % L;
  const long t = (long)blockIdx.x * (kThreads / L) + group;
  const long row = t < T ? t : T - 1L;
  float l[V], s[V], g[V];
  bool hit[V];
  load_logits<R, V>(logits, row, E, lane * V, l);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    g[i] = 0.0f;
    hit[i] = false;
  }
#pragma unroll 8
  for (int j = 0; j < k; ++j) {
    const int at = ids[row * k + j] - lane * V;
    const float ge = dw[row * k + j] * scale;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      g[i] += at == i ? ge : 0.0f;
      hit[i] = hit[i] || at == i;
    }
  }
  scores<L, V>(l, softmax, s);
  float total = 1.0f;
  if (renorm) {   // shares p of the chosen scores; g - <g, p>
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) c += hit[i] ? s[i] : 0.0f;
    total = group_sum<L>(c);
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) d += hit[i] && total > 0.0f ? g[i] * (s[i] / total) : 0.0f;
    d = group_sum<L>(d);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = hit[i] ? g[i] - d : 0.0f;
  } else if (softmax) {
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) d += g[i] * s[i];
    d = group_sum<L>(d);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] -= d;
  }
  if (t >= T) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float out = 0.0f;
    if (total > 0.0f) out = g[i] * (renorm ? s[i] / total : s[i]);
    g[i] = softmax ? out : out * sigmoid_complement(l[i]);
  }
  store_row<R, V>(dlogits, t, E, lane * V, g);
}

int check(const void* logits, int dtype, int T, int E, int k, int score) {
  if (T < 0 || E < 1 || E > kMaxExperts || k < 1 || k > kMaxTopK || k > E) return FG_EINVAL;
  if ((dtype != FG_BF16 && dtype != FG_FP32) || (score != FG_SCORE_SOFTMAX && score != FG_SCORE_SIGMOID))
    return FG_EINVAL;
  if (T == 0) return FG_OK;
  if (!logits || !aligned(logits, 16)) return FG_EINVAL;
  return FG_OK;
}

template <class R, int L, int V, class... Args>
void launch_v(bool grad, int T, hipStream_t s, const void* logits, const void* b, void* ids, void* w, Args... a) {
  const dim3 grid((unsigned)((T + kThreads / L - 1L) / (kThreads / L))), block(kThreads);
  if (grad)
    hipLaunchKernelGGL((route_topk_grad<R, L, V>), grid, block, 0, s, logits, (const int32_t*)b, (const float*)ids, w, T, a...);
  else if (b)
    hipLaunchKernelGGL((route_topk<R, L, V, true>), grid, block, 0, s, logits, (const float*)b, (int32_t*)ids, (float*)w, T, a...);
  else
    hipLaunchKernelGGL((route_topk<R, L, V, false>), grid, block, 0, s, logits, (const float*)b, (int32_t*)ids, (float*)w, T, a...);
}

template <class R, class... Args>
void launch_e(int E, bool grad, int T, Args... a) {
  if (T >= kPackTokens && E <= 64) launch_v<R, 16, 4>(grad, T, a...);
  else if (T >= kPackTokensWide && E > 64 && E <= 128) launch_v<R, 16, 8>(grad, T, a...);
  else if (E <= 64) launch_v<R, 64, 1>(grad, T, a...);
  else if (E <= 128) launch_v<R, 64, 2>(grad, T, a...);
  else if (E <= 256) launch_v<R, 64, 4>(grad, T, a...);
  else if (E <= 512) launch_v<R, 64, 8>(grad, T, a...);
  else launch_v<R, 64, 16>(grad, T, a...);
}

int route(bool grad, const void* logits, int dtype, const void* b, void* ids, void* w, int T, int E, int k,
          int score, int renorm, float scale, hipStream_t stream) {
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  const int softmax = score == FG_SCORE_SOFTMAX, norm = renorm != 0;
  if (dtype == FG_BF16)
    launch_e<RowBf16>(E, grad, T, stream, logits, b, ids, w, E, k, softmax, norm, scale);
  else
    launch_e<RowF32>(E, grad, T, stream, logits, b, ids, w, E, k, softmax, norm, scale);
  return hipGetLastError() == hipSuccess ? FG_OK : FG_ELAUNCH;
}

}  // namespace

extern "C" {

int fg_route_topk(const void* logits, int dtype, const float* bias, int32_t* ids, float* w, int T, int E, int k,
                  int score, int renorm, float scale, hipStream_t stream) {
  const int rc = check(logits, dtype, T, E, k, score);
  if (rc != FG_OK || T == 0) return rc;
  if (!ids || !w || !aligned(ids, 4) || !aligned(w, 4) || (bias && !aligned(bias, 4))) return FG_EINVAL;
  return route(false, logits, dtype, bias, ids, w, T, E, k, score, renorm, scale, stream);
}

int fg_route_topk_grad(const void* logits, int dtype, const int32_t* ids, const float* dw, void* dlogits, int T,
                       int E, int k, int score, int renorm, float scale, hipStream_t stream) {
  const int rc = check(logits, dtype, T, E, k, score);
  if (rc != FG_OK || T == 0) return rc;
  if (!ids || !dw || !dlogits || !aligned(ids, 4) || !aligned(dw, 4) || !aligned(dlogits, 16))
    return FG_EINVAL;
  return route(true, logits, dtype, ids, const_cast<float*>(dw), dlogits, T, E, k, score, renorm, scale, stream);
}

}  // extern "C"
