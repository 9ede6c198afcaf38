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
// One wave holds one token: lane i has experts [i * V, (i + 1) * V). Each of
// the k rounds is a wave-wide maximum over 32-bit order keys on the DPP path,
// a ballot that finds the lowest lane holding it, and that lane clearing its
// lowest such key; no LDS and no barrier. All sums are fp32 in a fixed order.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fg.h"
#include "fg_device.hpp"
#include "fg_wave.hpp"

namespace {

using namespace fg;

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr int kWaves = 4;   // tokens per workgroup

// Lane's V logits of one row (NaN and everything past E as -inf).
template <class R, int V>
__device__ __forceinline__ void load_logits(const void* logits, long row, int E, int lane, float* l) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    float v = -INFINITY;
    if (e < E) v = R::load1(logits, row * E + e);
    l[i] = v > -INFINITY ? v : -INFINITY;
  }
}

// Scores of the lane's V logits.
template <int V>
__device__ __forceinline__ void scores(const float* l, int softmax, float* s) {
  if (softmax) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = umax(m, order_key(l[i]));
    m = wave_max_u32(m);
    const float top = __uint_as_float((m >> 31) ? (m & 0x7fffffffu) : ~m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = l[i] > -INFINITY ? expf(l[i] - top) : 0.0f;
      sum += s[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = s[i] == 0.0f ? 0.0f : s[i] / sum;   // a row with nothing eligible has sum 0
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = l[i] > -INFINITY ? 1.0f / (1.0f + expf(-l[i])) : 0.0f;
  }
}

template <class R, int V>
__global__ __launch_bounds__(64 * kWaves) void route_topk(const void* __restrict__ logits,
                                                          const float* __restrict__ bias,
                                                          int32_t* __restrict__ ids, float* __restrict__ w,
                                                          int T, int E, int k, int softmax, int renorm,
                                                          float scale) {
  const long t = (long)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= T) return;
  const int lane = threadIdx.x & 63;
  float l[V], s[V];
  uint32_t key[V];
  load_logits<R, V>(logits, t, E, lane, l);
  scores<V>(l, softmax, s);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    float rank = l[i];
    if (bias && e < E && l[i] > -INFINITY) rank = s[i] + bias[e];
    key[i] = rank > -INFINITY ? order_key(rank) : 0u;
  }
  int id = -1;        // lane j ends with the j-th choice
  float chosen = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = umax(m, key[i]);
    const uint32_t best = wave_max_u32(m);
    if (best == 0u) break;   // nothing eligible is left
    const int lead = __builtin_ctzll(__ballot(m == best));
    int at = 0;
    float sc = 0.0f;
    bool open = lane == lead;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (open && key[i] == best) {
        key[i] = 0u;
        at = i;
        sc = s[i];
        open = false;
      }
    }
    const int e = lead * V + __builtin_amdgcn_readlane(at, lead);
    const float se = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(sc), lead));
    if (lane == j) {
      id = e;
      chosen = se;
    }
  }
  if (renorm) {
    const float sum = wave_sum(chosen);
    chosen = sum > 0.0f ? chosen / sum : 0.0f;
  }
  if (lane < k) {
    ids[t * k + lane] = id;
    w[t * k + lane] = chosen * scale;
  }
}

template <class R, int V>
__global__ __launch_bounds__(64 * kWaves) void route_topk_grad(const void* __restrict__ logits,
                                                               const int32_t* __restrict__ ids,
                                                               const float* __restrict__ dw,
                                                               void* __restrict__ dlogits, int T, int E, int k,
                                                               int softmax, int renorm, float scale) {
  const long t = (long)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= T) return;
  const int lane = threadIdx.x & 63;
  float l[V], s[V], g[V];
  bool hit[V];
  load_logits<R, V>(logits, t, E, lane, l);
  scores<V>(l, softmax, s);
  const int my_id = lane < k ? ids[t * k + lane] : -1;
  const float my_g = lane < k ? dw[t * k + lane] * scale : 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    g[i] = 0.0f;
    hit[i] = false;
  }
  for (int j = 0; j < k; ++j) {
    const int e = __builtin_amdgcn_readlane(my_id, j);
    const float ge = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(my_g), j));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (e == lane * V + i) {
        g[i] += ge;
        hit[i] = true;
      }
    }
  }
  float total = 1.0f;
  if (renorm) {   // shares p of the chosen scores; g - <g, p>
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) c += hit[i] ? s[i] : 0.0f;
    total = wave_sum(c);
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) d += hit[i] && total > 0.0f ? g[i] * (s[i] / total) : 0.0f;
    d = wave_sum(d);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = hit[i] ? g[i] - d : 0.0f;
  } else if (softmax) {
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) d += g[i] * s[i];
    d = wave_sum(d);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] -= d;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    float out = 0.0f;
    if (total > 0.0f) out = g[i] * (renorm ? s[i] / total : s[i]);
    if (!softmax) out *= 1.0f - s[i];
    if (e < E) R::store1(dlogits, t * E + e, out);
  }
}

int check(const void* logits, int dtype, int T, int E, int k, int score) {
  if (T < 0 || E < 1 || E > kMaxExperts || k < 1 || k > kMaxTopK || k > E) return FG_EINVAL;
  if ((dtype != FG_BF16 && dtype != FG_FP32) || (score != FG_SCORE_SOFTMAX && score != FG_SCORE_SIGMOID))
    return FG_EINVAL;
  if (T == 0) return FG_OK;
  if (!logits || !aligned(logits, dtype == FG_BF16 ? 2 : 4)) return FG_EINVAL;
  return FG_OK;
}

template <class R, int V, class... Args>
void launch_v(bool grad, int T, hipStream_t s, const void* logits, const void* b, void* ids, void* w, Args... a) {
  const dim3 grid((unsigned)((T + kWaves - 1L) / kWaves)), block(64 * kWaves);
  if (grad)
    hipLaunchKernelGGL((route_topk_grad<R, V>), grid, block, 0, s, logits, (const int32_t*)b, (const float*)ids, w, T, a...);
  else
    hipLaunchKernelGGL((route_topk<R, V>), grid, block, 0, s, logits, (const float*)b, (int32_t*)ids, (float*)w, T, a...);
}

template <class R, class... Args>
void launch_e(int E, Args... a) {
  if (E <= 64) launch_v<R, 1>(a...);
  else if (E <= 128) launch_v<R, 2>(a...);
  else if (E <= 256) launch_v<R, 4>(a...);
  else if (E <= 512) launch_v<R, 8>(a...);
  else launch_v<R, 16>(a...);
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
  if (!ids || !dw || !dlogits || !aligned(ids, 4) || !aligned(dw, 4) || !aligned(dlogits, dtype == FG_BF16 ? 2 : 4))
    return FG_EINVAL;
  return route(true, logits, dtype, ids, const_cast<float*>(dw), dlogits, T, E, k, score, renorm, scale, stream);
}

}  // extern "C"
