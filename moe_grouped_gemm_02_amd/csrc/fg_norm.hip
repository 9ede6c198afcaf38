// fg_norm.hip -- the norms around a block, with the block's gate and the residual scales:
//
//     u = y / sqrt(mean y^2 + eps) post          (y itself without post)
//     r = alpha x + beta gate u                  (x itself without y)
//     h = r / sqrt(mean r^2 + eps) pre           of r before its rounding to x's type
//
// with the gate per channel, per token or none, and h in x's type, as the E4M3 product's
// operand (1x128 scales) or as the 8-bit integer product's (one scale per row). And the
// gradient: with rh = r rx, yh = y ry (rx, ry the reciprocal roots), g the gate,
//
//     dR = dr + rx (z - rh mean(z rh)),  z = dh pre;          dx = alpha dR
//     dy = ry (v - yh mean(v yh)),       v = beta g post dR   (dy = v without post)
//     dpre = sum_t dh rh,   S = sum_t dR yh (times the token's gate)
//     dpost = beta g S,     dgate = beta post S  per channel, beta sum_n dR yh post per token
//
// Everything is fp32 between the loads and the stores. All is bound by memory traffic:
// a workgroup holds a row in registers (units of 8 elements a lane) through its sums and
// walks the rows with its columns' weights kept in registers too -- the post norm's
// weight, the channel's gate and beta fold into one -- so each row is read once, and the
// gradient's column sums S and sum dh rh stay in registers until a workgroup's rows are
// done; a second kernel adds the workgroups' sums in a fixed order.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fg.h"
#include "fg_device.hpp"
#include "fg_int8_quot.hpp"

namespace {

using namespace fg;

constexpr int kMaxCols = 16384;   // 1024 threads of 2 units
constexpr int kCUs = 256;

struct NormArgs {
  const void *x, *y;
  const float *pre, *post, *gate;
  void *r, *h;
  float* s;
  int T, N, gate_kind, out;
  float alpha, beta, eps, inv_n;
};

// A row (or a vector of weights) of n bytes as a buffer: lanes past its end load zeros,
// which add nothing to any sum, and store nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void* base, long byte, int n) {
  return __builtin_amdgcn_make_buffer_rsrc((char*)base + byte, 0, n, 0x20000);
}
// Unit i of it: 8 elements.
template <class R>
__device__ __forceinline__ void load8(__amdgpu_buffer_rsrc_t row, int i, float* f) {
#pragma unroll
  for (int c = 0; c < 8 / R::kPer16; ++c)
    R::unpack(__builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(row, i * 8 * R::kBytes + 16 * c, 0, 0)),
              f + c * R::kPer16);
}
template <class R>
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t row, int i, const float* f) {
#pragma unroll
  for (int c = 0; c < 8 / R::kPer16; ++c)
    __builtin_amdgcn_raw_buffer_store_b128(R::pack(f + c * R::kPer16), row, i * 8 * R::kBytes + 16 * c, 0, 0);
}
// 8 weights of the lane's columns, `other` where there is no such vector.
__device__ __forceinline__ void weights8(const float* w, int n, int i, float other, float* f) {
  if (w) {
    load8<RowF32>(row_of(w, 0, n * 4), i, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = other;
  }
}

// Sums over the workgroup, the same in every thread, in a fixed order. The slots of two
// calls in a row differ, so one barrier a call is enough.
template <int NTH, int V>
struct BlockSum {
  float (*part)[V][NTH / 64];
  int slot = 0;
  __device__ __forceinline__ void operator()(float* v) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = wave_sum(v[i]);
    if constexpr (NTH > 64) {
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) part[slot][i][wave] = v[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < NTH / 64; ++k) v[i] += part[slot][i][k];
      }
      slot ^= 1;
    }
  }
};

__device__ __forceinline__ float rstd_of(float sum, float inv_n, float eps) { return 1.0f / sqrtf(fmaf(sum, inv_n, eps)); }

template <class R, int NTH, int C>
__global__ __launch_bounds__(NTH) void block_norm(NormArgs a) {
  __shared__ float part[2][1][NTH / 64];
  __shared__ uint32_t top[2][NTH / 64];
  const int lane = threadIdx.x, per = a.N >> 3;
  BlockSum<NTH, 1> sum{part};
  float cw[C][8], pre[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * NTH + lane;
    float g[8];
    weights8(a.post, a.N, i, 1.0f, cw[c]);
    weights8(a.gate_kind == FG_GATE_CHANNEL ? a.gate : nullptr, a.N, i, 1.0f, g);
    weights8(a.pre, a.N, i, 0.0f, pre[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) cw[c][e] *= g[e] * a.beta;
  }
  int flip = 0;
  for (long t = blockIdx.x; t < a.T; t += gridDim.x) {
    float r[C][8], y[C][8];
    const long at = t * a.N;
    const int bytes = a.N * R::kBytes;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      load8<R>(row_of(a.x, at * R::kBytes, bytes), c * NTH + lane, r[c]);
      if (a.y) load8<R>(row_of(a.y, at * R::kBytes, bytes), c * NTH + lane, y[c]);
    }
    if (a.y) {
      float k = a.gate_kind == FG_GATE_TOKEN ? a.gate[t] : 1.0f;
      if (a.post) {
        float v[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[0] = fmaf(y[c][e], y[c][e], v[0]);
        sum(v);
        k *= rstd_of(v[0], a.inv_n, a.eps);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[c][e] = fmaf(y[c][e] * k, cw[c][e], a.alpha * r[c][e]);
        store8<R>(row_of(a.r, at * R::kBytes, bytes), c * NTH + lane, r[c]);
      }
    }
    if (!a.pre) continue;
    float v[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[0] = fmaf(r[c][e], r[c][e], v[0]);
    sum(v);
    const float rx = rstd_of(v[0], a.inv_n, a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) r[c][e] = r[c][e] * rx * pre[c][e];
    const __amdgpu_buffer_rsrc_t codes = row_of(a.h, at, a.N);   // 8-bit outputs
    if (a.out == FG_OUT_SAME) {
#pragma unroll
      for (int c = 0; c < C; ++c) store8<R>(row_of(a.h, at * R::kBytes, bytes), c * NTH + lane, r[c]);
    } else if (a.out == FG_OUT_INT8) {
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) m = amax_bits<8>(r[c], m);
      m = group_max_u32<64>(m);
      if constexpr (NTH > 64) {
        if ((lane & 63) == 0) top[flip][lane >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NTH / 64; ++w) m = umax(m, top[flip][w]);
        flip ^= 1;
      }
      const float s = int8_scale(__uint_as_float(m)), inv = 1.0f / s;
      if (lane == 0) a.s[t] = s;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int i = c * NTH + lane;
        uint32_t q[2];
        int8_encode<8>(r[c], s, inv, q);
        __builtin_amdgcn_raw_buffer_store_b64(u32x2v{q[0], q[1]}, codes, i * 8, 0, 0);
      }
    } else {
      // 16 lanes have a 1x128 block; a group is wholly inside the row or past it
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int i = c * NTH + lane;
        float s = block_scale(__uint_as_float(group_max_u32<16>(amax_bits<8>(r[c], 0u))));
        if (a.out == FG_OUT_E4M3_POW2) s = pow2_up(s);
        const float inv = 1.0f / s;
        u32x2v q;
        if (a.out == FG_OUT_E4M3_POW2) {
          q[0] = e4m3x4_mul(r[c][0], r[c][1], r[c][2], r[c][3], inv);
          q[1] = e4m3x4_mul(r[c][4], r[c][5], r[c][6], r[c][7], inv);
        } else if (s >= kQuotMin) {
          q[0] = e4m3x4_quot(r[c][0], r[c][1], r[c][2], r[c][3], s, inv);
          q[1] = e4m3x4_quot(r[c][4], r[c][5], r[c][6], r[c][7], s, inv);
        } else {
          q[0] = e4m3x4_div(r[c][0], r[c][1], r[c][2], r[c][3], s);
          q[1] = e4m3x4_div(r[c][4], r[c][5], r[c][6], r[c][7], s);
        }
        __builtin_amdgcn_raw_buffer_store_b64(q, codes, i * 8, 0, 0);
        if (i < per && (lane & 15) == 0) a.s[(long)(i >> 4) * a.T + t] = s;
      }
    }
  }
}

struct GradArgs {
  const void *r, *dh, *dr, *y;
  const float *pre, *post, *gate;
  void *dx, *dy;
  float* dgate;   // per token
  float* ws;      // [workgroups][2][N]: sum dh rh, S
  int T, N, gate_kind;
  float alpha, beta, eps, inv_n;
};

template <class R, int NTH, int C>
__global__ __launch_bounds__(NTH) void block_norm_grad(GradArgs a) {
  __shared__ float part3[2][3][NTH / 64], part1[2][1][NTH / 64];
  const int lane = threadIdx.x;
  BlockSum<NTH, 3> sum3{part3};
  BlockSum<NTH, 1> sum1{part1};
  float cw[C][8], pre[C][8], P[C][8], S[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * NTH + lane;
    float g[8];
    weights8(a.post, a.N, i, 1.0f, cw[c]);
    weights8(a.gate_kind == FG_GATE_CHANNEL ? a.gate : nullptr, a.N, i, 1.0f, g);
    weights8(a.pre, a.N, i, 0.0f, pre[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cw[c][e] *= g[e] * a.beta;
      P[c][e] = S[c][e] = 0.0f;
    }
  }
  for (long t = blockIdx.x; t < a.T; t += gridDim.x) {
    float r[C][8], dh[C][8], d[C][8], y[C][8];
    const long at = t * a.N * R::kBytes;
    const int bytes = a.N * R::kBytes;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * NTH + lane;
#pragma unroll
      for (int e = 0; e < 8; ++e) d[c][e] = 0.0f;
      if (a.pre) {
        load8<R>(row_of(a.r, at, bytes), i, r[c]);
        load8<R>(row_of(a.dh, at, bytes), i, dh[c]);
      }
      if (a.dr) load8<R>(row_of(a.dr, at, bytes), i, d[c]);
      if (a.y) load8<R>(row_of(a.y, at, bytes), i, y[c]);
    }
    float v[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (a.pre) {
          v[0] = fmaf(r[c][e], r[c][e], v[0]);
          v[1] = fmaf(dh[c][e] * pre[c][e], r[c][e], v[1]);
        }
        if (a.post) v[2] = fmaf(y[c][e], y[c][e], v[2]);
      }
    if (a.pre || a.post) sum3(v);
    if (a.pre) {
      const float rx = rstd_of(v[0], a.inv_n, a.eps);
      const float m = v[1] * rx * a.inv_n;   // mean of z rh
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float rh = r[c][e] * rx;
          d[c][e] = fmaf(rx, fmaf(-rh, m, dh[c][e] * pre[c][e]), d[c][e]);
          P[c][e] = fmaf(dh[c][e], rh, P[c][e]);
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = a.alpha * d[c][e];
      store8<R>(row_of(a.dx, at, bytes), c * NTH + lane, o);
    }
    if (!a.y) continue;
    const float ry = a.post ? rstd_of(v[2], a.inv_n, a.eps) : 1.0f;
    const float gt = a.gate_kind == FG_GATE_TOKEN ? a.gate[t] : 1.0f;
    float q[1] = {0.0f};   // sum of dR yh, times the folded weights
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[c][e] *= ry;
        S[c][e] = fmaf(gt * d[c][e], y[c][e], S[c][e]);
        d[c][e] *= cw[c][e];
        q[0] = fmaf(d[c][e], y[c][e], q[0]);
      }
    if (a.post || a.gate_kind == FG_GATE_TOKEN) sum1(q);
    if (a.gate_kind == FG_GATE_TOKEN && lane == 0) a.dgate[t] = q[0];
    const float m = a.post ? q[0] * a.inv_n : 0.0f, k = ry * gt;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = k * fmaf(-y[c][e], m, d[c][e]);
      store8<R>(row_of(a.dy, at, bytes), c * NTH + lane, o);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    store8<RowF32>(row_of(a.ws, (long)blockIdx.x * 8 * a.N, a.N * 4), c * NTH + lane, P[c]);
    store8<RowF32>(row_of(a.ws, (long)blockIdx.x * 8 * a.N + 4L * a.N, a.N * 4), c * NTH + lane, S[c]);
  }
}

// The workgroups' sums added up: 32 columns a workgroup, 8 threads a column.
struct SumArgs {
  const float *ws, *post, *gate;
  float *dpre, *dpost, *dgate;   // null: not asked for
  int groups, N;
  float beta;
};
constexpr int kSumCols = 32, kSumParts = 8;
__global__ __launch_bounds__(kSumCols * kSumParts) void block_norm_sums(SumArgs a) {
  __shared__ float part[2][kSumParts][kSumCols];
  const int col = threadIdx.x % kSumCols, p = threadIdx.x / kSumCols;
  const int n = blockIdx.x * kSumCols + col, at = n < a.N ? n : 0;
  float P = 0.0f, S = 0.0f;
  for (int g = p; g < a.groups; g += kSumParts) {
    P += a.ws[(long)g * 2 * a.N + at];
    S += a.ws[((long)g * 2 + 1) * a.N + at];
  }
  part[0][p][col] = P;
  part[1][p][col] = S;
  __syncthreads();
  if (p != 0 || n >= a.N) return;
  P = S = 0.0f;
#pragma unroll
  for (int k = 0; k < kSumParts; ++k) {
    P += part[0][k][col];
    S += part[1][k][col];
  }
  if (a.dpre) a.dpre[n] = P;
  if (a.dpost) a.dpost[n] = a.beta * (a.gate ? a.gate[n] : 1.0f) * S;
  if (a.dgate) a.dgate[n] = a.beta * (a.post ? a.post[n] : 1.0f) * S;
}

// Workgroups of the gradient for T rows of N columns.
int grad_threads(int N) { return N <= 512 ? 64 : N <= 2048 ? 256 : N <= 8192 ? 512 : 1024; }
int grad_groups(int T, int N) {
  const int most = kCUs * (1024 / grad_threads(N));
  return T < most ? T : most;
}

template <class R, int NTH, int C>
int launch_norm(const NormArgs& a, hipStream_t s) {
  const int most = kCUs * (1024 / NTH);
  hipLaunchKernelGGL((block_norm<R, NTH, C>), dim3(a.T < most ? a.T : most), dim3(NTH), 0, s, a);
  return hipGetLastError() == hipSuccess ? FG_OK : FG_ELAUNCH;
}
template <class R>
int launch_norm_of(const NormArgs& a, hipStream_t s) {
  const int per = a.N / 8;
  if (per <= 64) return launch_norm<R, 64, 1>(a, s);
  if (per <= 256) return launch_norm<R, 256, 1>(a, s);
  if (per <= 512) return launch_norm<R, 256, 2>(a, s);
  if (per <= 1024) return launch_norm<R, 256, 4>(a, s);
  return launch_norm<R, 1024, 2>(a, s);
}

template <class R, int NTH, int C>
int launch_grad(const GradArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((block_norm_grad<R, NTH, C>), dim3(grad_groups(a.T, a.N)), dim3(NTH), 0, s, a);
  return hipGetLastError() == hipSuccess ? FG_OK : FG_ELAUNCH;
}
template <class R>
int launch_grad_of(const GradArgs& a, hipStream_t s) {
  switch (grad_threads(a.N)) {
    case 64: return launch_grad<R, 64, 1>(a, s);
    case 256: return launch_grad<R, 256, 1>(a, s);
    case 512: return launch_grad<R, 512, 2>(a, s);
    default: return launch_grad<R, 1024, 2>(a, s);
  }
}

bool sizes_ok(int dtype, int T, int N, int gate_kind, float eps) {
  return T >= 0 && N >= 8 && N % 8 == 0 && N <= kMaxCols && (dtype == FG_BF16 || dtype == FG_FP32) &&
         gate_kind >= FG_GATE_NONE && gate_kind <= FG_GATE_TOKEN && eps > 0.0f;
}

}  // namespace

extern "C" {

int fg_block_norm(const void* x, const void* y, int dtype, const float* pre, const float* post, const float* gate,
                  int gate_kind, void* r, void* h, float* s, int out, int T, int N, float alpha, float beta, float eps,
                  hipStream_t stream) {
  if (!sizes_ok(dtype, T, N, gate_kind, eps) || out < FG_OUT_SAME || out > FG_OUT_INT8) return FG_EINVAL;
  const bool e4m3 = out == FG_OUT_E4M3 || out == FG_OUT_E4M3_POW2;
  if (pre && ((e4m3 && N % 128) || (out == FG_OUT_INT8 && N % 16))) return FG_EINVAL;
  if (T == 0) return FG_OK;
  // something to do, and what each part needs
  if (!x || (!y && !pre) || (y && !r) || (!y && (post || gate_kind != FG_GATE_NONE))) return FG_EINVAL;
  if ((gate_kind != FG_GATE_NONE) != (gate != nullptr) || (pre && (!h || (out != FG_OUT_SAME && !s)))) return FG_EINVAL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(r, 16) || !aligned(h, 16) || !aligned(pre, 4) || !aligned(post, 4) ||
      !aligned(gate, 4) || !aligned(s, 4))
    return FG_EINVAL;
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  const NormArgs a = {x, y, pre, post, gate, r, h, s, T, N, gate_kind, out, alpha, beta, eps, 1.0f / (float)N};
  return dtype == FG_BF16 ? launch_norm_of<RowBf16>(a, stream) : launch_norm_of<RowF32>(a, stream);
}

int fg_block_norm_grad_workspace(int T, int N, size_t* bytes) {
  if (!bytes || !sizes_ok(FG_BF16, T, N, FG_GATE_NONE, 1.0f)) return FG_EINVAL;
  *bytes = (size_t)grad_groups(T, N) * 2 * N * sizeof(float);
  return FG_OK;
}

int fg_block_norm_grad(const void* r, const void* dh, const void* dr, const void* y, int dtype, const float* pre,
                       const float* post, const float* gate, int gate_kind, void* dx, void* dy, float* dgate, float* dpre,
                       float* dpost, void* ws, int T, int N, float alpha, float beta, float eps, hipStream_t stream) {
  if (!sizes_ok(dtype, T, N, gate_kind, eps)) return FG_EINVAL;
  const bool channel = gate_kind == FG_GATE_CHANNEL, sums = pre || post || channel;
  if ((pre && !dpre) || (post && !dpost) || (channel && (!gate || !dgate))) return FG_EINVAL;
  if (T > 0) {   // without rows only the vectors matter
    if ((dh != nullptr) != (pre != nullptr) || (pre && !r) || (!dh && !dr) || !dx || !ws) return FG_EINVAL;
    if ((y != nullptr) != (dy != nullptr) || (!y && (post || gate_kind != FG_GATE_NONE))) return FG_EINVAL;
    if ((gate_kind != FG_GATE_NONE) != (gate != nullptr) || (gate && !dgate)) return FG_EINVAL;
  }
  if (!aligned(r, 16) || !aligned(dh, 16) || !aligned(dr, 16) || !aligned(y, 16) || !aligned(dx, 16) || !aligned(dy, 16) ||
      !aligned(pre, 4) || !aligned(post, 4) || !aligned(gate, 4) || !aligned(dgate, 4) || !aligned(dpre, 4) ||
      !aligned(dpost, 4) || !aligned(ws, 16))
    return FG_EINVAL;
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  if (T > 0) {
    const GradArgs a = {r, dh, dr, y, pre, post, gate, dx, dy, dgate, static_cast<float*>(ws), T, N, gate_kind,
                        alpha, beta, eps, 1.0f / (float)N};
    const int rc = dtype == FG_BF16 ? launch_grad_of<RowBf16>(a, stream) : launch_grad_of<RowF32>(a, stream);
    if (rc != FG_OK) return rc;
  }
  if (!sums) return FG_OK;
  const SumArgs b = {static_cast<const float*>(ws), post, channel ? gate : nullptr, pre ? dpre : nullptr,
                     post ? dpost : nullptr, channel ? dgate : nullptr, grad_groups(T, N), N, beta};
  hipLaunchKernelGGL(block_norm_sums, dim3((N + kSumCols - 1) / kSumCols), dim3(kSumCols * kSumParts), 0, stream, b);
  return hipGetLastError() == hipSuccess ? FG_OK : FG_ELAUNCH;
}

}  // extern "C"
