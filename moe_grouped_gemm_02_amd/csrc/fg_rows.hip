// fg_rows.hip -- token rows into and out of the grouped GEMMs' sorted layouts,
// and the gradient of the way back.
//
// With row = rows[t, j] the sorted row of token t's choice j (none where it is
// outside the layout, such as -1):
//
//   dispatch      Q[row] = e4m3(w[t, j] x[t] / s),  s = amax / 448 of each 1x128 block
//   combine       out[t] = base[t] + sum_j w[t, j] y[row]
//   combine_grad  dw[t, j] = <dout[t], y[row]>,  dy[row] = w[t, j] dout[t]
//
// in fp32 with one rounding at the end. The gradient of dispatch's copies is
// combine with all weights one.
//
// All are bound by memory traffic. Each goes by tokens, not by sorted rows: a
// token's row is read from HBM once and used for all its choices, and whole
// rows of several KB are read or written at each sorted row, so the indirection
// costs no bandwidth. A lane handles 16 consecutive elements (or 16 bytes), so
// eight lanes hold a 1x128 block and its largest value takes three DPP steps.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fg.h"
#include "fg_device.hpp"
#include "fg_e4m3_quot.hpp"
#include "fg_wave.hpp"

namespace {

using namespace fg;

constexpr int kThreads = 256;

// Sorted E4M3 rows: codes [GM][H], scales [G][H/128][M] with GM = G * M rows.
struct QuantOut {
  uint8_t* Q;
  float* sa;
  int H, M, GM;
};

// 16 elements of a row starting at element 16 * i.
template <class R>
__device__ __forceinline__ void load16(const void* x, long row, int H, int i, float* f) {
  const u32x4* p = (const u32x4*)((const char*)x + (row * H + 16L * i) * R::kBytes);
  constexpr int N = 16 / R::kPer16;
#pragma unroll
  for (int c = 0; c < N; ++c) R::unpack(p[c], f + c * R::kPer16);
}

__device__ __forceinline__ float amax16(const float* f) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}

// Codes of 16 values of a block with scale s.
__device__ __forceinline__ u32x4 encode16(const float* f, float s, bool pow2) {
  u32x4 q;
  const float inv = 1.0f / s;
  if (pow2) {
#pragma unroll
    for (int c = 0; c < 4; ++c) q[c] = e4m3x4_mul(f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3], inv);
  } else if (s >= kQuotMin) {
#pragma unroll
    for (int c = 0; c < 4; ++c) q[c] = e4m3x4_quot(f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3], s, inv);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) q[c] = e4m3x4_div(f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3], s);
  }
  return q;
}

// Stores unit i (16 codes) of sorted row `row`, and the block's scale from the
// first of its eight lanes.
__device__ __forceinline__ void store_unit(const QuantOut& o, int row, int i, u32x4 q, float s) {
  __builtin_nontemporal_store(q, (u32x4*)(o.Q + (long)row * o.H + 16L * i));
  if ((i & 7) == 0) {
    const int g = row / o.M, r = row - g * o.M;
    o.sa[((long)g * (o.H >> 7) + (i >> 3)) * o.M + r] = s;
  }
}

// Token and unit of this lane when a token has `per` units, lanes taken in order.
__device__ __forceinline__ bool unit_of(int per, int T, long* t, int* i) {
  if (gridDim.x < (1u << 23)) {   // below 2^31 units 32 bits do: a 64-bit division is half of combine's instructions
    const unsigned v = blockIdx.x * kThreads + threadIdx.x, q = v / (unsigned)per;
    *t = q;
    *i = (int)(v - q * (unsigned)per);
  } else {
    const long v = (long)blockIdx.x * kThreads + threadIdx.x;
    *t = v / per;
    *i = (int)(v - *t * per);
  }
  return *t < T;
}

// Dispatch: a wave takes 64 units (1024 columns) of one token, a workgroup those of
// kTokens tokens. The codes leave as they are made, a kilobyte of a sorted row per
// store. The scales, one float in each K-block's own column of sorted rows, wait
// until the workgroup's tokens are done: lanes then run over the slots, whose rows
// are neighbours where tokens chose the same expert, so a store writes runs of rows
// and not 64 lines.
//
// A slot's scale needs only the token's largest value: rounding is monotone, so the
// largest |w x| as rounded is |w| times the largest |x|, rounded.
constexpr int kUnits = 64, kUnitBlocks = kUnits / 8, kTokens = 4, kDispatchThreads = 64 * kTokens;

template <class R, bool POW2, bool W>
__global__ __launch_bounds__(kDispatchThreads) void dispatch_quant(const void* __restrict__ x,
                                                                   const int32_t* __restrict__ rows,
                                                                   const float* __restrict__ w, QuantOut o, int T,
                                                                   int k, int strips) {
  __shared__ float amax[kTokens][kUnitBlocks];
  const long t0 = (long)(blockIdx.x / (unsigned)strips) * kTokens;
  const int strip = blockIdx.x % (unsigned)strips;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = o.H >> 4, i = strip * kUnits + lane;   // whole groups of eight lanes have units
  const long t = t0 + wave;
  if (t < T) {   // uniform
    float f[16];
    load16<R>(x, t, o.H, i < per ? i : per - 8 + (lane & 7), f);
    const float m = group8_max(amax16(f));
    if ((lane & 7) == 0) amax[wave][lane >> 3] = m;
    float s = block_scale(m);
    if (POW2) s = pow2_up(s);
    u32x4 q = {0u, 0u, 0u, 0u};
    if (!W) q = encode16(f, s, POW2);
    for (int j = 0; j < k; ++j) {
      const int row = rows[t * k + j];
      if ((unsigned)row >= (unsigned)o.GM || i >= per) continue;
      if (W) {
        const float wj = w[t * k + j];
        s = block_scale(fabsf(wj) * m);
        if (POW2) s = pow2_up(s);
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = f[e] * wj;
        q = encode16(v, s, POW2);
      }
      // nontemporal: a later call reads the sorted rows, this one does not
      __builtin_nontemporal_store(q, (u32x4*)(o.Q + (long)row * o.H + 16L * i));
    }
  }
  __syncthreads();
  const int slots = (int)(T - t0 < kTokens ? T - t0 : kTokens) * k;
  const int KB = o.H >> 7, kb0 = strip * kUnitBlocks;
  const int blocks = KB - kb0 < kUnitBlocks ? KB - kb0 : kUnitBlocks;
  for (int s0 = 0; s0 < slots; s0 += 64) {
    const int sl = s0 + lane;
    if (sl >= slots) break;
    const int row = rows[t0 * k + sl];
    if ((unsigned)row >= (unsigned)o.GM) continue;
    const float wj = W ? fabsf(w[t0 * k + sl]) : 1.0f;
    const int g = row / o.M, token = sl / k;
    float* sa = o.sa + (long)g * KB * o.M + (row - g * o.M);
    for (int b = wave; b < blocks; b += kTokens) {
      float s = block_scale(W ? wj * amax[token][b] : amax[token][b]);
      if (POW2) s = pow2_up(s);
      sa[(long)(kb0 + b) * o.M] = s;
    }
  }
}

// STREAM: out is larger than the caches.
template <class R, bool W, bool STREAM>
__global__ __launch_bounds__(kThreads) void combine(const void* __restrict__ y, const int32_t* __restrict__ rows,
                                                    const float* __restrict__ w, const void* base,
                                                    void* out, int T, int k, int N, int n_rows) {
  long t;
  int i;
  const int per = N / R::kPer16;
  if (!unit_of(per, T, &t, &i)) return;
  float acc[R::kPer16];
  const u32x4* yv = (const u32x4*)y;
#pragma unroll
  for (int e = 0; e < R::kPer16; ++e) acc[e] = 0.0f;
  for (int j0 = 0; j0 < k && n_rows > 0; j0 += 4) {
    u32x4 v[4];
    float wj[4];
    bool ok[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int j = j0 + c;
      // Loads are not predicated (a branch each, and a wait): without a row the first one is
      // read and dropped. y's rows are read this once: past the caches, 110 against 127 us
      // at T 8192, k 4, N 7168.
      const int row = rows[t * k + (j < k ? j : j0)];
      ok[c] = j < k && (unsigned)row < (unsigned)n_rows;
      wj[c] = W ? w[t * k + (j < k ? j : j0)] : 1.0f;
      v[c] = __builtin_nontemporal_load(&yv[(long)(ok[c] ? row : 0) * per + i]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (!ok[c]) {
        v[c] = u32x4{0u, 0u, 0u, 0u};
        wj[c] = 0.0f;
      }
      float f[R::kPer16];
      R::unpack(v[c], f);
#pragma unroll
      for (int e = 0; e < R::kPer16; ++e) acc[e] = fmaf(wj[c], f[e], acc[e]);
    }
  }
  if (base) {
    float f[R::kPer16];
    R::unpack(((const u32x4*)base)[t * per + i], f);
#pragma unroll
    for (int e = 0; e < R::kPer16; ++e) acc[e] += f[e];
  }
  store16<STREAM>(&((u32x4*)out)[t * per + i], R::pack(acc));
}

// One workgroup of NTH threads per token: its row of dout stays in registers for a unit
// at a time while the choices' rows of y pass by, kGradChoices per sweep of the row.
constexpr int kGradChoices = 8;
constexpr int kFewTokens = 512;

// Sums acc over the workgroup in a fixed order and writes dw.
template <int NTH>
__device__ __forceinline__ void reduce_dw(float* acc, float (*part)[kGradChoices], float* dw, int n) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int c = 0; c < kGradChoices; ++c) {
    const float s = wave_sum(acc[c]);
    if (lane == 0) part[wave][c] = s;
  }
  __syncthreads();
  if ((int)threadIdx.x < n) {
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < NTH / 64; ++v) s += part[v][threadIdx.x];
    dw[threadIdx.x] = s;
  }
  __syncthreads();
}

// The bytes of y (all choices, T k N of them; how many have a row here the host does not
// know) from which combine_grad reads it past the caches. With dy / dw alone, N 7168, k 8, bf16: T 2048 116.6 / 60.2 -> 94.9 / 55.0 us, T
// 8192 400 / 179 -> 402 / 165; N 2048, k 8, T 8192 113 / 54 -> 98 / 49. Below, shorter
// batches lose: N 2048, k 8, T 1024 (34 MB) 13.3 / 9.0 -> 15.2 / 9.8 us. Stores of dy past
// them, and y in the E4M3 form, where a lane reads 32 bytes in two pieces, gain at some
// sizes what they lose at others and stay ordinary.
constexpr long long kGradStreamBytes = 128ll << 20;

template <class R, bool STREAM, int NTH>
__global__ __launch_bounds__(NTH) void combine_grad(const void* __restrict__ dout, const void* __restrict__ y,
                                                         const int32_t* __restrict__ rows,
                                                         const float* __restrict__ w, void* __restrict__ dy,
                                                         float* __restrict__ dw, int k, int N, int n_rows) {
  __shared__ float part[NTH / 64][kGradChoices];
  const long t = blockIdx.x;
  const int per = N / R::kPer16;
  const u32x4* dv = (const u32x4*)dout + t * per;
  for (int j0 = 0; j0 < k; j0 += kGradChoices) {
    const int n = k - j0 < kGradChoices ? k - j0 : kGradChoices;
    float acc[kGradChoices], wj[kGradChoices];
    int row[kGradChoices];
#pragma unroll
    for (int c = 0; c < kGradChoices; ++c) {
      const int r = c < n ? rows[t * k + j0 + c] : -1;
      row[c] = (unsigned)r < (unsigned)n_rows ? r : -1;
      wj[c] = c < n ? w[t * k + j0 + c] : 0.0f;
      acc[c] = 0.0f;
    }
    for (int i = threadIdx.x; i < per; i += NTH) {
      float d[R::kPer16];
      R::unpack(dv[i], d);
#pragma unroll
      for (int c = 0; c < kGradChoices; ++c) {
        if (row[c] < 0) continue;   // uniform
        float f[R::kPer16];
        const long at = (long)row[c] * per + i;
        R::unpack(load16b<STREAM>((const u32x4*)y + at), f);
#pragma unroll
        for (int e = 0; e < R::kPer16; ++e) {
          acc[c] = fmaf(d[e], f[e], acc[c]);
          f[e] = wj[c] * d[e];
        }
        if (dy) ((u32x4*)dy)[at] = R::pack(f);
      }
    }
    reduce_dw<NTH>(acc, part, dw + t * k + j0, n);
  }
}

template <class R, bool POW2, int NTH>
__global__ __launch_bounds__(NTH) void combine_grad_quant(const void* __restrict__ dout,
                                                               const void* __restrict__ y,
                                                               const int32_t* __restrict__ rows,
                                                               const float* __restrict__ w, QuantOut o,
                                                               float* __restrict__ dw, int k) {
  __shared__ float part[NTH / 64][kGradChoices];
  const long t = blockIdx.x;
  const int per = o.H >> 4;
  for (int j0 = 0; j0 < k; j0 += kGradChoices) {
    const int n = k - j0 < kGradChoices ? k - j0 : kGradChoices;
    float acc[kGradChoices], wj[kGradChoices];
    int row[kGradChoices];
#pragma unroll
    for (int c = 0; c < kGradChoices; ++c) {
      const int r = c < n ? rows[t * k + j0 + c] : -1;
      row[c] = (unsigned)r < (unsigned)o.GM ? r : -1;
      wj[c] = c < n ? w[t * k + j0 + c] : 0.0f;
      acc[c] = 0.0f;
    }
    for (int i = threadIdx.x; i < per; i += NTH) {   // whole groups of eight lanes
      float d[16];
      load16<R>(dout, t, o.H, i, d);
      const float top = group8_max(amax16(d));
#pragma unroll
      for (int c = 0; c < kGradChoices; ++c) {
        if (row[c] < 0) continue;
        float f[16];
        load16<R>(y, row[c], o.H, i, f);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          acc[c] = fmaf(d[e], f[e], acc[c]);
          f[e] = wj[c] * d[e];
        }
        float s = block_scale(fabsf(wj[c]) * top);   // as in dispatch
        if (POW2) s = pow2_up(s);
        store_unit(o, row[c], i, encode16(f, s, POW2), s);
      }
    }
    reduce_dw<NTH>(acc, part, dw + t * k + j0, n);
  }
}

bool type_ok(int dtype) { return dtype == FG_BF16 || dtype == FG_FP32; }

// Sizes of the E4M3 rows: G x M of them, H columns.
int check_quant(int dtype, int T, int k, int H, int G, int M, int scales) {
  if (T < 0 || k < 1 || H < 128 || H % 128 || H > (1 << 24) || G < 1 || M < (T > 0 ? 1 : 0) || !type_ok(dtype)) return FG_EINVAL;
  if ((scales != FG_SCALES_FP32 && scales != FG_SCALES_POW2) || (long long)G * M > 0x7fffffffLL) return FG_EINVAL;
  return FG_OK;
}

int check_rows(int dtype, int T, int k, int N, int n_rows) {
  if (T < 0 || k < 1 || N < 8 || N % 8 || N > (1 << 24) || n_rows < 0 || !type_ok(dtype)) return FG_EINVAL;
  return FG_OK;
}

// Workgroups of kThreads lanes for T tokens of `per` units; 0: too many.
unsigned unit_grid(int T, int per) {
  const long long n = ((long long)T * per + kThreads - 1) / kThreads;
  return n > 0x7fffffffLL ? 0u : (unsigned)n;
}

template <class R>
void launch_dispatch(bool pow2, hipStream_t s, const void* x, const int32_t* rows, const float* w,
                     const QuantOut& o, int T, int k) {
  const int strips = (o.H / 16 + kUnits - 1) / kUnits;
  const dim3 g((unsigned)((T + kTokens - 1L) / kTokens * strips)), b(kDispatchThreads);
  if (pow2 && w) hipLaunchKernelGGL((dispatch_quant<R, true, true>), g, b, 0, s, x, rows, w, o, T, k, strips);
  else if (pow2) hipLaunchKernelGGL((dispatch_quant<R, true, false>), g, b, 0, s, x, rows, w, o, T, k, strips);
  else if (w) hipLaunchKernelGGL((dispatch_quant<R, false, true>), g, b, 0, s, x, rows, w, o, T, k, strips);
  else hipLaunchKernelGGL((dispatch_quant<R, false, false>), g, b, 0, s, x, rows, w, o, T, k, strips);
}

// Threads of a gradient workgroup for rows of `per` units: no more than have one (256
// with a quarter at work: N 1024, k 2, T 4096 to E4M3, 16.6 us); with few tokens enough
// for the whole row at once, else 256, which leaves room for other workgroups. 256 / 1024
// threads, bf16: N 7168, k 8, T 1 / 64 / 256 10.4 / 15.2 / 17.9 against 6.1 / 8.0 / 12.1 us;
// N 4096, k 4, T 256 / 512 / 2048 7.8 / 9.5 / 30.5 against 6.4 / 10.8 / 44.8 us.
int grad_threads(int T, int per) { return per <= 64 ? 64 : per > 256 && T < kFewTokens ? 1024 : 256; }

template <class R, bool STREAM, class... Args>
void launch_grad(int T, int per, hipStream_t s, Args... a) {
  const dim3 g((unsigned)T);
  switch (grad_threads(T, per)) {
    case 64: hipLaunchKernelGGL((combine_grad<R, STREAM, 64>), g, dim3(64), 0, s, a...); break;
    case 256: hipLaunchKernelGGL((combine_grad<R, STREAM, 256>), g, dim3(256), 0, s, a...); break;
    default: hipLaunchKernelGGL((combine_grad<R, STREAM, 1024>), g, dim3(1024), 0, s, a...); break;
  }
}
template <class R, bool POW2, class... Args>
void launch_grad_quant(int T, int per, hipStream_t s, Args... a) {
  const dim3 g((unsigned)T);
  switch (grad_threads(T, per)) {
    case 64: hipLaunchKernelGGL((combine_grad_quant<R, POW2, 64>), g, dim3(64), 0, s, a...); break;
    case 256: hipLaunchKernelGGL((combine_grad_quant<R, POW2, 256>), g, dim3(256), 0, s, a...); break;
    default: hipLaunchKernelGGL((combine_grad_quant<R, POW2, 1024>), g, dim3(1024), 0, s, a...); break;
  }
}

template <class R, class... Args>
void launch_combine(bool weighted, bool big, dim3 g, hipStream_t s, Args... a) {
  const dim3 b(kThreads);
  if (weighted && big) hipLaunchKernelGGL((combine<R, true, true>), g, b, 0, s, a...);
  else if (weighted) hipLaunchKernelGGL((combine<R, true, false>), g, b, 0, s, a...);
  else if (big) hipLaunchKernelGGL((combine<R, false, true>), g, b, 0, s, a...);
  else hipLaunchKernelGGL((combine<R, false, false>), g, b, 0, s, a...);
}

int launched() { return hipGetLastError() == hipSuccess ? FG_OK : FG_ELAUNCH; }

}  // namespace

extern "C" {

int fg_dispatch_quant(const void* x, int dtype, const int32_t* rows, const float* w, void* Q, float* sa, int T,
                      int k, int H, int G, int M, int scales, hipStream_t stream) {
  const int rc = check_quant(dtype, T, k, H, G, M, scales);
  if (rc != FG_OK || T == 0) return rc;
  if (!x || !rows || !Q || !sa || !aligned(x, 16) || !aligned(rows, 4) || !aligned(Q, 16) || !aligned(sa, 4) ||
      (w && !aligned(w, 4)))
    return FG_EINVAL;
  if (((long long)T + kTokens - 1) / kTokens * ((H + 1023) / 1024) > 0x7fffffffLL) return FG_EINVAL;
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  const QuantOut o = {static_cast<uint8_t*>(Q), sa, H, M, G * M};
  const bool pow2 = scales == FG_SCALES_POW2;
  if (dtype == FG_BF16) launch_dispatch<RowBf16>(pow2, stream, x, rows, w, o, T, k);
  else launch_dispatch<RowF32>(pow2, stream, x, rows, w, o, T, k);
  return launched();
}

int fg_combine(const void* y, int dtype, const int32_t* rows, const float* w, const void* base, void* out, int T,
               int k, int N, int n_rows, hipStream_t stream) {
  const int rc = check_rows(dtype, T, k, N, n_rows);
  if (rc != FG_OK || T == 0) return rc;
  if ((!y && n_rows) || !rows || !out || !aligned(y, 16) || !aligned(rows, 4) || !aligned(out, 16) ||
      (w && !aligned(w, 4)) || (base && !aligned(base, 16)))
    return FG_EINVAL;
  const unsigned grid = unit_grid(T, dtype == FG_BF16 ? N / 8 : N / 4);
  if (grid == 0) return FG_EINVAL;
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  const dim3 g(grid);
  const bool big = (long long)T * N * (dtype == FG_BF16 ? 2 : 4) > kStreamBytes;
  if (dtype == FG_BF16) launch_combine<RowBf16>(w != nullptr, big, g, stream, y, rows, w, base, out, T, k, N, n_rows);
  else launch_combine<RowF32>(w != nullptr, big, g, stream, y, rows, w, base, out, T, k, N, n_rows);
  return launched();
}

int fg_combine_grad(const void* dout, const void* y, int dtype, const int32_t* rows, const float* w, void* dy,
                    float* dw, int T, int k, int N, int n_rows, hipStream_t stream) {
  const int rc = check_rows(dtype, T, k, N, n_rows);
  if (rc != FG_OK || T == 0) return rc;
  if (!dout || (!y && n_rows) || !rows || !w || !dw || !aligned(dout, 16) || !aligned(y, 16) || !aligned(rows, 4) ||
      !aligned(w, 4) || !aligned(dw, 4) || (dy && !aligned(dy, 16)))
    return FG_EINVAL;
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  const bool big = (long long)T * k * N * (dtype == FG_BF16 ? 2 : 4) > kGradStreamBytes;
  if (dtype == FG_BF16 && big) launch_grad<RowBf16, true>(T, N / 8, stream, dout, y, rows, w, dy, dw, k, N, n_rows);
  else if (dtype == FG_BF16) launch_grad<RowBf16, false>(T, N / 8, stream, dout, y, rows, w, dy, dw, k, N, n_rows);
  else if (big) launch_grad<RowF32, true>(T, N / 4, stream, dout, y, rows, w, dy, dw, k, N, n_rows);
  else launch_grad<RowF32, false>(T, N / 4, stream, dout, y, rows, w, dy, dw, k, N, n_rows);
  return launched();
}

int fg_combine_grad_quant(const void* dout, const void* y, int dtype, const int32_t* rows, const float* w, void* Q,
                          float* sq, float* dw, int T, int k, int N, int G, int M, int scales, hipStream_t stream) {
  const int rc = check_quant(dtype, T, k, N, G, M, scales);
  if (rc != FG_OK || T == 0) return rc;
  if (!dout || !y || !rows || !w || !Q || !sq || !dw || !aligned(dout, 16) || !aligned(y, 16) || !aligned(rows, 4) ||
      !aligned(w, 4) || !aligned(Q, 16) || !aligned(sq, 4) || !aligned(dw, 4))
    return FG_EINVAL;
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  const QuantOut o = {static_cast<uint8_t*>(Q), sq, N, M, G * M};
  const bool pow2 = scales == FG_SCALES_POW2;
  if (dtype == FG_BF16 && pow2) launch_grad_quant<RowBf16, true>(T, N / 16, stream, dout, y, rows, w, o, dw, k);
  else if (dtype == FG_BF16) launch_grad_quant<RowBf16, false>(T, N / 16, stream, dout, y, rows, w, o, dw, k);
  else if (pow2) launch_grad_quant<RowF32, true>(T, N / 16, stream, dout, y, rows, w, o, dw, k);
  else launch_grad_quant<RowF32, false>(T, N / 16, stream, dout, y, rows, w, o, dw, k);
  return launched();
}

}  // extern "C"
