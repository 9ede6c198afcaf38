// fg_int8_rows.hip -- rows as 8-bit integers with one scale each, the operands of the
// 8-bit integer product:
//
//     s = max(amax / 127, 2^-126) (1 for a row of zeros),  q = rint(v / s)
//
// with amax the row's largest |v|, the quotient rounded to fp32 and ties to even. v is
// a row as it is, a token's row times a weight in each of its plan rows, or the gated
// activation silu(gate) up of a first projection whose columns interleave gate and up
// every 128 (the layout of the fused E4M3 call).
//
// All are bound by memory traffic: a row is read once and stays in registers between
// its largest value and its codes. A lane holds units of 16 elements, 16 bytes of
// codes; a workgroup (or a wave, for rows of up to 1024) has one row, and a wave 8, 4 or 2 rows
// of up to 128, 256 or 512 side by side (65536 rows of 128 bf16 5.5 us, one a wave 15.6). Measured: 8192 rows
// of 7168 bf16 31 us (5.7 TB/s; fp32 51 us), dispatch of 8192 tokens, 4 of 64 experts, H 7168 67 us
// (weighted 72), of 128 tokens, k 8 4.3-4.6 us (latency; 8.9 with a load of each choice's row
// in turn), silu(gate) up of 2000 rows of 2048 in 5120 7.5 us (14.4 with expf, the IEEE
// division and half of the threads idle), of 8192 rows of 2048 15.6 us (5.4 TB/s; fp32 28), of
// 128 rows 3.2.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fg.h"
#include "fg_device.hpp"
#include "fg_int8_quot.hpp"

namespace {

using namespace fg;

constexpr int kMaxRow = 65536;   // 1024 threads of 4 units

// The row's largest value from its NTH threads' own.
template <int NTH>
__device__ __forceinline__ float row_amax(uint32_t m, uint32_t* part) {
  if constexpr (NTH == 8) {
    m = umax(m, dpp_u32<kQuadXor1>(m));
    m = umax(m, dpp_u32<kQuadXor2>(m));
    return __uint_as_float(umax(m, dpp_u32<kHalfMirror>(m)));
  }
  m = group_max_u32<NTH < 64 ? 16 : 64>(m);
  if constexpr (NTH == 32) m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
  if constexpr (NTH > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < NTH / 64; ++v) m = umax(m, part[v]);
  }
  return __uint_as_float(m);
}

// x / (1 + exp(-x)) to about 3 ulp, for x not below kSiluLow. exp(-x) = 2^h 2^l with h the rounded
// product -x log2 e and l what it misses (the hardware's 2^h alone is off by |x| 2^-24); the
// reciprocal is the hardware's. From 88 on 1 + exp(-x) is 1, and h and l stay finite.
constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147182f;
constexpr float kSiluLow = -87.0f;   // h below 126: exp(-x) and its reciprocal are normal numbers
__device__ __forceinline__ float silu(float x) {
  const float z = -fminf(x, 88.0f), h = z * kLog2e, l = fmaf(z, kLog2eLow, fmaf(z, kLog2e, -h));
  const float e = __builtin_amdgcn_exp2f(h);
  return x * __builtin_amdgcn_rcpf(1.0f + fmaf(e, l * kLn2, e));
}
// silu(x) u for x below kSiluLow, where 1 + exp(-x) is exp(-x): x exp(x) u, which a large u makes a number
// like any other. exp(x) is taken as a square; its root times 2^32 is a normal number down to x = -184,
// where x exp(x) u is below 2^-129 for every u and no code sees it: x stops there. (h / 2 + 32 is exact.)
// Minus infinity gives NaN, as inf / (1 + inf).
__device__ __forceinline__ float silu_low(float x, float u) {
  const float c = fmaxf(x, -184.0f), h = c * kLog2e, l = fmaf(c, kLog2eLow, fmaf(c, kLog2e, -h));
  const float b = __builtin_amdgcn_exp2f(fmaf(h, 0.5f, 32.0f));
  return fmaf(c * fmaf(b, l * kLn2, b) * (u * b), 0x1p-64f, x - x);
}
// silu(g) u of a lane's N pairs, into g. The values far below zero are put right in a branch that no wave takes
// whose gates are all ordinary (1001 tokens, k 3, I 2048 bf16 7.5 us with and without it; one row in a hundred
// with gates of 50 rms, which take it, 7.6; one formula for all gates 9.0).
template <int N>
__device__ __forceinline__ void silu_times(float* g, const float* u) {
  float least = g[0], v[N];
#pragma unroll
  for (int e = 1; e < N; ++e) least = fminf(least, g[e]);
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = silu(g[e]) * u[e];
  if (least < kSiluLow) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (g[e] < kSiluLow) v[e] = silu_low(g[e], u[e]);
  }
#pragma unroll
  for (int e = 0; e < N; ++e) g[e] = v[e];
}

enum Mode { kRows = 0, kDispatch = 1, kSwiglu = 2 };

struct RowArgs {
  const void* x;
  const int32_t* index;   // dispatch: rows [T][k]; swiglu: slots [rows] or null
  const float* w;         // dispatch: [T][k] or null
  uint8_t* q;
  float* s;
  int T, k, H, n_rows;
  long row0;   // of this launch
};

template <class R>
__device__ __forceinline__ void unit16(const char* at, float* f) {
  constexpr int N = 16 / R::kPer16;
#pragma unroll
  for (int c = 0; c < N; ++c) R::unpack(((const u32x4*)at)[c], f + c * R::kPer16);
}

__device__ __forceinline__ void store_codes(uint8_t* at, const uint32_t* q) {
  __builtin_nontemporal_store(u32x4{q[0], q[1], q[2], q[3]}, (u32x4*)at);
}

template <class R, int MODE, int NTH, int C>
__global__ __launch_bounds__(NTH <= 64 ? 256 : NTH) void quant_int8(RowArgs a) {
  static_assert(NTH >= 64 || (C == 1 && MODE != kDispatch), "short rows: a unit a lane, no choices over the wave");
  __shared__ uint32_t part[NTH > 64 ? NTH / 64 : 1];
  constexpr int kPerGroup = NTH <= 64 ? 256 / NTH : 1;   // rows of a workgroup
  const int lane = threadIdx.x % NTH, below = threadIdx.x / NTH;
  const long row = a.row0 + (long)blockIdx.x * kPerGroup + (NTH == 64 ? __builtin_amdgcn_readfirstlane(below) : below);
  if (row >= a.T) return;
  if (MODE == kSwiglu && a.index && a.index[row] < 0) return;   // uniform over the row's threads
  const int per = a.H >> 4;
  float f[C][16];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * NTH + lane, at = i < per ? i : per - 1;   // the last unit again: no branch around the loads
    if constexpr (MODE == kSwiglu) {
      // unit i: columns 16 i of the activation, gate at 256 (i / 8) + 16 (i % 8), up 128 further
      const char* g = (const char*)a.x + (row * 2 * a.H + (at >> 3) * 256L + (at & 7) * 16) * R::kBytes;
      float u[16];
      unit16<R>(g, f[c]);
      unit16<R>(g + 128 * R::kBytes, u);
      silu_times<16>(f[c], u);
    } else {
      unit16<R>((const char*)a.x + (row * a.H + 16L * at) * R::kBytes, f[c]);
    }
    m = amax_bits<16>(f[c], m);
  }
  const float amax = row_amax<NTH>(m, part);
  if constexpr (MODE != kDispatch) {
    const float s = int8_scale(amax), inv = 1.0f / s;
    if (lane == 0) a.s[row] = s;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * NTH + lane;
      uint32_t q[4];
      int8_encode<16>(f[c], s, inv, q);
      if (i < per) store_codes(a.q + row * a.H + 16L * i, q);
    }
  } else {
    // the choices' rows and weights in one load, a choice a lane; without weights all get
    // the same codes
    uint32_t q[C][4];
    float s = int8_scale(amax);
    const float inv = 1.0f / s;
    if (!a.w) {
#pragma unroll
      for (int c = 0; c < C; ++c) int8_encode<16>(f[c], s, inv, q[c]);
    }
    for (int j0 = 0; j0 < a.k; j0 += 64) {
      const int n = a.k - j0 < 64 ? a.k - j0 : 64;
      const int mine = (threadIdx.x & 63) < n ? (threadIdx.x & 63) : 0;
      const int rows = a.index[row * a.k + j0 + mine];
      const float weights = a.w ? a.w[row * a.k + j0 + mine] : 1.0f;
      for (int j = 0; j < n; ++j) {
        const int to = __builtin_amdgcn_readlane(rows, j);
        if ((unsigned)to >= (unsigned)a.n_rows) continue;
        if (a.w) {
          // rounding is monotone: the largest |w v| as rounded is |w| times the largest |v|, rounded
          const float wj = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(weights), j));
          s = int8_scale(fabsf(wj) * amax);
          const float winv = 1.0f / s;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = f[c][e] * wj;
            int8_encode<16>(v, s, winv, q[c]);
          }
        }
        if (lane == 0) a.s[to] = s;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int i = c * NTH + lane;
          if (i < per) store_codes(a.q + (long)to * a.H + 16L * i, q[c]);
        }
      }
    }
  }
}

// A grid has fewer than 2^32 threads (past that the runtime drops workgroups without a word):
// more rows take more launches.
template <class R, int MODE, int NTH, int C>
int launch_one(RowArgs a, hipStream_t s) {
  constexpr int kThreads = NTH <= 64 ? 256 : NTH, kRows = kThreads / NTH;
  constexpr long kMost = (1L << 31) / kThreads;
  const long groups = (a.T + kRows - 1L) / kRows;
  for (long g = 0; g < groups; g += kMost) {
    a.row0 = g * kRows;
    const long n = groups - g < kMost ? groups - g : kMost;
    hipLaunchKernelGGL((quant_int8<R, MODE, NTH, C>), dim3((unsigned)n), dim3(kThreads), 0, s, a);
    if (hipGetLastError() != hipSuccess) return FG_ELAUNCH;
  }
  return FG_OK;
}

template <class R, int MODE>
int launch_rows(const RowArgs& a, hipStream_t s) {
  const int per = a.H / 16;
  if constexpr (MODE != kDispatch) {
    if (per <= 8) return launch_one<R, MODE, 8, 1>(a, s);
    if (per <= 16) return launch_one<R, MODE, 16, 1>(a, s);
    if (per <= 32) return launch_one<R, MODE, 32, 1>(a, s);
  }
  if (per <= 64) return launch_one<R, MODE, 64, 1>(a, s);
  if (per <= 128) return launch_one<R, MODE, 128, 1>(a, s);
  if (per <= 256) return launch_one<R, MODE, 256, 1>(a, s);
  if (per <= 512) return launch_one<R, MODE, 256, 2>(a, s);
  if (per <= 1024) return launch_one<R, MODE, 256, 4>(a, s);
  return launch_one<R, MODE, 1024, 4>(a, s);
}

int check(int dtype, int T, int H) {
  return T < 0 || H < 16 || H % 16 || H > kMaxRow || (dtype != FG_BF16 && dtype != FG_FP32) ? FG_EINVAL : FG_OK;
}

template <int MODE>
int run(int dtype, const RowArgs& a, hipStream_t stream) {
  if (!a.x || !a.q || !a.s || !aligned(a.x, 16) || !aligned(a.q, 16) || !aligned(a.s, 4)) return FG_EINVAL;
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  return dtype == FG_BF16 ? launch_rows<RowBf16, MODE>(a, stream) : launch_rows<RowF32, MODE>(a, stream);
}

}  // namespace

extern "C" {

int fg_quant_int8(const void* x, int dtype, void* q, float* s, int M, int K, hipStream_t stream) {
  const int rc = check(dtype, M, K);
  if (rc != FG_OK || M == 0) return rc;
  return run<kRows>(dtype, RowArgs{x, nullptr, nullptr, static_cast<uint8_t*>(q), s, M, 1, K, M, 0}, stream);
}

int fg_dispatch_quant_int8(const void* x, int dtype, const int32_t* rows, const float* w, void* Q, float* s, int T,
                           int k, int H, int n_rows, hipStream_t stream) {
  const int rc = check(dtype, T, H);
  if (rc != FG_OK || k < 1 || n_rows < 0) return FG_EINVAL;
  if (T == 0 || n_rows == 0) return FG_OK;
  if (!rows || !aligned(rows, 4) || !aligned(w, 4)) return FG_EINVAL;
  return run<kDispatch>(dtype, RowArgs{x, rows, w, static_cast<uint8_t*>(Q), s, T, k, H, n_rows, 0}, stream);
}

int fg_swiglu_quant_int8(const void* h, int dtype, const int32_t* slots, void* Q, float* s, int rows, int I,
                         hipStream_t stream) {
  const int rc = check(dtype, rows, I);
  if (rc != FG_OK || I % 128) return FG_EINVAL;
  if (rows == 0) return FG_OK;
  if (!aligned(slots, 4)) return FG_EINVAL;
  return run<kSwiglu>(dtype, RowArgs{h, slots, nullptr, static_cast<uint8_t*>(Q), s, rows, 1, I, rows, 0}, stream);
}

}  // extern "C"
