// fg_int8_quot.hpp -- 8-bit integer codes and scales of rows, for the kernels that make
// the 8-bit integer product's operands.
#pragma once

#include "fg_e4m3_quot.hpp"
#include "fg_wave.hpp"

namespace fg {

// Scale of a row from the bits of its largest |v|: amax's own where that is infinite or
// NaN, so such a row shows in the product.
__device__ __forceinline__ float int8_scale(float amax) {
  return amax == 0.0f ? 1.0f : amax < 0x1p-126f * 127.0f ? 0x1p-126f : amax / 127.0f;
}

// Codes of N values: rint through the low byte of v / s + 1.5 * 2^23 (|v / s| < 128).
// The quotient is e4m3_quot's, which differs from the rounded one only within 2^-23 ulp
// of a middle of two floats; a code changes only where one of these is half an integer,
// and all such pairs were gone through (tests/test_int8_quotient.py).
__device__ __forceinline__ uint32_t byte4(float a, float b, float c, float d) {
  constexpr float kMagic = 12582912.0f;
  const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(b + kMagic), __float_as_uint(a + kMagic), 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(d + kMagic), __float_as_uint(c + kMagic), 0x0c0c0400u);
  return lo | (hi << 16);
}
template <int N>
__device__ __forceinline__ void int8_encode(const float* f, float s, float inv, uint32_t* q) {
  if (s >= kQuotMin) {
#pragma unroll
    for (int c = 0; c < N / 4; ++c)
      q[c] = byte4(e4m3_quot(f[4 * c], s, inv), e4m3_quot(f[4 * c + 1], s, inv), e4m3_quot(f[4 * c + 2], s, inv),
                   e4m3_quot(f[4 * c + 3], s, inv));
  } else {
#pragma unroll
    for (int c = 0; c < N / 4; ++c) q[c] = byte4(f[4 * c] / s, f[4 * c + 1] / s, f[4 * c + 2] / s, f[4 * c + 3] / s);
  }
}

// Largest |f| of N values as bits (a NaN's are above infinity's).
template <int N>
__device__ __forceinline__ uint32_t amax_bits(const float* f, uint32_t m) {
#pragma unroll
  for (int i = 0; i < N; ++i) m = umax(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}

}  // namespace fg
