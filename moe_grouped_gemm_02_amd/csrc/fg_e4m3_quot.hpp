// fg_e4m3_quot.hpp -- E4M3 codes of x / s without the IEEE division, for kernels
// that encode many blocks per byte they move (the row operators).
#pragma once

#include "fg_e4m3.hpp"

namespace fg {

// Codes of four values of a block whose scale s = amax / 448 and its correctly
// rounded reciprocal inv are given: the same codes as e4m3x4_div at a third of its
// instructions (an IEEE division takes about ten).
//
// q = x inv is within 2 ulp of x / s. One step q' = q + (x - q s) inv, the residual
// exact by FMA, leaves x / s + d with |d| < 2^-23 ulp before its rounding, so q' can
// differ from the rounded quotient only where x / s lies that close to the middle of
// two floats, and the codes only where one of these floats is a boundary between
// codes, which has at most 5 significant bits. That needs s within 8 units of a value
// of 4 significant bits, from either side; all such cases were gone through in exact
// arithmetic and give the rounded quotient (tests/test_e4m3_quotient.py). The residual
// is exact while s >= 2^-90 (kQuotMin) for every x whose code is not zero; below that
// the caller divides. The residual is taken as q s - x, which keeps the sign of a zero.
//
// The quotients are not clamped to +-448 as in e4m3x4_div: where amax / 448 was rounded
// down, amax / s is the float above 448 (6 to 8 blocks of 100), never more (every
// significand of amax was gone through), and its code is 448's all the same.
constexpr float kQuotMin = 8.0779357e-28f;   // 2^-90
__device__ __forceinline__ float e4m3_quot(float x, float s, float inv) {
  const float q = x * inv;
  return fmaf(-fmaf(q, s, -x), inv, q);
}
__device__ __forceinline__ uint32_t e4m3x4_quot(float x0, float x1, float x2, float x3, float s, float inv) {
  const uint32_t lo = e4m3_pk<false>(e4m3_quot(x0, s, inv), e4m3_quot(x1, s, inv), 0u);
  return e4m3_pk<true>(e4m3_quot(x2, s, inv), e4m3_quot(x3, s, inv), lo);
}

}  // namespace fg
