// fg_wave.hpp -- device helpers of the row operators (routing, sorting, row
// movement, adapters): reductions over 64-lane waves on the VALU's cross-lane
// path (DPP, no LDS round trip) and bf16 <-> fp32 rows in 16-byte pieces.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fg {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

// DPP controls: lane permutations inside quads and 16-lane rows, and the two
// row broadcasts that carry a row's last lane into the following rows.
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
constexpr int kBcast15 = 0x142, kBcast31 = 0x143;

// The lane's partner value under a DPP control; rows outside ROWS get 0.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, ROWS == 0xf);
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(dpp_u32<CTRL, ROWS>(__float_as_uint(v)));
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Reductions over each group of 16 lanes or over the wave (L = 16 or 64), the
// result in every lane of the group; sums in a fixed order.
template <int L>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t v) {
  v = umax(v, dpp_u32<kQuadXor1>(v));
  v = umax(v, dpp_u32<kQuadXor2>(v));
  v = umax(v, dpp_u32<kHalfMirror>(v));
  v = umax(v, dpp_u32<kMirror>(v));
  if (L == 64) {
    v = umax(v, dpp_u32<kBcast15, 0xa>(v));
    v = umax(v, dpp_u32<kBcast31, 0xc>(v));
    v = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
  }
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  v += dpp_f32<kQuadXor1>(v);
  v += dpp_f32<kQuadXor2>(v);
  v += dpp_f32<kHalfMirror>(v);
  v += dpp_f32<kMirror>(v);
  if (L == 64) {
    v += dpp_f32<kBcast15, 0xa>(v);
    v += dpp_f32<kBcast31, 0xc>(v);
    v = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
  }
  return v;
}
__device__ __forceinline__ float wave_sum(float v) { return group_sum<64>(v); }

// Largest value over each group of eight lanes, for values >= 0.
__device__ __forceinline__ float group8_max(float v) {
  v = fmaxf(v, dpp_f32<kQuadXor1>(v));
  v = fmaxf(v, dpp_f32<kQuadXor2>(v));
  return fmaxf(v, dpp_f32<kHalfMirror>(v));
}

// An order-preserving unsigned image of a float that is not NaN: a < b as
// floats exactly when image(a) < image(b); -0 and +0 share one image, and no
// float has image 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);   // -0 + 0 = +0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Two floats as a pair of bf16 (round to nearest even, NaN stays NaN): the
// gfx950 conversion instruction.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  bf16x2 v;
  v.x = (__bf16)a;
  v.y = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

// A 16-byte store, past the caches where STREAM. (A template: the two sides of a branch
// become one ordinary store.) Outputs larger than the L2s together (32 MB) go that way:
// no reader finds them there, and a kernel that leaves the L2s full of them makes the
// next one wait for the write-back. Ordinary / past the caches, calls one after another:
// on new inputs and outputs each time, combine of T 8192, k 4, N 7168 118.8 / 114.6 us,
// adapters of T 8192, N 4096 73-79 / 72-75 us. Into the same output again and again,
// which the 256 MB last-level cache then keeps, it is the other way: 110.2 / 115 and
// 67 / 68.6 us; a call alone 130 / 135 and 93 / 98 us.
template <bool STREAM>
__device__ __forceinline__ void store16(u32x4* p, u32x4 v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}
constexpr long long kStreamBytes = 32ll << 20;

// A 16-byte load, past the caches where STREAM.
template <bool STREAM>
__device__ __forceinline__ u32x4 load16b(const u32x4* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  else return *p;
}

// Element types of activations: 16 bytes of a row at a time.
struct RowBf16 {
  static constexpr int kPer16 = 8;   // elements in 16 bytes
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ void unpack(u32x4 r, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(r[i]);
      f[2 * i + 1] = bf16_hi(r[i]);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = bf16_pair(f[2 * i], f[2 * i + 1]);
    return r;
  }
  static __device__ __forceinline__ float load1(const void* p, long i) {
    return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  }
  static __device__ __forceinline__ void store1(void* p, long i, float f) {
    ((uint16_t*)p)[i] = (uint16_t)bf16_pair(f, f);
  }
};
struct RowF32 {
  static constexpr int kPer16 = 4;
  static constexpr int kBytes = 4;
  static __device__ __forceinline__ void unpack(u32x4 r, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(r[i]);
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(f[i]);
    return r;
  }
  static __device__ __forceinline__ float load1(const void* p, long i) { return ((const float*)p)[i]; }
  static __device__ __forceinline__ void store1(void* p, long i, float f) { ((float*)p)[i] = f; }
};

}  // namespace fg
