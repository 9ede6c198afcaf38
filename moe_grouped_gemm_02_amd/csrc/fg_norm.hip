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
//     dR = dr + rx (z - rh mean(z rh)),  z = dh pre;          dx = alpha dR (dR without y)
//     dy = ry (v - yh mean(v yh)),       v = beta g post dR   (dy = v without post)
//     dpre = sum_t dh rh,   S = sum_t dR yh (times the token's gate)
//     dpost = beta g S,     dgate = beta post S  per channel, beta sum_n dR yh post per token
//
// Everything is fp32 between the loads and the stores. All is bound by memory traffic:
// a workgroup holds a row in registers (units of 8 elements a lane) through its sums and
// walks the rows with its columns' weights kept in registers too -- the post norm's
// weight, the channel's gate and beta fold into one -- so each row is read once, and the
// gradient's column sums S and sum dh rh stay in registers until a workgroup's rows are
// done; a second kernel adds the workgroups' sums in a fixed order. The next row is on its
// way while this one goes through its barriers. Measured, T 8192, N 7168, bf16: forward to
// E4M3 84-86 us (4.9 TB/s; a row a workgroup at a time 108), as integers 83, in bf16 92-94, without y
// 41, 37 and 47; gradient 140 + 6.5 us (4.8 TB/s; without the row ahead, rows as floats 200 + 27). T 32
// forward 4.2 us, latency. T 1001, N 2048, fp32, gradient 12.8 + 3.9.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fg.h"
#include "fg_device.hpp"
#include "fg_int8_quot.hpp"

namespace {

using namespace fg;

constexpr int kMaxCols = 16384;   // 1024 threads of 2 units
constexpr int kCUs = 256;
constexpr int kNontemporal = 2;   // of a buffer access
constexpr int kNoUnit = 1 << 24;  // of a row: past its end

struct NormArgs {
  const void *x, *y;
  const float *pre, *post, *gate;
  void *r, *h;
  float* s;
  int T, N, rows, gate_kind, out;   // rows: of a workgroup, one after another
  float alpha, beta, eps, inv_n;
};

// A row (or a vector of weights) of n bytes as a buffer: lanes past its end load zeros,
// which add nothing to any sum, and store nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void* base, long byte, int n) {
  return __builtin_amdgcn_make_buffer_rsrc((char*)base + byte, 0, n, 0x20000);
}
// Unit i of it, 8 elements, as loaded and as floats. (Rows wait in registers as loaded:
// bf16 takes half the room that way.) STREAM: past the caches, for batches that do not
// fit them (kStreamBytes): T 8192, N 7168, bf16 93 -> 86 us forward, 155 -> 152 back.
template <class R, bool STREAM = false>
struct Unit {
  u32x4 raw[8 / R::kPer16];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t row, int i) {
#pragma unroll
    for (int c = 0; c < 8 / R::kPer16; ++c)
      raw[c] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(row, i * 8 * R::kBytes + 16 * c, 0, STREAM ? kNontemporal : 0));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int c = 0; c < 8 / R::kPer16; ++c) raw[c] = u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void unpack(float* f) const {
#pragma unroll
    for (int c = 0; c < 8 / R::kPer16; ++c) R::unpack(raw[c], f + c * R::kPer16);
  }
};
template <class R, bool STREAM = false>
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t row, int i, const float* f) {
#pragma unroll
  for (int c = 0; c < 8 / R::kPer16; ++c)
    __builtin_amdgcn_raw_buffer_store_b128(R::pack(f + c * R::kPer16), row, i * 8 * R::kBytes + 16 * c, 0,
                                           STREAM ? kNontemporal : 0);
}
// 8 weights of the lane's columns, `other` where there is no such vector.
__device__ __forceinline__ void weights8(const float* w, int n, int i, float other, float* f) {
  if (w) {
    Unit<RowF32> u;
    u.load(row_of(w, 0, n * 4), i);
    u.unpack(f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = other;
  }
}

// Short rows: a wave has 64 / L of them side by side, L lanes each (16 for up to 128 columns, 32
// for up to 256), and its sums and largest values are those of L lanes. T 65536, N 128, bf16, 1 / 4
// rows a wave: 13.2 / 6.9 us, with y 22.1 / 11.7, N 256, 1 / 2 rows 13.9 / 11.5, with y 28.7 / 25.3.
template <int L>
__device__ __forceinline__ float row_sum(float v) {
  if constexpr (L == 64) return wave_sum(v);
  v = group_sum<16>(v);
  if constexpr (L == 32) v += __shfl_xor(v, 16);
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
  if constexpr (L == 64) return group_max_u32<64>(m);
  m = group_max_u32<16>(m);
  if constexpr (L == 32) m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
  return m;
}

// Sums over the workgroup (or over a short row's L lanes), the same in every thread, in a fixed
// order. The slots of two calls in a row differ, so one barrier a call is enough.
template <int NTH, int V, int L = 64>
struct BlockSum {
  float (*part)[V][NTH / 64];
  int slot = 0;
  __device__ __forceinline__ void operator()(float* v) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = row_sum<L>(v[i]);
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

// Y: with a block's output.
template <class R, int NTH, int C, int L, bool Y, bool STREAM>
__global__ __launch_bounds__(NTH) void block_norm(NormArgs a) {
  static_assert(L == 64 || (NTH == 64 && C == 1), "short rows: a wave a workgroup");
  constexpr int kRows = 64 / L;   // a step's rows
  __shared__ float part[2][1][NTH / 64];
  __shared__ uint32_t top[2][NTH / 64];
  const int lane = L < 64 ? threadIdx.x % L : threadIdx.x, below = L < 64 ? threadIdx.x / L : 0, per = a.N >> 3;
  BlockSum<NTH, 1, L> sum{part};
  // the lane's unit c of a step's rows, which follow one another in memory
  auto unit = [&](int c) { return L == 64 ? c * NTH + lane : lane < per ? below * per + lane : kNoUnit; };
  float cw[C][8], pre[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * NTH + lane;
    weights8(a.pre, a.N, i, 0.0f, pre[c]);
    if (Y) {
      float g[8];
      weights8(a.post, a.N, i, 1.0f, cw[c]);
      weights8(a.gate_kind == FG_GATE_CHANNEL ? a.gate : nullptr, a.N, i, 1.0f, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) cw[c][e] *= g[e] * a.beta;
    }
  }
  int flip = 0;
  auto rows_at = [&](const void* base, long t, int bytes) {   // one step's rows
    return row_of(base, t * bytes, L == 64 ? bytes : (int)(a.T - t < kRows ? a.T - t : kRows) * bytes);
  };
  const int bytes = a.N * R::kBytes;
  const long t0 = (long)blockIdx.x * a.rows, t1 = t0 + a.rows < a.T ? t0 + a.rows : a.T;
  Unit<R, STREAM> nx[C], ny[C];   // the next row, on its way
  auto fetch = [&](long t) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      nx[c].load(rows_at(a.x, t, bytes), unit(c));
      if (Y) ny[c].load(rows_at(a.y, t, bytes), unit(c));
    }
  };
  fetch(t0);
  for (long t = t0; t < t1; t += kRows) {
    const long mine = t + below;   // the lane's row
    Unit<R, STREAM> x[C], y[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      x[c] = nx[c];
      y[c] = ny[c];
    }
    if (t + kRows < t1) fetch(t + kRows);
    float r[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) x[c].unpack(r[c]);
    if (Y) {
      float k = a.gate_kind == FG_GATE_TOKEN && mine < a.T ? a.gate[mine] : 1.0f;
      if (a.post) {
        float v[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float f[8];
          y[c].unpack(f);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[0] = fmaf(f[e], f[e], v[0]);
        }
        sum(v);
        k *= rstd_of(v[0], a.inv_n, a.eps);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float f[8];
        y[c].unpack(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[c][e] = fmaf(f[e] * k, cw[c][e], a.alpha * r[c][e]);
        store8<R, STREAM>(rows_at(a.r, t, bytes), unit(c), r[c]);
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
    const __amdgpu_buffer_rsrc_t codes = rows_at(a.h, t, a.N);   // 8-bit outputs
    if (a.out == FG_OUT_SAME) {
#pragma unroll
      for (int c = 0; c < C; ++c) store8<R, STREAM>(rows_at(a.h, t, bytes), unit(c), r[c]);
    } else if (a.out == FG_OUT_INT8) {
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) m = amax_bits<8>(r[c], m);
      m = row_max<L>(m);
      if constexpr (NTH > 64) {
        if ((lane & 63) == 0) top[flip][lane >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NTH / 64; ++w) m = umax(m, top[flip][w]);
        flip ^= 1;
      }
      const float s = int8_scale(__uint_as_float(m)), inv = 1.0f / s;
      if (lane == 0 && mine < a.T) a.s[mine] = s;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        uint32_t q[2];
        int8_encode<8>(r[c], s, inv, q);
        __builtin_amdgcn_raw_buffer_store_b64(u32x2v{q[0], q[1]}, codes, unit(c) * 8, 0, STREAM ? kNontemporal : 0);
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
        __builtin_amdgcn_raw_buffer_store_b64(q, codes, unit(c) * 8, 0, STREAM ? kNontemporal : 0);
        if (i < per && mine < a.T && (lane & 15) == 0) a.s[(long)(i >> 4) * a.T + mine] = s;
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
  int T, N, rows, gate_kind;
  float alpha, beta, eps, inv_n;
};

// LEAN: rows of more than 8192, whose 1024 threads have 128 registers each: the weights are
// read again for each row (from the L2), the columns' sums are kept in LDS (each thread its
// own, no barrier), and fp32 rows are not fetched ahead. T 4096, N 16384 bf16 / fp32 245 / 594
// us with the sums in registers (which spill), 184 / 375 so.
template <class R, int NTH, int C, int L, bool LEAN, bool STREAM>
__global__ __launch_bounds__(NTH) void block_norm_grad(GradArgs a) {
  static_assert(L == 64 || (NTH == 64 && C == 1 && !LEAN), "short rows: a wave a workgroup");
  constexpr int kRows = 64 / L;   // a step's rows
  __shared__ float part3[2][3][NTH / 64], part1[2][1][NTH / 64];
  const int lane = L < 64 ? threadIdx.x % L : threadIdx.x, below = L < 64 ? threadIdx.x / L : 0, per = a.N >> 3;
  BlockSum<NTH, 3, L> sum3{part3};
  BlockSum<NTH, 1, L> sum1{part1};
  auto unit = [&](int c) { return L == 64 ? c * NTH + lane : lane < per ? below * per + lane : kNoUnit; };
  constexpr bool AHEAD = !LEAN || R::kBytes == 2;
  constexpr int kSums = LEAN ? C * 2 * NTH : 1;   // in pieces of four columns
  __shared__ f32x4v lds_sums[2][kSums];
  float cw[LEAN ? 1 : C][8], pre[LEAN ? 1 : C][8], P[LEAN ? 1 : C][8], S[LEAN ? 1 : C][8];
  // adds v to the sums of the lane's columns: P (which = 0) or S
  auto add_sums = [&](int which, float (*reg)[8], int c, const float* v) {
    if constexpr (LEAN) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f32x4v& at = lds_sums[which][(c * 2 + h) * NTH + lane];
        at += f32x4v{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) reg[c][e] += v[e];
    }
  };
  auto read_pre = [&](int c) { weights8(a.pre, a.N, c * NTH + lane, 0.0f, pre[LEAN ? 0 : c]); };
  auto read_cw = [&](int c) {
    float g[8], *w = cw[LEAN ? 0 : c];
    weights8(a.post, a.N, c * NTH + lane, 1.0f, w);
    weights8(a.gate_kind == FG_GATE_CHANNEL ? a.gate : nullptr, a.N, c * NTH + lane, 1.0f, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= g[e] * a.beta;
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (!LEAN) {
      read_pre(c);
      read_cw(c);
    }
    if constexpr (LEAN) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        lds_sums[0][(c * 2 + h) * NTH + lane] = lds_sums[1][(c * 2 + h) * NTH + lane] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) P[c][e] = S[c][e] = 0.0f;
    }
  }
  const int bytes = a.N * R::kBytes;
  auto rows_at = [&](const void* base, long t) {   // one step's rows
    return row_of(base, t * bytes, L == 64 ? bytes : (int)(a.T - t < kRows ? a.T - t : kRows) * bytes);
  };
  const long t0 = (long)blockIdx.x * a.rows, t1 = t0 + a.rows < a.T ? t0 + a.rows : a.T;
  Unit<R, STREAM> nr[C], nh[C], nd[C], ny[C];   // the next row, on its way
#pragma unroll
  for (int c = 0; c < C; ++c) nd[c].zero();
  auto fetch = [&](long t) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = unit(c);
      if (a.pre) {
        nr[c].load(rows_at(a.r, t), i);
        nh[c].load(rows_at(a.dh, t), i);
      }
      if (a.y) ny[c].load(rows_at(a.y, t), i);
      if (a.dr) nd[c].load(rows_at(a.dr, t), i);
    }
  };
  if (AHEAD) fetch(t0);
  for (long t = t0; t < t1; t += kRows) {
    const long mine = t + below;   // the lane's row
    Unit<R, STREAM> r[C], dh[C], y[C];
    float d[C][8];
    if (!AHEAD) fetch(t);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      r[c] = nr[c];
      dh[c] = nh[c];
      y[c] = ny[c];
      nd[c].unpack(d[c]);
    }
    if (AHEAD && t + kRows < t1) fetch(t + kRows);
    float v[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[8], g[8];
      if (a.pre) {
        if (LEAN) read_pre(c);
        r[c].unpack(f);
        dh[c].unpack(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[0] = fmaf(f[e], f[e], v[0]);
          v[1] = fmaf(g[e] * pre[LEAN ? 0 : c][e], f[e], v[1]);
        }
      }
      if (a.post) {
        y[c].unpack(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[2] = fmaf(f[e], f[e], v[2]);
      }
    }
    if (a.pre || a.post) sum3(v);
    if (a.pre) {
      const float rx = rstd_of(v[0], a.inv_n, a.eps);
      const float m = v[1] * rx * a.inv_n;   // mean of z rh
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float f[8], g[8], s[8];
        if (LEAN) read_pre(c);
        r[c].unpack(f);
        dh[c].unpack(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float rh = f[e] * rx;
          d[c][e] = fmaf(rx, fmaf(-rh, m, g[e] * pre[LEAN ? 0 : c][e]), d[c][e]);
          s[e] = g[e] * rh;
        }
        add_sums(0, P, c, s);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = a.alpha * d[c][e];
      store8<R, STREAM>(rows_at(a.dx, t), unit(c), o);
    }
    if (!a.y) continue;
    const float ry = a.post ? rstd_of(v[2], a.inv_n, a.eps) : 1.0f;
    const float gt = a.gate_kind == FG_GATE_TOKEN && mine < a.T ? a.gate[mine] : 1.0f;
    float q[1] = {0.0f};   // sum of dR yh, times the folded weights
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[8], s[8];
      if (LEAN) read_cw(c);
      y[c].unpack(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float yh = f[e] * ry;
        s[e] = gt * d[c][e] * yh;
        d[c][e] *= cw[LEAN ? 0 : c][e];
        q[0] = fmaf(d[c][e], yh, q[0]);
      }
      add_sums(1, S, c, s);
    }
    if (a.post || a.gate_kind == FG_GATE_TOKEN) sum1(q);
    if (a.gate_kind == FG_GATE_TOKEN && lane == 0 && mine < a.T) a.dgate[mine] = q[0];
    const float m = a.post ? q[0] * a.inv_n : 0.0f, k = ry * gt;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[8], o[8];
      y[c].unpack(f);
#pragma unroll   // without post m is 0, and an infinite y would make NaN of it
      for (int e = 0; e < 8; ++e) o[e] = k * (a.post ? fmaf(-f[e] * ry, m, d[c][e]) : d[c][e]);
      store8<R, STREAM>(rows_at(a.dy, t), unit(c), o);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = LEAN ? lds_sums[which][LEAN ? (c * 2 + e / 4) * NTH + lane : 0][e % 4] : (which ? S : P)[LEAN ? 0 : c][e];
#pragma unroll
      for (int d = L; d < 64; d *= 2)   // the rows that were side by side; their lanes then store the same
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += __shfl_xor(v[e], d);
      store8<RowF32>(row_of(a.ws, ((long)blockIdx.x * 2 + which) * 4 * a.N, a.N * 4), c * NTH + lane, v);
    }
}

// The workgroups' sums added up in a fixed order: 16 columns of P or of S a workgroup, 64
// threads a column.
struct SumArgs {
  const float *ws, *post, *gate;
  float *dpre, *dpost, *dgate;   // null: not asked for
  int groups, N;
  float beta;
};
constexpr int kSumCols = 16, kSumParts = 64;
__global__ __launch_bounds__(kSumCols * kSumParts) void block_norm_sums(SumArgs a) {
  __shared__ float part[kSumParts][kSumCols + 1];
  const bool of_s = blockIdx.y != 0;
  if (of_s ? !a.dpost && !a.dgate : !a.dpre) return;
  const int col = threadIdx.x % kSumCols, p = threadIdx.x / kSumCols;
  const int n = blockIdx.x * kSumCols + col, at = n < a.N ? n : 0;
  const float* w = a.ws + (of_s ? a.N : 0) + at;
  float s = 0.0f;
#pragma unroll 8
  for (int g = p; g < a.groups; g += kSumParts) s += w[(long)g * 2 * a.N];
  part[p][col] = s;
  __syncthreads();
  if (p >= 4) return;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < kSumParts / 4; ++k) s += part[p * (kSumParts / 4) + k][col];
  // four lanes of the first wave have a column's quarters, 16 lanes apart
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  if (p != 0 || n >= a.N) return;
  if (!of_s) a.dpre[n] = s;
  const bool rows = a.groups > 0;   // without rows zeros, infinite weights or not
  if (of_s && a.dpost) a.dpost[n] = rows ? a.beta * (a.gate ? a.gate[n] : 1.0f) * s : 0.0f;
  if (of_s && a.dgate) a.dgate[n] = rows ? a.beta * (a.post ? a.post[n] : 1.0f) * s : 0.0f;
}

// Threads of a workgroup and rows it takes one after another, for T rows of N columns: as
// many workgroups as are resident together, so each has a run of neighbouring rows (whose
// E4M3 scales are neighbours in memory and meet in one XCD's L2).
// Half of a workgroup's lanes idle cost up to a third: 8192 x 640 bf16 on 256 / 128 threads 9.2 / 6.4 us,
// with y 14.4 / 10.0, gradient 29.8 / 20.9; 192 threads for 1152 columns gain 6-15% without y, nothing else.
int norm_threads(int N) { return N <= 512 ? 64 : N <= 1024 ? 128 : N <= 2048 ? 256 : N <= 8192 ? 512 : 1024; }
int step_rows(int N) { return N <= 128 ? 4 : N <= 256 ? 2 : 1; }   // 64 / L
int norm_rows(int T, int N, bool y) {
  const int most = kCUs * ((y ? 1024 : 1536) / norm_threads(N)), n = step_rows(N);
  const long long steps = ((long long)T + n - 1) / n;
  return n * (int)((steps + most - 1) / most);
}
// The gradient's workgroups each write their sums and the second kernel reads them, 16 bytes a
// column against a row's 10 (bf16) to 20: batches of some size take two or four steps a workgroup
// at least. us, 1 (or as the most workgroups give) / 2 / 4 steps, bf16: 200 x 2048 8.8 / 8.2 / 9.0,
// 200 x 7168 20.2 / 16.5 / 16.7, 512 x 1024 9.9 / 9.1 / 10.3, 1001 x 2048 18.4 / 18.3 / 14.3, 2048 x 512
// 17.3 / 12.6 / 11.3; 2 / 4: 8192 x 256 15.6 / 13.8, 8192 x 64 8.2 / 9.2.
int grad_rows(int T, int N) {
  const int most = kCUs * (N <= 2048 ? 512 / norm_threads(N) : 1);
  const int n = step_rows(N);
  const long long steps = ((long long)T + n - 1) / n;
  const int each = (int)((steps + most - 1) / most);
  const int least = steps >= (N > 256 ? 640 : 4096) ? 4 : steps >= (N > 512 ? 192 : 1024) ? 2 : 1;
  return n * (each > least ? each : least);
}
int grad_groups(int T, int N) { return (int)(((long long)T + grad_rows(T, N) - 1) / grad_rows(T, N)); }

template <class R>
bool streams(int T, int N) { return (long long)T * N * R::kBytes > kStreamBytes; }

template <class R, int NTH, int C, int L = 64>
int launch_norm(NormArgs a, hipStream_t s) {
  a.rows = norm_rows(a.T, a.N, a.y != nullptr);
  const dim3 g((unsigned)(((long long)a.T + a.rows - 1) / a.rows)), b(NTH);
  const bool stream = streams<R>(a.T, a.N);
  if (a.y && stream) hipLaunchKernelGGL((block_norm<R, NTH, C, L, true, true>), g, b, 0, s, a);
  else if (a.y) hipLaunchKernelGGL((block_norm<R, NTH, C, L, true, false>), g, b, 0, s, a);
  else if (stream) hipLaunchKernelGGL((block_norm<R, NTH, C, L, false, true>), g, b, 0, s, a);
  else hipLaunchKernelGGL((block_norm<R, NTH, C, L, false, false>), g, b, 0, s, a);
  return hipGetLastError() == hipSuccess ? FG_OK : FG_ELAUNCH;
}
template <class R>
int launch_norm_of(const NormArgs& a, hipStream_t s) {
  if (a.N <= 128) return launch_norm<R, 64, 1, 16>(a, s);
  if (a.N <= 256) return launch_norm<R, 64, 1, 32>(a, s);
  if (a.N <= 512) return launch_norm<R, 64, 1>(a, s);
  if (a.N <= 1024) return launch_norm<R, 128, 1>(a, s);
  if (a.N <= 2048) return launch_norm<R, 256, 1>(a, s);
  if (a.N <= 4096) return launch_norm<R, 512, 1>(a, s);
  if (a.N <= 8192) return launch_norm<R, 512, 2>(a, s);
  return launch_norm<R, 1024, 2>(a, s);
}

template <class R, int NTH, int C, int L = 64, bool LEAN = false>
int launch_grad(GradArgs a, hipStream_t s) {
  a.rows = grad_rows(a.T, a.N);
  const dim3 g(grad_groups(a.T, a.N)), b(NTH);
  if (streams<R>(a.T, a.N)) hipLaunchKernelGGL((block_norm_grad<R, NTH, C, L, LEAN, true>), g, b, 0, s, a);
  else hipLaunchKernelGGL((block_norm_grad<R, NTH, C, L, LEAN, false>), g, b, 0, s, a);
  return hipGetLastError() == hipSuccess ? FG_OK : FG_ELAUNCH;
}
template <class R>
int launch_grad_of(const GradArgs& a, hipStream_t s) {
  if (a.N <= 128) return launch_grad<R, 64, 1, 16>(a, s);
  if (a.N <= 256) return launch_grad<R, 64, 1, 32>(a, s);
  if (a.N <= 512) return launch_grad<R, 64, 1>(a, s);
  if (a.N <= 1024) return launch_grad<R, 128, 1>(a, s);
  if (a.N <= 2048) return launch_grad<R, 256, 1>(a, s);
  if (a.N <= 4096) return launch_grad<R, 512, 1>(a, s);
  if (a.N <= 8192) return launch_grad<R, 512, 2>(a, s);
  return launch_grad<R, 1024, 2, 64, true>(a, s);
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
  if (y && pre && r == h) return FG_EINVAL;   // two outputs
  if (pre && out != FG_OUT_SAME && (h == x || h == y)) return FG_EINVAL;   // codes lie over other rows
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(r, 16) || !aligned(h, 16) || !aligned(pre, 4) || !aligned(post, 4) ||
      !aligned(gate, 4) || !aligned(s, 4))
    return FG_EINVAL;
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  const NormArgs a = {x, y, pre, post, gate, r, h, s, T, N, 1, gate_kind, out, alpha, beta, eps, 1.0f / (float)N};
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
    if ((gate_kind != FG_GATE_NONE) != (gate != nullptr) || (gate && !dgate) || dx == dy) return FG_EINVAL;
  }
  if (!aligned(r, 16) || !aligned(dh, 16) || !aligned(dr, 16) || !aligned(y, 16) || !aligned(dx, 16) || !aligned(dy, 16) ||
      !aligned(pre, 4) || !aligned(post, 4) || !aligned(gate, 4) || !aligned(dgate, 4) || !aligned(dpre, 4) ||
      !aligned(dpost, 4) || !aligned(ws, 16))
    return FG_EINVAL;
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  if (T > 0) {
    const GradArgs a = {r, dh, dr, y, pre, post, gate, dx, dy, dgate, static_cast<float*>(ws), T, N, 1, gate_kind,
                        y ? alpha : 1.0f, beta, eps, 1.0f / (float)N};   // without y the stream is x itself
    const int rc = dtype == FG_BF16 ? launch_grad_of<RowBf16>(a, stream) : launch_grad_of<RowF32>(a, stream);
    if (rc != FG_OK) return rc;
  }
  if (!sums) return FG_OK;
  const SumArgs b = {static_cast<const float*>(ws), post, channel ? gate : nullptr, pre ? dpre : nullptr,
                     post ? dpost : nullptr, channel ? dgate : nullptr, grad_groups(T, N), N, beta};
  hipLaunchKernelGGL(block_norm_sums, dim3((N + kSumCols - 1) / kSumCols, 2), dim3(kSumCols * kSumParts), 0, stream, b);
  return hipGetLastError() == hipSuccess ? FG_OK : FG_ELAUNCH;
}

}  // extern "C"
