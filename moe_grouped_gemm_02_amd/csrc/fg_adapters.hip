// fg_adapters.hip -- low-rank adapters of many requests at once beside a shared
// projection. Token t with adapter a gets
//
//     out[t] = D[t] + scale[a] * (x[t] A[a]^T) B[a]^T,   A [L][R][K], B [L][N][R],
//
// with x, A, B, D, out in bf16 and everything between in fp32. The tokens come
// sorted by adapter (a contiguous plan whose segments start at multiples of
// `align` rows), so a tile of rows has one adapter and both products run on the
// matrix cores.
//
// Two launches, because every output column needs the whole sum over K:
//   shrink  h = x A^T. A workgroup takes one tile of rows and one part of K, its
//           four waves a quarter of that part each; v_mfma_f32_16x16x32_bf16 on
//           fragments loaded straight from global memory (nothing is used twice
//           within a wave, so LDS would add only a copy). The waves' sums meet in
//           LDS, the parts' in the workspace, both added in a fixed order.
//   expand  out = D + h B^T. A workgroup takes one tile of rows and a strip of
//           columns; h is summed over the parts, scaled, and split into two bf16
//           (h = hi + lo to 2^-17) so that rounding it costs nothing visible:
//           the work is bound by the rows of D, not by the matrix cores. For
//           R <= 16 both halves fit one 32-deep MFMA, hi against k 0..15 and lo
//           against k 16..31 with B's fragment repeated.
//
// K order in a fragment: both operands of an MFMA may take their 32 k values in
// any common order; lane quarter q takes the 16 consecutive values at 16 q of a
// 64-wide step over two MFMAs, so a row's 64 values are one 128-byte line.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fg.h"
#include "fg_device.hpp"
#include "fg_wave.hpp"

namespace {

using namespace fg;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kMaxRank = 128;
constexpr int kStepK = 64;

struct AdapterArgs {
  const uint16_t *D, *x, *A, *B;
  const float* scales;
  const int32_t *rows, *slots, *m_indices;
  uint16_t* out;
  float* ws;              // [parts][cap][16 * TR]
  int T, L, R, K, N, cap;
  int parts;              // parts of K
  int strip;              // columns of one expand workgroup
  int tiles;              // row tiles
};

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

__device__ __forceinline__ f32x4v mfma(u32x4 a, u32x4 b, f32x4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

// TM: 16-row groups of a tile, TR: 16-column groups of the rank.
template <int TM, int TR>
__global__ __launch_bounds__(kThreads) void adapter_shrink(AdapterArgs p) {
  constexpr int RT = 16 * TM, RC = 16 * TR, RP = RC + 4;
  __shared__ float red[kWaves][RT][RP];
  const int tile = blockIdx.x, r0 = tile * RT;
  const int a = p.m_indices[r0];
  if ((unsigned)a >= (unsigned)p.L) return;   // no token in this tile (uniform)
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lrow = lane & 15, q = lane >> 4;

  // rows without a token repeat the tile's first one; their sums are not stored
  const int first = p.slots[r0];
  const uint16_t* xp[TM];
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int s = p.slots[r0 + 16 * m + lrow];
    const int tok = (unsigned)s < (unsigned)p.T ? s : (unsigned)first < (unsigned)p.T ? first : 0;
    xp[m] = p.x + (long)tok * p.K + 16 * q;
  }
  const uint16_t* ap[TR];
#pragma unroll
  for (int c = 0; c < TR; ++c) {
    const int r = 16 * c + lrow < p.R ? 16 * c + lrow : p.R - 1;
    ap[c] = p.A + ((long)a * p.R + r) * p.K + 16 * q;
  }
  const int steps = p.K / kStepK;
  const int lanes = p.parts * kWaves, me = blockIdx.y * kWaves + wave;
  const int s0 = (int)((long)steps * me / lanes), s1 = (int)((long)steps * (me + 1) / lanes);

  f32x4v acc[TR][TM];
#pragma unroll
  for (int c = 0; c < TR; ++c)
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[c][m] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int s = s0; s < s1; ++s) {
    u32x4 xf[TM][2], af[TR][2];
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      const u32x4* v = (const u32x4*)(xp[m] + (long)s * kStepK);
      xf[m][0] = v[0];
      xf[m][1] = v[1];
    }
#pragma unroll
    for (int c = 0; c < TR; ++c) {
      const u32x4* v = (const u32x4*)(ap[c] + (long)s * kStepK);
      af[c][0] = v[0];
      af[c][1] = v[1];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < TR; ++c)
#pragma unroll
        for (int m = 0; m < TM; ++m) acc[c][m] = mfma(af[c][h], xf[m][h], acc[c][m]);
  }
  // lane holds ranks 16 c + 4 q + v of row 16 m + lrow
#pragma unroll
  for (int c = 0; c < TR; ++c)
#pragma unroll
    for (int m = 0; m < TM; ++m) *(f32x4v*)&red[wave][16 * m + lrow][16 * c + 4 * q] = acc[c][m];
  __syncthreads();
  for (int i = tid; i < RT * RC / 4; i += kThreads) {
    const int row = i / (RC / 4), col = 4 * (i - row * (RC / 4));
    if ((unsigned)p.slots[r0 + row] >= (unsigned)p.T) continue;
    f32x4v sum = *(const f32x4v*)&red[0][row][col];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += *(const f32x4v*)&red[w][row][col];
    *(f32x4v*)(p.ws + ((long)blockIdx.y * p.cap + r0 + row) * RC + col) = sum;
  }
}

template <int TM, int TR>
__global__ __launch_bounds__(kThreads) void adapter_expand(AdapterArgs p) {
  constexpr int RT = 16 * TM, RC = 16 * TR;
  constexpr int KF = TR == 1 ? 1 : TR / 2;        // 32-deep fragments of the rank
  constexpr int HP = (TR == 1 ? 32 : RC) + 8;     // bf16 of one LDS row (+16 bytes against bank conflicts)
  constexpr int HL = TR == 1 ? 1 : 2;             // hi (and lo) planes
  __shared__ __attribute__((aligned(16))) uint16_t hs[HL][RT][HP];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lrow = lane & 15, q = lane >> 4;
  const int n_lo = blockIdx.y * p.strip, n_hi = n_lo + p.strip < p.N ? n_lo + p.strip : p.N;
  if ((int)blockIdx.x >= p.tiles) {
    // tokens without an adapter pass through (launched only where out is not D)
    const int t0 = ((int)blockIdx.x - p.tiles) * 16;
    for (int t = t0; t < t0 + 16 && t < p.T; ++t) {
      if ((unsigned)p.rows[t] < (unsigned)p.cap) continue;
      for (int n = n_lo + 8 * tid; n < n_hi; n += 8 * kThreads)
        *(u32x4*)(p.out + (long)t * p.N + n) = *(const u32x4*)(p.D + (long)t * p.N + n);
    }
    return;
  }
  const int r0 = blockIdx.x * RT;
  const int a = p.m_indices[r0];
  if ((unsigned)a >= (unsigned)p.L) return;
  const float scale = p.scales[a];
  for (int i = tid; i < RT * RC / 4; i += kThreads) {
    const int row = i / (RC / 4), col = 4 * (i - row * (RC / 4));
    f32x4v h = {0.f, 0.f, 0.f, 0.f};
    if ((unsigned)p.slots[r0 + row] < (unsigned)p.T && col < p.R) {
      for (int c = 0; c < p.parts; ++c) h += *(const f32x4v*)(p.ws + ((long)c * p.cap + r0 + row) * RC + col);
      h *= scale;
    }
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      hi[e] = bf16_pair(h[2 * e], h[2 * e + 1]);
      lo[e] = bf16_pair(h[2 * e] - bf16_lo(hi[e]), h[2 * e + 1] - bf16_hi(hi[e]));
    }
    *(u32x2v*)&hs[0][row][col] = u32x2v{hi[0], hi[1]};
    if (TR == 1) *(u32x2v*)&hs[0][row][16 + col] = u32x2v{lo[0], lo[1]};
    else *(u32x2v*)&hs[HL - 1][row][col] = u32x2v{lo[0], lo[1]};
  }
  __syncthreads();
  u32x4 hf[HL][KF][TM];
#pragma unroll
  for (int e = 0; e < HL; ++e)
#pragma unroll
    for (int f = 0; f < KF; ++f)
#pragma unroll
      for (int m = 0; m < TM; ++m) hf[e][f][m] = *(const u32x4*)&hs[e][16 * m + lrow][32 * f + 8 * q];
  int tok[TM];
#pragma unroll
  for (int m = 0; m < TM; ++m) tok[m] = p.slots[r0 + 16 * m + lrow];

  // Columns in pairs of 16-wide sub-tiles: sub-tile e's operand row i is column
  // 8 (i / 4) + 4 e + i % 4, so a lane's results of the pair are the eight
  // consecutive columns 8 q .. 8 q + 7 and D moves in 16-byte pieces.
  const uint16_t* Ba = p.B + (long)a * p.N * p.R;
  const int brow = 8 * (lrow >> 2) + (lrow & 3);
  for (int n0 = n_lo + 32 * wave; n0 < n_hi; n0 += 32 * kWaves) {
    u32x4 bf[2][KF];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int f = 0; f < KF; ++f) {
        const int n = n0 + brow + 4 * e;
        const int r = TR == 1 ? 8 * (q & 1) : 32 * f + 8 * q;
        bf[e][f] = n < p.N && r < p.R ? *(const u32x4*)(Ba + (long)n * p.R + r) : u32x4{0u, 0u, 0u, 0u};
      }
    const int col = n0 + 8 * q;
    u32x4 d[TM];
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      const bool ok = (unsigned)tok[m] < (unsigned)p.T && col < p.N;
      d[m] = ok ? *(const u32x4*)(p.D + (long)tok[m] * p.N + col) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      f32x4v acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int h = HL - 1; h >= 0; --h)   // the small halves first
#pragma unroll
        for (int f = 0; f < KF; ++f)
#pragma unroll
          for (int e = 0; e < 2; ++e) acc[e] = mfma(bf[e][f], hf[h][f][m], acc[e]);
      float v[8];
      RowBf16::unpack(d[m], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += acc[e >> 2][e & 3];
      if ((unsigned)tok[m] < (unsigned)p.T && col < p.N)
        *(u32x4*)(p.out + (long)tok[m] * p.N + col) = RowBf16::pack(v);
    }
  }
}

// 16-column groups of the rank as compiled: 1, 2, 4 or 8.
int rank_groups(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

// Rows of one tile: 64 where the plan's segments allow it, else 32 or 16.
int tile_rows(int align) { return align % 64 == 0 ? 64 : align % 32 == 0 ? 32 : 16; }

// Parts of K: enough workgroups to fill the chip, at least one step of K a wave.
int k_parts(int tiles, int K) {
  const int most = K / (kStepK * kWaves) > 1 ? K / (kStepK * kWaves) : 1;
  int parts = 1;
  while (parts < 8 && 2 * parts <= most && (long)tiles * parts < 512) parts *= 2;
  return parts;
}

int sizes(int R, int K, int cap, int align) {
  if (R < 8 || R % 8 || R > kMaxRank || K < 128 || K % 128 || K > (1 << 24) || align < 16 || align % 16 || cap < 0 ||
      cap % align)
    return FG_EINVAL;
  return FG_OK;
}

template <int TM, int TR>
void launch(const AdapterArgs& p, hipStream_t s) {
  hipLaunchKernelGGL((adapter_shrink<TM, TR>), dim3(p.tiles, p.parts), dim3(kThreads), 0, s, p);
}
template <int TM, int TR>
void launch_expand(const AdapterArgs& p, hipStream_t s) {
  const unsigned copies = p.out != p.D ? (unsigned)((p.T + 15L) / 16) : 0u;
  hipLaunchKernelGGL((adapter_expand<TM, TR>), dim3(p.tiles + copies, (p.N + p.strip - 1) / p.strip), dim3(kThreads), 0,
                     s, p);
}

template <int TM>
void launch_rank(const AdapterArgs& p, int tr, bool expand, hipStream_t s) {
  switch (tr) {
    case 1: expand ? launch_expand<TM, 1>(p, s) : launch<TM, 1>(p, s); break;
    case 2: expand ? launch_expand<TM, 2>(p, s) : launch<TM, 2>(p, s); break;
    case 4: expand ? launch_expand<TM, 4>(p, s) : launch<TM, 4>(p, s); break;
    default: expand ? launch_expand<TM, 8>(p, s) : launch<TM, 8>(p, s); break;
  }
}

}  // namespace

extern "C" {

int fg_adapters_workspace(int R, int K, int cap, int align, size_t* bytes) {
  if (!bytes || sizes(R, K, cap, align) != FG_OK) return FG_EINVAL;
  *bytes = (size_t)k_parts(cap / tile_rows(align), K) * cap * (16 * rank_groups(R)) * sizeof(float);
  return FG_OK;
}

int fg_adapters(const void* D, const void* x, const void* A, const void* B, const float* scales, const int32_t* rows,
                const int32_t* slots, const int32_t* m_indices, void* out, void* ws, int T, int L, int R, int K, int N,
                int cap, int align, hipStream_t stream) {
  if (T < 0 || L < 1 || N < 8 || N % 8 || N > (1 << 24) || sizes(R, K, cap, align) != FG_OK) return FG_EINVAL;
  if (T == 0) return FG_OK;
  if (cap < 1) return FG_EINVAL;   // a plan of T > 0 tokens has rows
  if (!D || !x || !A || !B || !scales || !rows || !slots || !m_indices || !out || !ws) return FG_EINVAL;
  if (!aligned(D, 16) || !aligned(x, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(out, 16) ||
      !aligned(ws, 16) || !aligned(scales, 4) || !aligned(rows, 4) || !aligned(slots, 4) || !aligned(m_indices, 4))
    return FG_EINVAL;
  const int st = current_device(nullptr);
  if (st != FG_OK) return st;
  AdapterArgs p = {};
  p.D = static_cast<const uint16_t*>(D);
  p.x = static_cast<const uint16_t*>(x);
  p.A = static_cast<const uint16_t*>(A);
  p.B = static_cast<const uint16_t*>(B);
  p.scales = scales;
  p.rows = rows;
  p.slots = slots;
  p.m_indices = m_indices;
  p.out = static_cast<uint16_t*>(out);
  p.ws = static_cast<float*>(ws);
  p.T = T;
  p.L = L;
  p.R = R;
  p.K = K;
  p.N = N;
  p.cap = cap;
  const int rt = tile_rows(align), tr = rank_groups(R);
  p.tiles = cap / rt;
  p.parts = k_parts(p.tiles, K);
  // columns of an expand workgroup: long strips read h once for more of D, short ones fill the chip
  p.strip = 1024;
  while (p.strip > 128 && (long)p.tiles * ((N + p.strip - 1) / p.strip) < 512) p.strip /= 2;
  for (int e = 0; e < 2; ++e) {
    if (rt == 64) launch_rank<4>(p, tr, e, stream);
    else if (rt == 32) launch_rank<2>(p, tr, e, stream);
    else launch_rank<1>(p, tr, e, stream);
    if (hipGetLastError() != hipSuccess) return FG_ELAUNCH;
  }
  return FG_OK;
}

}  // extern "C"
