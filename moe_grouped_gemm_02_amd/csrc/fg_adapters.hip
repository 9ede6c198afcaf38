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
//   shrink  h = x A^T. A workgroup takes one tile of rows and one part of K; the
//           parts' sums meet in the workspace and are added in a fixed order.
//   expand  out = D + h B^T. A workgroup takes one tile of rows and a strip of
//           columns; h is summed over the parts, scaled, and cut into three bf16 of
//           eight bits each, which hold all 24 bits of it: the work is bound by moving
//           D, not by the matrix cores (T 8192, N 4096, R 64: 39.6 us, 39.1 with two
//           pieces, whose 17 bits let 0.16% of the outputs miss the correctly rounded
//           bf16; with three it is 0.02%). For R <= 16 the two lower pieces fit one
//           32-deep MFMA, one against k 0..15 and one against k 16..31 with B's
//           fragment repeated.
// Each has a kernel for 16-row tiles (decode), where A and B are read once and go
// straight into fragments, and one for 64-row tiles (prompts), where four waves share
// them through LDS.
//
// Times. T 8192, L 8, R 64, K 7168, N 4096 moves 263 MB: 50 us at the 5.25 TB/s of a
// large copy; shrink takes 27 us (37 where 124 or more tiles are in use: some compute
// units then hold three of its workgroups, and at about 25 bytes a clock their loads
// into LDS are the limit), expand 39-40. 64 tokens of 64 adapters, R 16: 15 MB and two
// launches, 6.2 and 6.0 us, mostly latency: plan, rows, operands one after another.
// 16- against 64-row tiles, both launches: R 16, L 8, T 128 / 256 / 1024: 9.7 / 11.0 /
// 17.1 against 10.6 / 10.7 / 14.4 us; L 64, T 1024 / 2048 19.5 / 25.8 against 21.3 / 21.6:
// 64 pays from about 32 tokens an adapter on.
//
// K order in a fragment: both operands of an MFMA may take their 32 k values in any
// common order. With 16-row tiles lane quarter q takes the 16 consecutive values at
// 16 q of a 64-wide step over two MFMAs, so a row's 64 values are one 128-byte line.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "fg.h"
#include "fg_device.hpp"
#include "fg_wave.hpp"

namespace {

using namespace fg;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kMaxRank = 128;
constexpr int kStepK = 64;
constexpr size_t kSpareBytes = 64 * 16;

struct AdapterArgs {
  const uint16_t *D, *x, *A, *B;
  const float* scales;
  const int32_t *rows, *slots, *m_indices;
  const int32_t* used;    // rows of the plan in use (its offsets[L])
  uint16_t* out;
  float* ws;              // [parts][cap][16 * TR]
  uint16_t* spare;        // 64 x 16 bytes that hold nothing
  int T, L, R, K, N, cap;
  int parts;              // parts of K
  int strip;              // columns of one expand workgroup
  bool stream;            // out is larger than the caches
  int tiles, tiles_up8;   // row tiles, and their number rounded up to 8
  int copies;             // workgroups of expand that pass tokens through (a multiple of 8)
};

// The row tile of position i of the tiles_up8 in a launch: workgroups go round-robin
// to the 8 XCDs, and each XCD gets a run of the tiles in use, so that an adapter's A
// and B pass through one or two of the L2s and not through all. -1: no tile.
__device__ __forceinline__ int tile_of(const AdapterArgs& p, int i, int rows) {
  const int in_use = *p.used / rows, U = in_use < p.tiles ? in_use : p.tiles;
  const int xcd = i & 7, lo = (int)((long)U * xcd >> 3), hi = (int)((long)U * (xcd + 1) >> 3);
  const int tile = lo + (i >> 3);
  return tile < hi ? tile : -1;
}

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

__device__ __forceinline__ f32x4v mfma(u32x4 a, u32x4 b, f32x4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

// TR: 16-column groups of the rank.
//
// 16-row tiles (decode: few tokens per adapter, so A is read once and nothing is
// shared): the four waves split the part's K, each lane's fragments come straight
// from global memory, two steps under way, and the waves' sums meet in LDS.
template <int TR>
__global__ __launch_bounds__(kThreads) void adapter_shrink16(AdapterArgs p) {
  constexpr int RT = 16, RC = 16 * TR, RP = RC + 4;
  __shared__ float red[kWaves][RT][RP];
  const int tile = tile_of(p, blockIdx.x, RT), r0 = tile * RT;
  if (tile < 0) return;
  const int a = p.m_indices[r0];
  if ((unsigned)a >= (unsigned)p.L) return;   // no token in this tile (uniform)
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lrow = lane & 15, q = lane >> 4;

  // rows without a token repeat the tile's first one; their sums are not stored
  const int first = p.slots[r0], mine = p.slots[r0 + lrow];
  const int tok = (unsigned)mine < (unsigned)p.T ? mine : (unsigned)first < (unsigned)p.T ? first : 0;
  const uint16_t* xp = p.x + (long)tok * p.K + 16 * q;
  const uint16_t* ap[TR];
#pragma unroll
  for (int c = 0; c < TR; ++c) {
    const int r = 16 * c + lrow < p.R ? 16 * c + lrow : p.R - 1;
    ap[c] = p.A + ((long)a * p.R + r) * p.K + 16 * q;
  }
  const int steps = p.K / kStepK;
  const int lanes = p.parts * kWaves, me = blockIdx.y * kWaves + wave;
  const int s0 = steps * me / lanes, s1 = steps * (me + 1) / lanes;

  f32x4v acc[TR];
#pragma unroll
  for (int c = 0; c < TR; ++c) acc[c] = f32x4v{0.f, 0.f, 0.f, 0.f};
  struct Step {
    u32x4 x[2], a[TR][2];
  };
  const auto load = [&](Step& f, int s) {
    const u32x4* v = (const u32x4*)(xp + (long)s * kStepK);
    f.x[0] = v[0];
    f.x[1] = v[1];
#pragma unroll
    for (int c = 0; c < TR; ++c) {
      const u32x4* u = (const u32x4*)(ap[c] + (long)s * kStepK);
      f.a[c][0] = u[0];
      f.a[c][1] = u[1];
    }
  };
  const auto multiply = [&](const Step& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < TR; ++c) acc[c] = mfma(f.a[c][h], f.x[h], acc[c]);
  };
  // Loads are issued unconditionally (past the end the last step again): behind a
  // branch the compiler could not count them and would wait for the step ahead too.
  Step f[2];
  if (s0 < s1) {
    const int last = s1 - 1;
    load(f[0], s0);
    for (int s = s0; s < s1; s += 2) {
      load(f[1], s + 1 < last ? s + 1 : last);
      multiply(f[0]);
      if (s + 1 < s1) {
        load(f[0], s + 2 < last ? s + 2 : last);
        multiply(f[1]);
      }
    }
  }
  // lane holds ranks 16 c + 4 q + v of row lrow
#pragma unroll
  for (int c = 0; c < TR; ++c) *(f32x4v*)&red[wave][lrow][16 * c + 4 * q] = acc[c];
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

// 16 bytes per lane from global memory straight into LDS at lds_at + 16 * lane
// (no register in between; counted by vmcnt like any load).
__device__ __forceinline__ void dma16(const void* src, uint32_t lds_at) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(src), "s"(lds_at) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// shrink for 64-row tiles: wave w owns rows 16 w .. 16 w + 15 over the whole part
// of K, so nothing is summed across waves and A, used by all four, is worth
// staging. A ring of kStages LDS stages of 64 k (x rows and A rows, one 128-byte
// line each) is filled by direct global-to-LDS loads kStages - 1 steps ahead. One
// barrier per step both publishes a stage and frees the one before it. A row's
// 16-byte chunk c sits at position c ^ (row & 7), which spreads the 16 rows that a
// quarter wave reads over the banks.
constexpr int kStages = 3;

template <int TR>
__global__ __launch_bounds__(kThreads) void adapter_shrink64(AdapterArgs p) {
  constexpr int RT = 64, RC = 16 * TR;
  constexpr int AI = TR > 2 ? TR / 2 : 1;           // A loads per wave and stage
  constexpr int kStageBytes = RT * 128 + RC * 128;
  __shared__ __attribute__((aligned(128))) uint8_t ring[kStages * kStageBytes];
  const int tile = tile_of(p, blockIdx.x, RT), r0 = tile * RT;
  if (tile < 0) return;
  const int a = p.m_indices[r0];
  if ((unsigned)a >= (unsigned)p.L) return;   // no token in this tile (uniform)
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lrow = lane & 15, q = lane >> 4;
  const int steps = p.K / kStepK;
  const int part = blockIdx.y, s0 = steps * part / p.parts, s1 = steps * (part + 1) / p.parts;

  // a load instruction covers eight rows; its lanes fetch their row's chunks in swizzled order
  const int first = p.slots[r0];
  const int chunk = 8 * ((lane & 7) ^ (lane >> 3));   // in elements
  const uint16_t *xp[2], *ap[AI];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = p.slots[r0 + 16 * wave + 8 * i + (lane >> 3)];
    // rows without a token repeat the tile's first one; their sums are not stored
    const int tok = (unsigned)s < (unsigned)p.T ? s : (unsigned)first < (unsigned)p.T ? first : 0;
    xp[i] = p.x + (long)tok * p.K + (long)s0 * kStepK + chunk;
  }
  int arow[AI];
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    arow[i] = 8 * ((wave * AI + i) % (2 * TR));       // waves without a share repeat another's load
    const int r = arow[i] + (lane >> 3) < p.R ? arow[i] + (lane >> 3) : p.R - 1;
    ap[i] = p.A + ((long)a * p.R + r) * p.K + (long)s0 * kStepK + chunk;
  }
  const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)ring;
  // Issues the loads of one step into a stage; past the end the last step again, so that every
  // wave always has the same number of loads under way.
  int to_go = s1 - s0 - 1;
  const auto issue = [&](int stage) {
    const uint32_t at = lds0 + stage * kStageBytes;
#pragma unroll
    for (int i = 0; i < 2; ++i) dma16(xp[i], at + (16 * wave + 8 * i) * 128);
#pragma unroll
    for (int i = 0; i < AI; ++i) dma16(ap[i], __builtin_amdgcn_readfirstlane(at + (RT + arow[i]) * 128));
    const int adv = to_go > 0 ? kStepK : 0;
    --to_go;
#pragma unroll
    for (int i = 0; i < 2; ++i) xp[i] += adv;
#pragma unroll
    for (int i = 0; i < AI; ++i) ap[i] += adv;
  };
  f32x4v acc[TR];
#pragma unroll
  for (int c = 0; c < TR; ++c) acc[c] = f32x4v{0.f, 0.f, 0.f, 0.f};
  if (s0 < s1) {   // uniform over the workgroup
    for (int i = 0; i < kStages - 1; ++i) issue(i);
    int stage = 0;
    for (int s = s0; s < s1; ++s) {
      // this stage's loads are the oldest; the later stages' stay under way
      wait_vm<(kStages - 2) * (2 + AI)>();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the last step's LDS reads are done
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      issue(stage == 0 ? kStages - 1 : stage - 1);
      const uint8_t* st = ring + stage * kStageBytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = ((4 * h + q) ^ (lrow & 7)) << 4;
        const u32x4 xf = *(const u32x4*)(st + (16 * wave + lrow) * 128 + at);
#pragma unroll
        for (int c = 0; c < TR; ++c)
          acc[c] = mfma(*(const u32x4*)(st + (RT + 16 * c + lrow) * 128 + at), xf, acc[c]);
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    wait_vm<0>();   // nothing may land in LDS after the workgroup has ended
  }
  const int row = r0 + 16 * wave + lrow;
  if ((unsigned)p.slots[row] >= (unsigned)p.T) return;
  float* out = p.ws + ((long)blockIdx.y * p.cap + row) * RC + 4 * q;
#pragma unroll
  for (int c = 0; c < TR; ++c) *(f32x4v*)(out + 16 * c) = acc[c];
}

// Two floats as a pair of bf16, their lower 16 bits dropped.
__device__ __forceinline__ uint32_t bf16_pair_cut(float a, float b) {
  return (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u);
}

// A lane's fragments of h: row `row` of the tile, its parts summed, scaled and cut
// into three pieces: the upper eight bits of the significand, the upper eight of what
// is left of it, and the rest, which has eight at most. Both differences are exact.
// (Bits of h below 2^-133, bf16's smallest, are lost.) TR == 1: half of the first piece
// in the lanes of k 0 .. 15 and in the others (not zeros: 0 times an infinite weight
// is NaN), then the second piece and the third.
template <int TR>
struct HFrags {
  static constexpr int KF = TR == 1 ? 1 : TR / 2;   // 32-deep fragments of the rank
  static constexpr int HL = TR == 1 ? 2 : 3;        // fragments of the pieces
  u32x4 f[HL][KF];
};
// `first`: the tile's first row, read in the place of rows without a token.
template <int TR>
__device__ __forceinline__ void load_h(const AdapterArgs& p, int row, int first, bool real, float scale, int q,
                                       HFrags<TR>& h) {
  constexpr int RC = 16 * TR, KF = HFrags<TR>::KF;
  constexpr int kTogether = KF > 2 ? 2 : 4;   // parts whose loads are under way together
  f32x4v v[KF][2];
#pragma unroll
  for (int k = 0; k < KF; ++k) v[k][0] = v[k][1] = f32x4v{0.f, 0.f, 0.f, 0.f};
  const float* src = p.ws + (long)(real ? row : first) * RC + (TR == 1 ? 8 * (q & 1) : 8 * q);
  const long stride = (long)p.cap * RC;
  for (int c = 0; c < p.parts; c += kTogether) {
    f32x4v u[kTogether][KF][2];
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const float* part = src + stride * (c + i < p.parts ? c + i : c);
#pragma unroll
      for (int k = 0; k < KF; ++k) {
        u[i][k][0] = *(const f32x4v*)(part + 32 * k);
        u[i][k][1] = *(const f32x4v*)(part + 32 * k + 4);
      }
    }
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      if (c + i < p.parts) {   // uniform
#pragma unroll
        for (int k = 0; k < KF; ++k) {
          v[k][0] += u[i][k][0];
          v[k][1] += u[i][k][1];
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < KF; ++k) {
    if (!real || (TR == 1 ? 8 * (q & 1) : 32 * k + 8 * q) >= p.R) v[k][0] = v[k][1] = f32x4v{0.f, 0.f, 0.f, 0.f};
    u32x4 piece[3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x = v[k][e >> 1][2 * (e & 1)] * scale, y = v[k][e >> 1][2 * (e & 1) + 1] * scale;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        piece[i][e] = bf16_pair_cut(x, y);
        x -= bf16_lo(piece[i][e]);
        y -= bf16_hi(piece[i][e]);
      }
    }
    if constexpr (TR == 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) h.f[0][0][e] = bf16_pair_cut(bf16_lo(piece[0][e]) * 0.5f, bf16_hi(piece[0][e]) * 0.5f);
      h.f[1][0] = q < 2 ? piece[1] : piece[2];
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i) h.f[i][k] = piece[i];
    }
  }
}

// Tokens without an adapter pass through: workgroup `block` of the launch's first
// p.copies takes 16 tokens, each wave four, all its loads under way before the
// first store.
template <bool STREAM>
__device__ __forceinline__ void copy_tokens(const AdapterArgs& p, int block) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long t0 = ((long)block * kWaves + wave) * 4;
  long tok[4];
  bool pass[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // past the last token: the last one, not stored
    tok[i] = t0 + i < p.T ? t0 + i : p.T - 1;
    pass[i] = (unsigned)p.rows[tok[i]] >= (unsigned)p.cap && t0 + i < p.T;
  }
  if (!(pass[0] || pass[1] || pass[2] || pass[3])) return;
  for (int n = 8 * lane; n < p.N; n += 8 * 64) {
    u32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *(const u32x4*)(p.D + tok[i] * p.N + n);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (pass[i]) store16<STREAM>((u32x4*)(p.out + tok[i] * p.N + n), v[i]);
  }
}

// Columns go in pairs of 16-wide sub-tiles: sub-tile e's operand row i is column
// 8 (i / 4) + 4 e + i % 4 of the pair's 32, so a lane's results of the pair are the
// eight consecutive columns 8 q .. 8 q + 7 and D moves in 16-byte pieces.
__device__ __forceinline__ int pair_row(int i, int e) { return 8 * (i >> 2) + 4 * e + (i & 3); }

// A lane's eight columns of D as the products' starting values, and back as bf16.
__device__ __forceinline__ void start_pair(u32x4 d, f32x4v* acc) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    acc[e >> 1][2 * (e & 1)] = bf16_lo(d[e]);
    acc[e >> 1][2 * (e & 1) + 1] = bf16_hi(d[e]);
  }
}
// The first pieces' products and the lower pieces' as one sum. Where the lower sum is
// no number, an h or a weight is infinite or NaN (inf - inf in a lower piece, 0 x inf in
// a product), and the first pieces alone give what whole values would: they have the
// signs of h and are zero only where it is.
__device__ __forceinline__ f32x4v join(f32x4v top, f32x4v rest) {
  f32x4v r;
#pragma unroll
  for (int v = 0; v < 4; ++v) r[v] = top[v] + (__builtin_isfinite(rest[v]) ? rest[v] : 0.0f);
  return r;
}
__device__ __forceinline__ u32x4 end_pair(const f32x4v* acc) {
  u32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = bf16_pair(acc[e >> 1][2 * (e & 1)], acc[e >> 1][2 * (e & 1) + 1]);
  return r;
}

// Expand for 16-row tiles: each wave has its own columns, 32 at a time, and B's
// fragments come straight from global memory (B is read once).
template <int TR>
__global__ __launch_bounds__(kThreads) void adapter_expand16(AdapterArgs p) {
  using H = HFrags<TR>;
  if ((int)blockIdx.x < p.copies) return copy_tokens<false>(p, blockIdx.x);
  const int job = blockIdx.x - p.copies, strip = job / p.tiles_up8;
  const int tile = tile_of(p, job - strip * p.tiles_up8, 16), r0 = tile * 16;
  if (tile < 0) return;
  const int a = p.m_indices[r0];
  if ((unsigned)a >= (unsigned)p.L) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lrow = lane & 15, q = lane >> 4;
  const int n_lo = strip * p.strip, n_hi = n_lo + p.strip < p.N ? n_lo + p.strip : p.N;
  const int tok = p.slots[r0 + lrow];
  const bool real = (unsigned)tok < (unsigned)p.T;
  const int first = p.slots[r0];
  const uint16_t* drow = p.D + (long)(real ? tok : (unsigned)first < (unsigned)p.T ? first : 0) * p.N;
  H h;
  load_h<TR>(p, r0 + lrow, r0, real, p.scales[a], q, h);
  const uint16_t* Ba = p.B + (long)a * p.N * p.R;
  for (int n0 = n_lo + 32 * wave; n0 < n_hi; n0 += 32 * kWaves) {
    u32x4 bf[2][H::KF];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int f = 0; f < H::KF; ++f) {
        const int n = n0 + pair_row(lrow, e);
        const int r = TR == 1 ? 8 * (q & 1) : 32 * f + 8 * q;
        // loads are not predicated: outside B and D any valid piece is read and dropped
        bf[e][f] = *(const u32x4*)(Ba + (long)(n < n_hi ? n : n_hi - 1) * p.R + (r < p.R ? r : 0));
        if (r >= p.R) bf[e][f] = u32x4{0u, 0u, 0u, 0u};
      }
    const int col = n0 + 8 * q;
    const bool ok = real && col < n_hi;
    const u32x4 d = *(const u32x4*)(drow + (col < n_hi ? col : n_lo));
    f32x4v acc[2], rest[2];
    start_pair(d, acc);
    rest[0] = rest[1] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int l = H::HL - 1; l >= 0; --l)   // the small pieces first
#pragma unroll
      for (int f = 0; f < H::KF; ++f)
#pragma unroll
        for (int e = 0; e < 2; ++e) (l ? rest : acc)[e] = mfma(bf[e][f], h.f[l][f], (l ? rest : acc)[e]);
#pragma unroll
    for (int e = 0; e < 2; ++e) acc[e] = join(acc[e], rest[e]);
    if (ok) *(u32x4*)(p.out + (long)tok * p.N + col) = end_pair(acc);
  }
}

// Expand for 64-row tiles: wave w owns rows 16 w .. 16 w + 15, and B, used by all
// four waves, goes through LDS: 128 columns at a time, which are one contiguous
// piece of global memory, loaded straight into one of two LDS buffers while the
// other is in use. With B fetched by each wave on its own (half-line pieces of 16
// rows per instruction) its loads took 22 us of 55 at T = 8192, N = 4096, R = 64.
// A row's 16-byte chunk c sits at c ^ key(n) where the chunks per row are a power of
// two, key(n) spreading the rows that eight neighbouring lanes read over the banks.
//
// The products leave the matrix cores with 16 rows to an instruction; they turn round
// in LDS, 64 columns at a time, so that each load of D and store of out covers whole
// 128-byte lines of eight rows. Straight from the registers, 64-byte halves of 16 rows,
// the kernel took 38 or 46 us by the relative placing of D and out; so 37-39 us for either.
constexpr int kCols = 128, kHalf = 64;

__device__ __forceinline__ int swizzle_key(int n, int chunks) {
  return (chunks & (chunks - 1)) ? 0 : ((n & 3) | ((n >> 1) & 4)) & (chunks - 1);
}

// FULL: R is 16 TR, every fragment is of ranks below R. STREAM: out is larger than
// the caches.
template <int TR, bool FULL, bool STREAM>
__global__ __launch_bounds__(kThreads) void adapter_expand64(AdapterArgs p) {
  using H = HFrags<TR>;
  constexpr int NI = TR;                       // loads per wave and buffer: 128 columns x 2 TR chunks / 256
  __shared__ __attribute__((aligned(128))) uint8_t ring[2][NI * kThreads * 16];
  __shared__ float turn[kWaves][16][kHalf + 4];
  if ((int)blockIdx.x < p.copies) return copy_tokens<STREAM>(p, blockIdx.x);
  const int job = blockIdx.x - p.copies, strip = job / p.tiles_up8;
  const int tile = tile_of(p, job - strip * p.tiles_up8, 64), r0 = tile * 64;
  if (tile < 0) return;
  const int a = p.m_indices[r0];
  if ((unsigned)a >= (unsigned)p.L) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lrow = lane & 15, q = lane >> 4;
  const int n_lo = strip * p.strip, n_hi = n_lo + p.strip < p.N ? n_lo + p.strip : p.N;
  const int chunks = FULL ? 2 * TR : p.R >> 3;   // 16-byte chunks of a row of B
  const uint16_t* Ba = p.B + (long)a * p.N * p.R;
  const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)&ring[0][0];
  // This lane's LDS chunks hold row bn of the buffer's 128, chunk bc of it: at byte boff from the
  // buffer's first row in B. Rows past the buffer's 128 (R below 16 TR) or past N repeat a
  // valid one; nothing reads them.
  const int row_bytes = 16 * chunks;
  int boff[NI], bmax[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int g = (i * kWaves + wave) * 64 + lane, bn = g / chunks;
    const int bc = (g - bn * chunks) ^ swizzle_key(bn, chunks);
    boff[i] = (bn < kCols ? bn : kCols - 1) * row_bytes + 16 * bc;
    bmax[i] = 16 * bc;
  }
  const auto issue = [&](int buffer, int n0) {
    const char* base = (const char*)Ba + (long)n0 * row_bytes;
    const int left = (p.N - 1 - n0) < kCols ? (p.N - 1 - n0) * row_bytes : kCols * row_bytes;   // last row of B from here
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int most = left + bmax[i];
      dma16(base + (boff[i] < most ? boff[i] : most),
            lds0 + buffer * (NI * kThreads * 16) + (i * kWaves + wave) * 1024);
    }
  };
  issue(0, n_lo);
  const bool real = (unsigned)p.slots[r0 + 16 * wave + lrow] < (unsigned)p.T;
  // the two rows of D and out that this lane moves (8 i + lane / 8 of the wave's 16), at its
  // eight columns of a half round
  const uint16_t* drow[2];
  uint16_t* orow[2];
  bool has[2];
  const int dcol = 8 * (lane & 7);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int tok = p.slots[r0 + 16 * wave + 8 * i + (lane >> 3)];
    has[i] = (unsigned)tok < (unsigned)p.T;
    drow[i] = p.D + (long)(has[i] ? tok : 0) * p.N + dcol;
    orow[i] = p.out + (long)(has[i] ? tok : 0) * p.N + dcol;
  }
  uint16_t* spare = p.spare + 8 * lane;
  H h;
  load_h<TR>(p, r0 + 16 * wave + lrow, r0, real, p.scales[a], q, h);
  constexpr int NG = kCols / 32;
  int cc[H::KF];   // this lane's chunk of a row of B in each fragment
#pragma unroll
  for (int f = 0; f < H::KF; ++f) {
    const int c = TR == 1 ? q & 1 : 4 * f + q;
    cc[f] = FULL || c < chunks ? c : 0;
  }
  u32x4 d[2][NG];
  const auto load_d = [&](u32x4* v, int n0) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int at = n0 + kHalf * (g >> 1);
      v[g] = *(const u32x4*)(drow[g & 1] + (at + dcol < n_hi ? at : n_lo - dcol));   // outside: the strip's first
    }
  };
  load_d(d[0], n_lo);
  // Each round issues the next one's loads, then its own NG stores. Loads and stores
  // count down in order, so a wait for a load also waits for every store before it; at
  // a round's end only its own stores stay under way. For the count to be exact no
  // store is skipped: lanes without an output write to spare memory. (Loads two rounds
  // ahead, with a third buffer, were slower: 47 against 42 us.)
  wait_vm<0>();
  __builtin_amdgcn_s_waitcnt(0x0f70);
  const auto round = [&](auto which, int r) {
    constexpr int B = decltype(which)::value;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the other buffer's reads are done
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const int n0 = n_lo + kCols * r, next = n0 + kCols < n_hi ? n0 + kCols : n_lo;   // after the last, the first again
    issue(B ^ 1, next);
    load_d(d[B ^ 1], next);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x4v acc[2], rest[2];
      acc[0] = acc[1] = rest[0] = rest[1] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int f = 0; f < H::KF; ++f) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int n = 32 * g + pair_row(lrow, e);
          // ranks past R: any chunk, dropped (a predicated read would be a branch and a wait of its own)
          u32x4 b = *(const u32x4*)(ring[B] + ((n * chunks + (cc[f] ^ swizzle_key(n, chunks))) << 4));
          if (!FULL && cc[f] != (TR == 1 ? q & 1 : 4 * f + q)) b = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
          for (int l = H::HL - 1; l > 0; --l) rest[e] = mfma(b, h.f[l][f], rest[e]);
          acc[e] = mfma(b, h.f[0][f], acc[e]);
        }
      }
      float* to = &turn[wave][lrow][32 * (g & 1) + 8 * q];
      *(f32x4v*)to = join(acc[0], rest[0]);
      *(f32x4v*)(to + 4) = join(acc[1], rest[1]);
      if (g & 1) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the wave's own LDS accesses, in order
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float* from = &turn[wave][8 * i + (lane >> 3)][dcol];
          f32x4v sum[2];
          start_pair(d[B][g - 1 + i], sum);
          sum[0] += *(const f32x4v*)from;
          sum[1] += *(const f32x4v*)(from + 4);
          const int at = n0 + kHalf * (g >> 1);
          store16<STREAM>((u32x4*)(has[i] && at + dcol < n_hi ? orow[i] + at : spare), end_pair(sum));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<NG>();
    // The same wait in the compiler's own terms. It does not see the loads into LDS, so
    // its waits for d would take them for older operations and wait for the next round's.
    __builtin_amdgcn_s_waitcnt(0x0f70 | NG);
  };
  const int rounds = (n_hi - n_lo + kCols - 1) / kCols;
  for (int r = 0; r < rounds; r += 2) {
    round(std::integral_constant<int, 0>{}, r);
    if (r + 1 < rounds) round(std::integral_constant<int, 1>{}, r + 1);
  }
  wait_vm<0>();   // nothing may land in LDS after the workgroup has ended
}

// 16-column groups of the rank as compiled: 1, 2, 4 or 8.
int rank_groups(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

// Rows of one tile: 64 where the plan's segments allow it, else 16.
int tile_rows(int align) { return align % 64 == 0 ? 64 : 16; }

// Parts of K: enough workgroups to fill the chip, at least one step of K a wave.
// Every part is one more partial h, rows x rank, for each expand workgroup to read.
// 16-row tiles, 64 tokens of 64 adapters (K 7168, N 4096, R 16): 2 / 4 / 8 parts take
// 8.6 / 5.8 / 5.6 us in shrink and 5.6 / 6.2 / 8.3 us in expand, so those stop at 256
// workgroups. Both launches in a graph, at most 4 / 8 / 16 parts: one token, R 16, 7.3 /
// 6.9 / 7.5 us; one token, R 64, 12.4 / 10.0 / 9.9; 64-row tiles, T 1024 of 8 adapters, R
// 16, 15.1 / 13.5 / 15.0; R 64, 21.8 / 24.2 / 35.3 us.
int k_parts(int tiles, int rt, int K, int R) {
  const int most = K / (kStepK * kWaves) > 1 ? K / (kStepK * kWaves) : 1;
  const int limit = rt == 64 && R > 32 ? 4 : 8;
  const long fill = rt == 64 ? 512 : 256;
  int parts = 1;
  while (parts < limit && 2 * parts <= most && (long)tiles * parts < fill) parts *= 2;
  return parts;
}

int sizes(int R, int K, int cap, int align) {
  if (R < 8 || R % 8 || R > kMaxRank || K < 128 || K % 128 || K > (1 << 24) || align < 16 || align % 16 || cap < 0 ||
      cap % align)
    return FG_EINVAL;
  return FG_OK;
}

template <int TR>
void launch(const AdapterArgs& p, bool wide, hipStream_t s) {
  const dim3 g1(p.tiles_up8, p.parts), g2(p.copies + p.tiles_up8 * ((p.N + p.strip - 1) / p.strip)), b(kThreads);
  if (wide) {
    hipLaunchKernelGGL(adapter_shrink64<TR>, g1, b, 0, s, p);
    const bool full = p.R == 16 * TR;
    if (full && p.stream) hipLaunchKernelGGL((adapter_expand64<TR, true, true>), g2, b, 0, s, p);
    else if (full) hipLaunchKernelGGL((adapter_expand64<TR, true, false>), g2, b, 0, s, p);
    else if (p.stream) hipLaunchKernelGGL((adapter_expand64<TR, false, true>), g2, b, 0, s, p);
    else hipLaunchKernelGGL((adapter_expand64<TR, false, false>), g2, b, 0, s, p);
  } else {
    hipLaunchKernelGGL(adapter_shrink16<TR>, g1, b, 0, s, p);
    hipLaunchKernelGGL(adapter_expand16<TR>, g2, b, 0, s, p);
  }
}

}  // namespace

extern "C" {

int fg_adapters_workspace(int R, int K, int cap, int align, size_t* bytes) {
  if (!bytes || sizes(R, K, cap, align) != FG_OK) return FG_EINVAL;
  *bytes = kSpareBytes + (size_t)k_parts(cap / tile_rows(align), tile_rows(align), K, R) * cap * (16 * rank_groups(R)) * sizeof(float);
  return FG_OK;
}

int fg_adapters(const void* D, const void* x, const void* A, const void* B, const float* scales, const int32_t* rows,
                const int32_t* slots, const int32_t* m_indices, const int32_t* offsets, void* out, void* ws, int T, int L, int R, int K, int N,
                int cap, int align, hipStream_t stream) {
  if (T < 0 || L < 1 || N < 8 || N % 8 || N > (1 << 24) || sizes(R, K, cap, align) != FG_OK) return FG_EINVAL;
  if (T == 0) return FG_OK;
  if (cap < 1) return FG_EINVAL;   // a plan of T > 0 tokens has rows
  if (!D || !x || !A || !B || !scales || !rows || !slots || !m_indices || !offsets || !out || !ws) return FG_EINVAL;
  if (!aligned(D, 16) || !aligned(x, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(out, 16) ||
      !aligned(ws, 16) || !aligned(scales, 4) || !aligned(rows, 4) || !aligned(slots, 4) || !aligned(m_indices, 4) ||
      !aligned(offsets, 4))
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
  p.used = offsets + L;
  p.out = static_cast<uint16_t*>(out);
  p.spare = static_cast<uint16_t*>(ws);
  p.ws = static_cast<float*>(ws) + kSpareBytes / sizeof(float);
  p.T = T;
  p.L = L;
  p.R = R;
  p.K = K;
  p.N = N;
  p.cap = cap;
  const int rt = tile_rows(align);
  p.tiles = cap / rt;
  p.tiles_up8 = (p.tiles + 7) / 8 * 8;
  p.parts = k_parts(p.tiles, rt, K, R);
  p.stream = (long long)T * N * 2 > kStreamBytes;
  p.copies = out != D ? (int)((T + 127L) / 128 * 8) : 0;
  // Columns of an expand workgroup: long strips load h less often, short ones fill the
  // chip. 64-row tiles, T 8192, N 4096, R 64: 512 / 1024 / 2048 columns take 40 / 37 / 37
  // us; both launches of 512 / 4096 tokens of 8 adapters, R 128, with strips for 256 or
  // for 512 workgroups: 25.5 / 55 against 31 / 62 us. 16-row tiles, 1024 tokens of 64
  // adapters, R 16 / 64: 18.5 / 38.4 us for 512 workgroups, 19.8 / 39.6 for 1024.
  p.strip = 1024;
  while (p.strip > 128 && (long)p.tiles * ((N + p.strip - 1) / p.strip) < (rt == 64 ? 256 : 512)) p.strip /= 2;
  if ((long)p.copies + (long)p.tiles_up8 * ((N + p.strip - 1) / p.strip) > 0x7fffffffL) return FG_EINVAL;
  switch (rank_groups(R)) {
    case 1: launch<1>(p, rt == 64, stream); break;
    case 2: launch<2>(p, rt == 64, stream); break;
    case 4: launch<4>(p, rt == 64, stream); break;
    default: launch<8>(p, rt == 64, stream); break;
  }
  if (hipGetLastError() != hipSuccess) return FG_ELAUNCH;
  return FG_OK;
}

}  // extern "C"
