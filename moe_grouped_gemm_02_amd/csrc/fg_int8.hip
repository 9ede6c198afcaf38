// fg_int8.hip -- host side of the 8-bit integer product: argument validation, tile
// choice and launch behind the C ABI declared in include/fg.h.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fg.h"
#include "fg_device.hpp"
#include "fg_int8_tiles.hpp"

namespace {

using namespace fg;
using namespace fg::int8_cfg;

// A round of a tile over the compute units takes fixed + kblocks * kblock us, fitted to the times of
// 200 dense problems of 200 to 8192 rows.
struct Tile {
  int bm, bn;
  double fixed, kblock;
};
constexpr Tile kTiles[] = {{256, 256, 5.0, 1.25}, {256, 128, 3.5, 0.80}, {128, 256, 3.5, 0.78},
                           {128, 128, 2.6, 0.52}, {64, 128, 1.2, 0.345}, {128, 160, 2.7, 0.60}};
constexpr int kNumTiles = sizeof(kTiles) / sizeof(kTiles[0]);
constexpr int kWide = 0, kNarrow = 1, kHalf = 2;
constexpr int kMaxK = 131056;     // 128^2 K < 2^31: the 32-bit sum is exact
constexpr int kMaxN = 4194296;    // 256 rows of N bf16 stay below 2^31 bytes

// A grid has fewer than 2^32 threads (past that the runtime drops workgroups without a word),
// a tile at most 512.
constexpr long kMaxTiles = (1L << 23) - 1;

long ceil_div(long a, long b) { return (a + b - 1) / b; }

constexpr double kLaunch = 2.0;

// Estimated us of `tiles` tiles of one shape after the launch; a partial round is faster a K-block.
double tiles_us(const Tile& t, long tiles, long cus, double kblocks) {
  const double fill = tiles < cus ? (double)tiles / (double)cus : 1.0;
  return (double)ceil_div(tiles, cus) * (t.fixed + kblocks * t.kblock * (0.85 + 0.15 * fill));
}

// Estimated us of weights that come from memory, as `bytes` that no cache keeps do: each of the
// columns' workgroups fetches at most `rate` GB/s, all 5200 (128 tiles of 64 x 128 28 GB/s each, 256 20).
double stream_us(long groups, int columns, int K, long cus, double bytes, double rate) {
  if (bytes < 64.0e6) return 0.0;
  const double rounds = 0.5 * ((double)ceil_div(groups, cus) + (groups > cus ? (double)groups / (double)cus : 1.0));
  const double share = 5200.0 / (double)(groups < cus ? groups : cus);
  return rounds * columns * (double)K * 1e-3 / (rate < share ? rate : share);
}

#ifdef FG_TESTING
// Test build only (libfg_testing.so): this thread's later calls run on one of the compiled
// choices, with at most so many workgroups where these walk their tiles.
thread_local int t_tile = -1, t_grid = 0;
#endif

struct Choice {
  int tile = -1;
  long grid = 0, tiles_a = 0;
  int n_split = 0;
};

// The kernel that streams the weights (int8_skinny), by row blocks of 16 tm rows and 16, 32 or 64
// columns. A workgroup loads its rows and columns once, at some 90 GB/s a CU from the L2s, so a
// round takes what its rows + columns ask for, and small blocks on all CUs are faster than
// large ones on a few. Measured, us, K 7168, blocks (rows x columns) and the best tile:
//   M 16   N 2048  16x16 5.3  16x32 6.4  16x64 8.6  tile 17.9    N 7168  16x16 11.0  16x32 9.9  16x64 10.2  tile 18.6
//   M 128  N 256  16x16 4.1  32x16 4.9  128x16 10.3  tile 17.5    N 1024  32x16 6.6  32x32 7.5  64x16 8.6  128x16 11.5  tile 18.5
//          N 4096  64x32 10.6  32x64 11.0  128x16 14.2  tile 18.6    N 7168  128x32 16.7  64x64 17.6  32x64 17.9  tile 19.2
//   M 1024 N 256  16x64 9.3  32x64 10.8  128x16 18.3  tile 18.4    N 1024  128x32 16.7  64x64 17.9  tile 18.8
//          N 2048  64x64 23.2  128x32 31.1  tile 20.4
// and K 1024: M 16, N 4096  16x64 3.2  16x32 3.7  tile 4.9    M 256, N 2048  32x64 4.2  64x32 4.4  tile 5.2
struct SkinnyTime {
  int tm;
  double least[3];   // us at K to 0, for 16, 32 and 64 columns; 0: no such kernel
};
constexpr SkinnyTime kSkinnyTimes[] = {{1, {3.5, 3.5, 3.1}}, {2, {3.6, 3.6, 4.0}}, {3, {3.6, 4.0, 5.1}},
                                       {4, {4.0, 4.2, 5.0}}, {6, {3.8, 4.6, 6.0}}, {8, {4.2, 5.2, 0.0}}};

Choice skinny_choice(int M, int N, int G, int tm, int i) {
  Choice c;
  c.tile = kSkinny + 3 * (tm - 1) + i;
  c.grid = ceil_div(M, 16 * tm) * ceil_div(N, 16 << i) * G;
  return c;
}

// The fastest of them and its estimated time in us (1e30: none). Of 220 random dense and masked
// problems the choice among these and the tiles is 1.4% from the fastest measured on average and 24%
// at most, of 90 contiguous ones, whose padding the host does not know, 6% and 47% (12% faster than
// the best tile on average, 24% slower at most).
Choice skinny(int layout, int M, int N, int K, int G, int cus, double bytes, double& us) {
  Choice best;
  const int experts = layout == FG_LAYOUT_MASKED ? G : 1;   // whose rows are apart
  us = 1e30;
  // rows that start within a 128-byte line take more loads, few waves feel it most
  const double k = (double)K / 7168.0 * (K % 128 ? 1.25 : 1.0), k64 = (double)K / 7168.0 * (K % 64 ? 1.5 : K % 128 ? 1.25 : 1.0);
  for (const SkinnyTime& s : kSkinnyTimes) {
    if (s.tm > 1 && 8 * s.tm >= M) break;   // half of the rows and more past M
    if (layout == FG_LAYOUT_CONTIGUOUS && 8 % s.tm) continue;   // within a block of 128 rows
    for (int i = 0; i < 3; ++i) {
      if (s.least[i] == 0.0) continue;
      const Choice c = skinny_choice(M, N, experts, s.tm, i);
      if (c.grid > kMaxTiles) continue;
      // with two waves (64 columns, 48 rows and more) the loads' latency counts
      const bool two = s.tm >= 3 && i == 2, wide = s.tm == 8 && i == 1;
      const double base = two ? 4.7 : wide ? 4.8 : 2.4, sum = (two ? 1.5 : wide ? 1.15 : 1.3) * (s.tm + (1 << i)) * (i < 2 ? k : k64);
      double at = base + sum > s.least[i] ? base + sum : s.least[i];
      if (c.grid > cus) {   // a further round; workgroups of 64 columns are resident in twos
        const long rounds = ceil_div(c.grid, cus);
        at += (double)(rounds - 1) * (i < 2        ? sum + 1.5
                                      : s.tm == 1  ? 0.9 * sum + 0.3
                                      : s.tm == 2  ? 0.9 * sum + 1.0
                                      : s.tm == 6  ? 0.5 * sum + 5.0
                                      : rounds > 2 ? sum + 1.8
                                                   : 0.35 * sum + 0.7);
      }
      if (layout == FG_LAYOUT_CONTIGUOUS) at = 1.1 * at + 0.4;   // the look-up, experts that share less of the caches
      const double stream = stream_us((long)experts * ceil_div(N, 16 << i), 16 << i, K, cus, bytes, 60.0);
      if (stream > 0.85 * at) at = stream + 0.15 * at;
      if (at < us) {
        us = at;
        best = c;
      }
    }
  }
  return best;
}

// The shape whose tiles, in rounds over the compute units, take the least estimated
// time; dense problems also try whole rounds of 256x256 tiles with the remaining
// columns on 256x128, contiguous ones the run-following kernel.
Choice choose(int layout, int M, int N, int K, int G, int cus) {
  Choice best;
  double cost = 0.0;
  const double kb = (double)ceil_div(K, 128), bytes = (double)(layout == FG_LAYOUT_DENSE ? 1 : G) * N * K;
  // contiguous: the experts' look-up in each round; blocks of one expert that are apart in time fetch
  // its weights again where no cache keeps them
  const bool contiguous = layout == FG_LAYOUT_CONTIGUOUS;
  const long blocks = ceil_div(M, 128);
  const double lookup = contiguous ? 1.2 : 0.0;
  const double again = contiguous && blocks > G && bytes >= 64.0e6 ? bytes / 5.2e6 * (1.0 - (double)G / (double)blocks) : 0.0;
  for (int i = 0; i < kNumTiles; ++i) {
    const Tile& t = kTiles[i];
    if (contiguous && t.bm > 128) continue;   // a tile's rows are one expert's
    const long tiles = ceil_div(M, t.bm) * ceil_div(N, t.bn) * (layout == FG_LAYOUT_MASKED ? G : 1);
    if (tiles > kMaxTiles) continue;
    double c = tiles_us(t, tiles, cus, kb) + (double)ceil_div(tiles, cus) * lookup + again;
    if (!contiguous) {
      const double stream = stream_us(tiles / ceil_div(M, t.bm), t.bn, K, cus, bytes, t.bn == 256 ? 22.0 : 28.0) * (K % 128 ? 1.15 : 1.0);
      if (stream > c) c = stream;
    }
    if (best.tile < 0 || c < cost) {
      best.tile = i;
      best.grid = tiles;
      cost = c;
    }
  }
  if (contiguous && blocks <= kRunMaxBlocks && G <= kRunMaxExperts) {
    // G runs, half of them odd (as many as leave whole pairs): full two-block tiles and single blocks per column
    const long runs = G < blocks ? G : blocks, S = runs / 2 + ((blocks - runs / 2) & 1), F = (blocks - S) / 2;
    const long tn = ceil_div(N, 256), items = blocks * tn, grid = items < cus ? items : cus;
    const double tf = tiles_us(kTiles[kWide], cus, cus, kb), th = tiles_us(kTiles[kHalf], cus, cus, kb);
    const long full = F * tn, rest = full % grid;
    // a last partial round of full tiles leaves CUs for single blocks
    const long left = S * tn - (rest ? grid - rest : 0);
    const double c = (double)(full / grid) * tf + (rest && 2 * rest + S * tn <= grid ? th : rest ? tf : 0.0) +
                     (left > 0 ? (double)ceil_div(left, grid) * th : 0.0) - (left > 0 && left % grid && 4 * (left % grid) <= grid ? 0.5 * th : 0.0) +
                     lookup + 0.45 * again;   // a last round in quarters
    if (c < cost) {
      best.tile = kRuns;
      best.grid = grid;
      cost = c;
    }
  }
  if (layout == FG_LAYOUT_DENSE) {
    const long tm = ceil_div(M, 256);
    for (long nc = N / 256 * 256; nc >= 256; nc -= 256) {
      const long a = tm * (nc / 256);
      if (a % cus) continue;
      if (nc == N) break;   // whole rounds on the wide tile alone
      const long b = tm * ceil_div(N - nc, 128);
      const double c = tiles_us(kTiles[kWide], a, cus, kb) + tiles_us(kTiles[kNarrow], b, cus, kb);
      if (c < cost) {
        best.tile = kSplit;
        best.n_split = (int)nc;
        best.tiles_a = a;
        best.grid = (a > b ? a : b) < cus ? (a > b ? a : b) : cus;
        cost = c;
      }
      break;
    }
  }
  const long experts = layout == FG_LAYOUT_MASKED ? G : 1, w = ceil_div(M, kSkinnyRows) * ceil_div(N, 64) * experts;
  if (w <= 4 * cus || M <= 16) {
    double us;
    const Choice c = skinny(layout, M, N, K, G, cus, contiguous ? 0.0 : bytes, us);
    if (us < (contiguous ? 0.93 : 0.97) * (kLaunch + cost)) return c;
  }
  return best;
}

#ifdef FG_TESTING
bool forced(int layout, int M, int N, int G, int cus, Choice& c) {
  c = Choice();
  c.tile = t_tile;
  if (t_tile < kNumTiles) {
    const Tile& t = kTiles[t_tile];
    c.grid = ceil_div(M, t.bm) * ceil_div(N, t.bn) * (layout == FG_LAYOUT_MASKED ? G : 1);
    return layout != FG_LAYOUT_CONTIGUOUS || t.bm <= 128;
  }
  if (t_tile >= kSkinny) {
    // 16 t_grid rows a workgroup, or all up to 128
    int tm = t_grid ? t_grid : (int)ceil_div(M < kSkinnyRows ? M : kSkinnyRows, 16);
    if (!t_grid && tm > 4) tm = tm <= 6 ? 6 : 8;
    c = skinny_choice(M, N, layout == FG_LAYOUT_MASKED ? G : 1, tm, t_tile - kSkinny);
    bool there = false;
    for (const SkinnyTime& s : kSkinnyTimes) there |= s.tm == tm && s.least[t_tile - kSkinny] > 0.0;
    return there && (layout != FG_LAYOUT_CONTIGUOUS || 8 % tm == 0);
  }
  c.grid = t_grid > 0 ? t_grid : cus;
  if (t_tile == kRuns) return layout == FG_LAYOUT_CONTIGUOUS;
  c.n_split = N / 512 * 256;
  c.tiles_a = ceil_div(M, 256) * (c.n_split / 256);
  return t_tile == kSplit && layout == FG_LAYOUT_DENSE && c.n_split > 0;
}
#endif

int run(int layout, const void* A, const float* sa, const void* B, const float* sb, void* D, const int32_t* index,
        int M, int N, int K, int G, hipStream_t stream) {
  if (M < 0 || N < 0 || N % 8 || N > kMaxN || K < 16 || K % 16 || K > kMaxK || G < 1) return FG_EINVAL;
  if (M == 0 || N == 0) return FG_OK;
  if (!A || !sa || !B || !sb || !D || (layout != FG_LAYOUT_DENSE && !index)) return FG_EINVAL;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(D, 16) || !aligned(sa, 4) || !aligned(sb, 4) || !aligned(index, 4))
    return FG_EINVAL;
  // the largest tiles, of which choose() always has one
  const Tile& top = kTiles[layout == FG_LAYOUT_CONTIGUOUS ? kHalf : kWide];
  if ((layout == FG_LAYOUT_MASKED ? (double)G : 1.0) * ceil_div(M, top.bm) * ceil_div(N, top.bn) > kMaxTiles) return FG_EINVAL;
  int cus = 0;
  const int st = current_device(&cus);
  if (st != FG_OK) return st;
  Choice c = choose(layout, M, N, K, G, cus);
#ifdef FG_TESTING
  if (t_tile >= 0 && (!forced(layout, M, N, G, cus, c) || c.grid > kMaxTiles)) return FG_EINVAL;
#endif
  const Tile& t = kTiles[c.tile < kNumTiles ? c.tile : kWide];
  Params p = {};
  p.A = static_cast<const uint8_t*>(A);
  p.sa = sa;
  p.B = static_cast<const uint8_t*>(B);
  p.sb = sb;
  p.D = static_cast<uint16_t*>(D);
  p.m_indices = p.masked_m = index;
  p.M = M;
  p.N = N;
  p.K = K;
  p.G = G;
  p.KB = (int)ceil_div(K, 128);
  p.tiles_m = (int)ceil_div(M, c.tile >= kSkinny ? 16 * ((c.tile - kSkinny) / 3 + 1) : t.bm);
  p.tiles_n = (int)ceil_div(N, c.tile >= kSkinny ? 16 << (c.tile - kSkinny) % 3 : t.bn);
  p.n_split = c.n_split;
  p.tiles_a = (int)c.tiles_a;
  hipError_t e;
  switch (layout) {
    case FG_LAYOUT_DENSE: e = launch_int8<kDense>(c.tile, p, (int)c.grid, stream); break;
    case FG_LAYOUT_CONTIGUOUS: e = launch_int8<kContiguous>(c.tile, p, (int)c.grid, stream); break;
    default: e = launch_int8<kMasked>(c.tile, p, (int)c.grid, stream);
  }
  return e == hipSuccess ? FG_OK : FG_ELAUNCH;
}

}  // namespace

extern "C" {

int fg_gemm_int8_nt(const void* A, const float* sa, const void* B, const float* sb, void* D, int M, int N, int K,
                    hipStream_t stream) {
  return run(FG_LAYOUT_DENSE, A, sa, B, sb, D, nullptr, M, N, K, 1, stream);
}

int fg_grouped_contiguous_int8(const void* A, const float* sa, const void* B, const float* sb, void* D,
                               const int32_t* m_indices, int M, int N, int K, int G, hipStream_t stream) {
  return run(FG_LAYOUT_CONTIGUOUS, A, sa, B, sb, D, m_indices, M, N, K, G, stream);
}

int fg_grouped_masked_int8(const void* A, const float* sa, const void* B, const float* sb, void* D,
                           const int32_t* masked_m, int G, int M_max, int N, int K, hipStream_t stream) {
  return run(FG_LAYOUT_MASKED, A, sa, B, sb, D, masked_m, M_max, N, K, G, stream);
}

#ifdef FG_TESTING
int fgt_force_int8(int tile, int grid) {
  if (tile < -1 || tile > kSkinny + 2 || grid < 0) return FG_EINVAL;
  t_tile = tile;
  t_grid = grid;
  return FG_OK;
}
#endif

}  // extern "C"
