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

struct Tile {
  int bm, bn, waves;
  double eff;   // fraction of the matrix-core rate the tile's K loop sustains
};
constexpr Tile kTiles[] = {{256, 256, Cfg0::W, 0.80}, {256, 128, Cfg1::W, 0.75}, {128, 256, Cfg2::W, 0.75},
                           {128, 128, Cfg3::W, 0.70}, {64, 128, Cfg4::W, 0.60}, {128, 160, Cfg5::W, 0.70}};
constexpr int kNumTiles = sizeof(kTiles) / sizeof(kTiles[0]);
constexpr int kWide = 0, kNarrow = 1, kHalf = 2;
constexpr int kMaxK = 131056;     // 128^2 K < 2^31: the 32-bit sum is exact
constexpr int kMaxN = 4194296;    // 256 rows of N bf16 stay below 2^31 bytes

// A grid has fewer than 2^32 threads (past that the runtime drops workgroups without a word),
// a tile at most 512.
constexpr long kMaxTiles = (1L << 23) - 1;

long ceil_div(long a, long b) { return (a + b - 1) / b; }

// Estimated cycles of one tile over kblocks K-blocks: its matrix-core time at 8192
// operations per clock, or its loads into LDS at what the path sustains, and a start and end.
double tile_cycles(const Tile& t, double kblocks) {
  const double mfma = t.bm * t.bn * 256.0 / (8192.0 * t.eff), mem = (t.bm + t.bn) * 128.0 / (t.waves >= 8 ? 30.0 : 24.0);
  return kblocks * (mfma > mem ? mfma : mem) + 4000.0;
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

// The kernel that streams the weights (int8_skinny), or none where tiles are faster. By the
// workgroups w of 128 rows and 64 columns: enough of them share a CU's time, few need narrower
// columns to reach all CUs. Measured, us, K 7168, 16 / 32 / 64 columns and the best tile:
//   M 16   N 2048 (w 32) 5.3 / 6.4 / 8.5 / 17.9    N 4096 (64) 6.9 / 7.1 / 8.8 / 18.1    N 7168 (112) 10.9 / 9.9 / 10.1 / 18.6
//          N 14336 (224) 24.4 / 21.1 / 17.6 / 28.7    N 28672 (448) 46.9 / 42.7 / 37.6 / 37.6
//   M 64   N 4096 9.6 / 10.5 / 17.5 / 18.6    N 7168 16.5 / 11.9 / 17.6 / 19.0    N 14336 42.9 / 29.8 / 25.4 / 32.9
//          N 28672 77.9 / 58.9 / 46.7 / 42.4
//   M 128  N 4096 14.5 / 15.9 / - / 18.6    N 7168 25.6 / 17.1 / - / 19.2    N 14336 62.7 / 41.4 / - / 33.5
//   M 512  N 1024 13.7 / 15.9 / - / 18.3    M 2048, N 256 19.8 / 20.9 / - / 18.4    M 4096, N 128, K 1024 8.6 / 7.3 / - / 5.2
// A short K leaves most of the waves without a piece: few rows then go by 64 columns, which have
// the fewest, and more rows by tiles. Same order, us:
//   M 16   N 4096  K 512 3.7 / 3.6 / 3.2 / 4.2    K 1024 3.7 / 3.6 / 3.2 / 4.9    K 2048 3.7 / 4.0 / 4.3 / 6.6
//          N 7168  K 512 5.5 / 3.7 / 3.2 / 4.2    K 1024 5.5 / 3.7 / 4.0 / 4.9
//   M 128  N 1024  K 256 4.2 / 5.2 / - / 3.9    K 512 4.2 / 5.2 / - / 4.3
//          N 7168  K 512 7.4 / 5.4 / - / 4.5    K 1024 7.8 / 5.6 / - / 5.5
//   masked, 8 experts, N 2048: M_max 64  K 2048 13.9 / 11.0 / 10.6 / 9.0    K 7168 41.0 / 29.2 / 26.3 / 33.1
//                              M_max 96  K 2048 16.3 / 12.3 / 12.0 / 9.0    K 4608 25.9 / 19.9 / 19.2 / 15.2
//                                        K 7168 47.9 / 33.5 / 28.8 / 32.6
//           10 experts, N 1728: M_max 40  K 4608 21.1 / 18.7 / 18.0 / 15.1
Choice skinny(int layout, int M, int N, int K, int G, int force = -1) {
  Choice c;
  if (layout != FG_LAYOUT_MASKED) G = 1;
  const long w = ceil_div(M, kSkinnyRows) * ceil_div(N, 64) * G;
  int i = M > 4 * kSkinnyRows ? -1 : w <= 64 ? 0 : w <= 128 ? 1 : (w <= 256 && M <= 96) || M <= 16 ? 2 : -1;
  if (M <= 16 && K <= 1536 && K * w <= 90000) i = 2;
  if (M > 32 && K <= (w > 128 ? M > 64 ? 6000 : 20 * w : w > 64 ? 768 : 256)) i = -1;
  if (force >= 0) i = force;
  if (i < 0) return c;
  int steps = (int)ceil_div(M < kSkinnyRows ? M : kSkinnyRows, 16);
  if (steps > 4) steps = steps <= 6 ? 6 : 8;
  c.tile = kSkinny + 3 * (steps - 1) + i;
  c.grid = ceil_div(M, 16 * steps) * ceil_div(N, 16 << i) * G;
  return c.grid <= kMaxTiles ? c : Choice();
}

// The shape whose tiles, in rounds over the compute units, take the fewest estimated
// cycles; dense problems also try whole rounds of 256x256 tiles with the remaining
// columns on 256x128, contiguous ones the run-following kernel.
Choice choose(int layout, int M, int N, int K, int G, int cus) {
  Choice best;
  if (layout != FG_LAYOUT_CONTIGUOUS) best = skinny(layout, M, N, K, G);
  if (best.tile >= 0) return best;
  double cost = 0.0;
  const double kb = (double)ceil_div(K, 128);
  for (int i = 0; i < kNumTiles; ++i) {
    const Tile& t = kTiles[i];
    if (layout == FG_LAYOUT_CONTIGUOUS && t.bm > 128) continue;   // a tile's rows are one expert's
    const long tiles = ceil_div(M, t.bm) * ceil_div(N, t.bn) * (layout == FG_LAYOUT_MASKED ? G : 1);
    if (tiles > kMaxTiles) continue;
    const double c = (double)ceil_div(tiles, cus) * tile_cycles(t, kb);
    if (best.tile < 0 || c < cost) {
      best.tile = i;
      best.grid = tiles;
      cost = c;
    }
  }
  if (layout == FG_LAYOUT_CONTIGUOUS && ceil_div(M, 128) <= kRunMaxBlocks && G <= kRunMaxExperts) {
    // G runs, half of them odd (as many as leave whole pairs): full two-block tiles and single blocks per column
    const long nblk = ceil_div(M, 128), runs = G < nblk ? G : nblk, S = runs / 2 + ((nblk - runs / 2) & 1), F = (nblk - S) / 2;
    const long tn = ceil_div(N, 256), items = nblk * tn, grid = items < cus ? items : cus;
    const double tf = tile_cycles(kTiles[kWide], kb), th = tile_cycles(kTiles[kHalf], kb);
    const long full = F * tn, rest = full % grid;
    const double c = rest && 2 * rest + S * tn <= grid ? (double)(full / grid) * tf + th
                                                       : (double)ceil_div(full, grid) * tf + (double)ceil_div(S * tn, grid) * th;
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
      const double c = (double)(a / cus) * tile_cycles(kTiles[kWide], kb) + (double)ceil_div(b, cus) * tile_cycles(kTiles[kNarrow], kb);
      if (c < cost) {
        best.tile = kSplit;
        best.n_split = (int)nc;
        best.tiles_a = a;
        best.grid = (a > b ? a : b) < cus ? (a > b ? a : b) : cus;
      }
      break;
    }
  }
  return best;
}

#ifdef FG_TESTING
bool forced(int layout, int M, int N, int K, int G, int cus, Choice& c) {
  c = Choice();
  c.tile = t_tile;
  if (t_tile < kNumTiles) {
    const Tile& t = kTiles[t_tile];
    c.grid = ceil_div(M, t.bm) * ceil_div(N, t.bn) * (layout == FG_LAYOUT_MASKED ? G : 1);
    return layout != FG_LAYOUT_CONTIGUOUS || t.bm <= 128;
  }
  if (t_tile >= kSkinny) {
    c = skinny(layout, M, N, K, G, t_tile - kSkinny);
    return layout != FG_LAYOUT_CONTIGUOUS && !(M > 96 && t_tile == kSkinny + 2);
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
  if ((layout == FG_LAYOUT_MASKED ? G : 1) * ceil_div(M, top.bm) * ceil_div(N, top.bn) > kMaxTiles) return FG_EINVAL;
  int cus = 0;
  const int st = current_device(&cus);
  if (st != FG_OK) return st;
  Choice c = choose(layout, M, N, K, G, cus);
#ifdef FG_TESTING
  if (t_tile >= 0 && (!forced(layout, M, N, K, G, cus, c) || c.grid > kMaxTiles)) return FG_EINVAL;
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
