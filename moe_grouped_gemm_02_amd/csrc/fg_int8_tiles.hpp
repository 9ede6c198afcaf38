// fg_int8_tiles.hpp -- the compiled tile configurations of the 8-bit integer product
// and the launcher of one layout (fg_int8_launch.hip, built once per layout).
#pragma once

#include <hip/hip_runtime.h>

#include "fg_int8_kernel.hpp"

namespace fg {
namespace int8_cfg {
// rows x columns of D per workgroup; the host's tile table lists them in this order
using Cfg0 = Int8Cfg<256, 256, 4, 2, 2, 3>;
using Cfg1 = Int8Cfg<256, 128, 4, 2, 3, 3>;
using Cfg2 = Int8Cfg<128, 256, 2, 4, 3, 3>;
using Cfg3 = Int8Cfg<128, 128, 2, 2, 4, 3>;
using Cfg4 = Int8Cfg<64, 128, 2, 2, 3, 3>;
using Cfg5 = Int8Cfg<128, 160, 4, 1, 3, 3>;
using CfgQ = Int8Cfg<64, 128, 2, 4, 4, 1>;   // quarters of Cfg2's tiles
constexpr int kSplit = 6;   // dense: int8_gemm_split<Cfg0, Cfg1>
constexpr int kRuns = 7;    // contiguous: int8_gemm_runs<Cfg0, Cfg2, CfgQ>
// row blocks of 16 TM rows (contiguous: TM 1, 2, 4, 8): int8_skinny on kSkinny + 3 * (TM - 1) + i, i for 16, 32 or 64 columns.
// LDS up to 160 KB where there is one workgroup a CU at most, 80 KB or less where two are resident (64 columns).
constexpr int kSkinny = 8, kSkinnyRows = 128;
template <int TM, int I>
struct Skinny;
#define FG_SKINNY(TM, I, W, S) \
  template <>                  \
  struct Skinny<TM, I> : SkinnyCfg<TM, 1 << I, W, S> {};
FG_SKINNY(1, 0, 8, 5) FG_SKINNY(1, 1, 8, 3) FG_SKINNY(1, 2, 4, 2)
FG_SKINNY(2, 0, 8, 3) FG_SKINNY(2, 1, 4, 4) FG_SKINNY(2, 2, 3, 2)
FG_SKINNY(3, 0, 4, 4) FG_SKINNY(3, 1, 4, 3) FG_SKINNY(3, 2, 2, 2)
FG_SKINNY(4, 0, 4, 4) FG_SKINNY(4, 1, 4, 3) FG_SKINNY(4, 2, 2, 2)
FG_SKINNY(6, 0, 4, 2) FG_SKINNY(6, 1, 4, 2) FG_SKINNY(6, 2, 2, 2)
FG_SKINNY(8, 0, 4, 2) FG_SKINNY(8, 1, 4, 2)
#undef FG_SKINNY
}  // namespace int8_cfg

template <int LAYOUT>
hipError_t launch_int8(int tile, const Params& p, int grid, hipStream_t s);

}  // namespace fg
