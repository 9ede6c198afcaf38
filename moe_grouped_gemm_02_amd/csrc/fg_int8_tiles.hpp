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
constexpr int kSplit = 5;   // dense: int8_gemm_split<Cfg0, Cfg1>
constexpr int kRuns = 6;    // contiguous: int8_gemm_runs<Cfg0, Cfg2>
}  // namespace int8_cfg

template <int LAYOUT>
hipError_t launch_int8(int tile, const Params& p, int grid, hipStream_t s);

}  // namespace fg
