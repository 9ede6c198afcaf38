// fg_int8_launch.hip -- kernel instantiations of the 8-bit integer product for one
// layout: FG_INT8_LAYOUT = 0 dense, 1 contiguous, 2 masked.
#include <hip/hip_runtime.h>

#include "fg_int8_tiles.hpp"

#ifndef FG_INT8_LAYOUT
#error "FG_INT8_LAYOUT selects the layout of this object"
#endif

namespace fg {

namespace {
template <int LAYOUT, class C>
hipError_t launch_tile(const Params& p, int grid, hipStream_t s) {
  if constexpr (LAYOUT == kContiguous && C::BM > 128) {
    return hipErrorInvalidValue;   // 256-row tiles follow the experts' runs (kRuns)
  } else {
    hipLaunchKernelGGL((int8_gemm<LAYOUT, C>), dim3(grid), dim3(C::THREADS), 0, s, p);
    return hipGetLastError();
  }
}
template <int LAYOUT, class C>
hipError_t launch_one_skinny(const Params& p, int grid, hipStream_t s) {
  if constexpr (LAYOUT == kContiguous && 8 % C::TM != 0) {
    return hipErrorInvalidValue;   // a block of rows is within one of 128
  } else {
    hipLaunchKernelGGL((int8_skinny<LAYOUT, C>), dim3(grid), dim3(64 * C::WAVES), 0, s, p);
    return hipGetLastError();
  }
}
template <int LAYOUT, int TM>
hipError_t launch_skinny(int i, const Params& p, int grid, hipStream_t s) {
  switch (i) {
    case 0: return launch_one_skinny<LAYOUT, int8_cfg::Skinny<TM, 0>>(p, grid, s);
    case 1: return launch_one_skinny<LAYOUT, int8_cfg::Skinny<TM, 1>>(p, grid, s);
    default:
      if constexpr (TM <= 6) return launch_one_skinny<LAYOUT, int8_cfg::Skinny<TM, 2>>(p, grid, s);
      else return hipErrorInvalidValue;
  }
}
}  // namespace

template <int LAYOUT>
hipError_t launch_int8(int tile, const Params& p, int grid, hipStream_t s) {
  using namespace int8_cfg;
  switch (tile) {
    case 0: return launch_tile<LAYOUT, Cfg0>(p, grid, s);
    case 1: return launch_tile<LAYOUT, Cfg1>(p, grid, s);
    case 2: return launch_tile<LAYOUT, Cfg2>(p, grid, s);
    case 3: return launch_tile<LAYOUT, Cfg3>(p, grid, s);
    case 4: return launch_tile<LAYOUT, Cfg4>(p, grid, s);
    case 5: return launch_tile<LAYOUT, Cfg5>(p, grid, s);
    case kSplit:
      if constexpr (LAYOUT == kDense) {
        hipLaunchKernelGGL((int8_gemm_split<Cfg0, Cfg1>), dim3(grid), dim3(Cfg0::THREADS), 0, s, p);
        return hipGetLastError();
      } else {
        return hipErrorInvalidValue;
      }
    case kRuns:
      if constexpr (LAYOUT == kContiguous) {
        hipLaunchKernelGGL((int8_gemm_runs<Cfg0, Cfg2, CfgQ>), dim3(grid), dim3(Cfg0::THREADS), 0, s, p);
        return hipGetLastError();
      } else {
        return hipErrorInvalidValue;
      }
    default: break;
  }
  const int i = (tile - kSkinny) % 3;
  switch ((tile - kSkinny) / 3 + 1) {
    case 1: return launch_skinny<LAYOUT, 1>(i, p, grid, s);
    case 2: return launch_skinny<LAYOUT, 2>(i, p, grid, s);
    case 3: return launch_skinny<LAYOUT, 3>(i, p, grid, s);
    case 4: return launch_skinny<LAYOUT, 4>(i, p, grid, s);
    case 6: return launch_skinny<LAYOUT, 6>(i, p, grid, s);
    case 8: return launch_skinny<LAYOUT, 8>(i, p, grid, s);
    default: return hipErrorInvalidValue;
  }
}

template hipError_t launch_int8<FG_INT8_LAYOUT>(int, const Params&, int, hipStream_t);

}  // namespace fg
