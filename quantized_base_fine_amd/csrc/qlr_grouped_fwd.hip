// Instantiations of the tiled expert product (qlr_tile.h): forward, y = x W'_e^T.
#include "qlr_tile.h"

namespace qlr {

namespace {

template <int BITS>
hipError_t launch_b(const TileArgs& a, const Levels& lv, hipStream_t s) {
  return launch_tile<TILE_CODED, BITS>(a, lv, s);
}

}  // namespace

hipError_t launch_grouped_gemm(const TileArgs& a, const Levels& lv, hipStream_t s) {
  switch (a.bits) {
    case 2: return launch_b<2>(a, lv, s);
    case 3: return launch_b<3>(a, lv, s);
    case 4: return launch_b<4>(a, lv, s);
    default: return launch_b<8>(a, lv, s);
  }
}

}  // namespace qlr
