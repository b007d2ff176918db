// Instantiations of the tiled product (qlr_tile.h): the gated block's forward.
#include "qlr_tile.h"

namespace qlr {

hipError_t launch_gated_gemm(const TrainArgs& a, const Levels& lv, hipStream_t s) {
  switch (a.bits) {
    case 2: return launch_tile<TILE_GATED, 2>(a, lv, s);
    case 3: return launch_tile<TILE_GATED, 3>(a, lv, s);
    case 4: return launch_tile<TILE_GATED, 4>(a, lv, s);
    default: return launch_tile<TILE_GATED, 8>(a, lv, s);
  }
}

}  // namespace qlr
