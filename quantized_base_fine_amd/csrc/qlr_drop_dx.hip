// Instantiations of the tiled product (qlr_tile.h): input gradient under adapter dropout.
#include "qlr_tile.h"

namespace qlr {

hipError_t launch_drop_dx(const TrainArgs& a, const Levels& lv, hipStream_t s) {
  switch (a.bits) {
    case 2: return launch_tile<TILE_TRD, 2>(a, lv, s);
    case 3: return launch_tile<TILE_TRD, 3>(a, lv, s);
    case 4: return launch_tile<TILE_TRD, 4>(a, lv, s);
    default: return launch_tile<TILE_TRD, 8>(a, lv, s);
  }
}

}  // namespace qlr
