// Instantiations of the tiled product (qlr_tile.h): the layer's forward over ranges of its contraction.
#include "qlr_tile.h"

namespace qlr {

namespace {

template <int BITS>
hipError_t launch_lin(TrainArgs a, const Levels& lv, hipStream_t s) {
  a.rest = 0;
  return a.M <= 64 ? launch_tile_t<TILE_LIN, BITS, 64, 128>(a, lv, s) : launch_tile_t<TILE_LIN, BITS, 128, 128>(a, lv, s);
}

}  // namespace

hipError_t launch_drop_fwd(const TrainArgs& a, const Levels& lv, hipStream_t s) {
  switch (a.bits) {
    case 2: return launch_lin<2>(a, lv, s);
    case 3: return launch_lin<3>(a, lv, s);
    case 4: return launch_lin<4>(a, lv, s);
    default: return launch_lin<8>(a, lv, s);
  }
}

}  // namespace qlr
