// Tile products of the dense operators with fp16 operands.
#include "dense_tile.hpp"

namespace moe {
hipError_t launch_tile_f16(const TileArgs& a, int oa, int ob, int kind, hipStream_t st) {
  return launch_tile_t<_Float16>(a, oa, ob, kind, st);
}
}  // namespace moe
