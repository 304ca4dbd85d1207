// Tile products of the dense operators with bf16 operands.
#include "dense_tile.hpp"

namespace moe {
hipError_t launch_tile_bf16(const TileArgs& a, int oa, int ob, int kind, hipStream_t st) {
  return launch_tile_t<__bf16>(a, oa, ob, kind, st);
}
}  // namespace moe
