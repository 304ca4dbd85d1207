// Tile products of the dense operators with fp16 operands.
#include "dense_tile.hpp"

namespace moe {

hipError_t launch_forward_f16(const TileArgs& a, int kind, hipStream_t st) { return launch_forward_t<_Float16>(a, kind, st); }

hipError_t launch_backward_f16(const TileArgs& dx, const TileArgs& dw, const BiasSumArgs& db, hipStream_t st) {
  return launch_backward_t<_Float16>(dx, dw, db, st);
}

}  // namespace moe
