// Tile products of the dense operators with bf16 operands.
#include "dense_tile.hpp"

namespace moe {

hipError_t launch_forward_bf16(const TileArgs& a, int kind, hipStream_t st) { return launch_forward_t<__bf16>(a, kind, st); }

hipError_t launch_backward_bf16(const TileArgs& dx, const TileArgs& dw, const BiasSumArgs& db, hipStream_t st) {
  return launch_backward_t<__bf16>(dx, dw, db, st);
}

}  // namespace moe
