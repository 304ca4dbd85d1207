// Tile products of the loss with bf16 operands.
#include "loss_tile.hpp"

namespace moe {

hipError_t launch_loss_bf16(const TileArgs& a, int* tiles, hipStream_t st) { return launch_loss_t<__bf16>(a, tiles, st); }
hipError_t launch_loss_dz_bf16(const TileArgs& a, hipStream_t st) { return launch_loss_dz_t<__bf16>(a, st); }
hipError_t launch_loss_dx_bf16(const TileArgs& a, hipStream_t st) { return launch_loss_dx_t<__bf16>(a, st); }
hipError_t launch_loss_dw_bf16(const TileArgs& a, hipStream_t st) { return launch_loss_dw_t<__bf16>(a, st); }

}  // namespace moe
