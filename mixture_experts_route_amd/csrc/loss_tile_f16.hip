// Tile products of the loss with fp16 operands.
#include "loss_tile.hpp"

namespace moe {

hipError_t launch_loss_f16(const TileArgs& a, int* tiles, hipStream_t st) { return launch_loss_t<_Float16>(a, tiles, st); }
hipError_t launch_loss_dz_f16(const TileArgs& a, hipStream_t st) { return launch_loss_dz_t<_Float16>(a, st); }
hipError_t launch_loss_dx_f16(const TileArgs& a, hipStream_t st) { return launch_loss_dx_t<_Float16>(a, st); }
hipError_t launch_loss_dw_f16(const TileArgs& a, hipStream_t st) { return launch_loss_dw_t<_Float16>(a, st); }

}  // namespace moe
