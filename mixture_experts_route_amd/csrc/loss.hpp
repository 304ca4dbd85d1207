// The loss over an output head (moe_loss_*): launches of its tile products.
#pragma once

#include "checks.hpp"
#include "dense.hpp"

namespace moe {

// loss_tile_bf16.hip, loss_tile_f16.hip.  Logits with the forward's epilogue (*tiles: tiles_j, the rows of LossEpi::part),
// with the gradient's, and the two products that follow, summed onto earlier ones.
hipError_t launch_loss_bf16(const TileArgs& a, int* tiles, hipStream_t st);
hipError_t launch_loss_f16(const TileArgs& a, int* tiles, hipStream_t st);
hipError_t launch_loss_dz_bf16(const TileArgs& a, hipStream_t st);
hipError_t launch_loss_dz_f16(const TileArgs& a, hipStream_t st);
hipError_t launch_loss_dx_bf16(const TileArgs& a, hipStream_t st);
hipError_t launch_loss_dx_f16(const TileArgs& a, hipStream_t st);
hipError_t launch_loss_dw_bf16(const TileArgs& a, hipStream_t st);
hipError_t launch_loss_dw_f16(const TileArgs& a, hipStream_t st);

}  // namespace moe
