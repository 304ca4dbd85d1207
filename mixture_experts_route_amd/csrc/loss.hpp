// The loss over an output head (moe_loss_*): launches of its tile products.
#pragma once

#include "checks.hpp"
#include "dense.hpp"

namespace moe {

// Up to 64 tokens are bound by the weights' bytes, and 64-square tiles, five steps deep, draw them faster than a larger
// tile's mostly empty rows (5 tokens, 100003 x 2048: 86 us, 128-square 92).
inline int few_tokens_kernel(const TileArgs& a, int kernel) {
  const bool few = a.M <= 64 && g_dense_plan.kernel == MOE_DENSE_AUTO;
  return few && (kernel == MOE_DENSE_TILE128 || kernel == MOE_DENSE_TILE256) ? MOE_DENSE_TILE64 : kernel;
}

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
