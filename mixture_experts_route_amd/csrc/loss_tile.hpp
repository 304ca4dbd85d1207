// Tile products of the loss, by operand type.
#pragma once

#include "dense_tile.hpp"
#include "loss.hpp"

namespace moe {

template <typename T>
hipError_t launch_loss_t(const TileArgs& args, int* tiles, hipStream_t st) {
  TileArgs a = args;
  DensePlan plan{};
  double us;
  const hipError_t e = prepare_tile<kRows, kRows, kEpiLoss>(a, plan, us, st);
  if (e != hipSuccess) return e;
  plan.kernel = few_tokens_kernel(a, plan.kernel);
  const int tile = plan.kernel == MOE_DENSE_TILE256 ? 256 : plan.kernel == MOE_DENSE_TILE64 || plan.kernel == MOE_DENSE_ANY64 ? 64 : 128;
  *tiles = (a.N + tile - 1) / tile;
  return start_plan<T, kRows, kRows, kEpiLoss>(a, plan.kernel, st);
}

template <typename T>
hipError_t launch_loss_dz_t(const TileArgs& a, hipStream_t st) { return launch_tile_k<T, kRows, kRows, kEpiLossDz>(a, st); }

// (k_tile_any of 128-square tiles is five registers over in this one: three scratch stores and three loads of a lane)
template <typename T>
hipError_t launch_loss_dx_t(const TileArgs& a, hipStream_t st) { return launch_tile_k<T, kRows, kCols, kEpiSum>(a, st); }

template <typename T>
hipError_t launch_loss_dw_t(const TileArgs& a, hipStream_t st) { return launch_tile_k<T, kCols, kCols, kEpiSum>(a, st); }

}  // namespace moe
