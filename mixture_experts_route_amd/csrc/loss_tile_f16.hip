// Tile products of the loss with fp16 operands.
#include "dense_tile.hpp"
#include "loss.hpp"

namespace moe {

hipError_t launch_loss_f16(const TileArgs& args, int* tiles, hipStream_t st) {
  TileArgs a = args;
  DensePlan plan{};
  double us;
  const hipError_t e = prepare_tile<kRows, kRows, kEpiLoss>(a, plan, us, st);
  if (e != hipSuccess) return e;
  plan.kernel = few_tokens_kernel(a, plan.kernel);
  const int tile = plan.kernel == MOE_DENSE_TILE256 ? 256 : plan.kernel == MOE_DENSE_TILE64 || plan.kernel == MOE_DENSE_ANY64 ? 64 : 128;
  *tiles = (a.N + tile - 1) / tile;
  return start_plan<_Float16, kRows, kRows, kEpiLoss>(a, plan.kernel, st);
}

hipError_t launch_loss_dz_f16(const TileArgs& a, hipStream_t st) { return launch_tile_k<_Float16, kRows, kRows, kEpiLossDz>(a, st); }

hipError_t launch_loss_dx_f16(const TileArgs& a, hipStream_t st) { return launch_tile_k<_Float16, kRows, kCols, kEpiSum>(a, st); }

hipError_t launch_loss_dw_f16(const TileArgs& a, hipStream_t st) { return launch_tile_k<_Float16, kCols, kCols, kEpiSum>(a, st); }

}  // namespace moe
