// The experts' products with fp16 operands.
#include "experts_tile.hpp"

namespace moe {

hipError_t launch_experts_forward_f16(const GroupArgs& g, int kind, hipStream_t st) { return launch_experts_forward_t<_Float16>(g, kind, st); }

hipError_t launch_experts_dx_f16(const GroupArgs& g, hipStream_t st) { return launch_experts<_Float16, kRows, kCols, kEpiStore>(g, st); }

hipError_t launch_experts_dw_f16(const GroupArgs& g, hipStream_t st) { return launch_experts<_Float16, kCols, kCols, kEpiStore>(g, st); }

}  // namespace moe
