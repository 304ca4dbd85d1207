// The experts' products with bf16 operands.
#include "experts_tile.hpp"

namespace moe {

hipError_t launch_experts_forward_bf16(const GroupArgs& g, int kind, hipStream_t st) { return launch_experts_forward_t<__bf16>(g, kind, st); }

hipError_t launch_experts_dx_bf16(const GroupArgs& g, hipStream_t st) { return launch_experts<__bf16, kRows, kCols, kEpiStore>(g, st); }

hipError_t launch_experts_dw_bf16(const GroupArgs& g, hipStream_t st) { return launch_experts<__bf16, kCols, kCols, kEpiStore>(g, st); }

}  // namespace moe
