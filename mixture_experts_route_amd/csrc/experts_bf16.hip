// The experts' products with bf16 operands.
#include "experts_tile.hpp"

namespace moe {

hipError_t launch_experts_forward_bf16(const GroupArgs& g, int kind, hipStream_t st) { return launch_experts_forward_t<__bf16>(g, kind, st); }

hipError_t launch_experts_backward_bf16(const GroupArgs& dx, const GroupArgs& dw, hipStream_t st) {
  return launch_experts_backward_t<__bf16>(dx, dw, st);
}

}  // namespace moe
