// The experts' products with fp16 operands.
#include "experts_tile.hpp"

namespace moe {

hipError_t launch_experts_forward_f16(const GroupArgs& g, int kind, hipStream_t st) { return launch_experts_forward_t<_Float16>(g, kind, st); }

hipError_t launch_experts_backward_f16(const GroupArgs& dx, const GroupArgs& dw, hipStream_t st) {
  return launch_experts_backward_t<_Float16>(dx, dw, st);
}

}  // namespace moe
