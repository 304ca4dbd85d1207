// The experts' products (moe_experts_*): launch arguments.
#pragma once

#include "checks.hpp"
#include "dense.hpp"

namespace moe {

// A tile product per expert.  tile.a[] are whole [rows][..] matrices of which expert e has the rows offsets[e] ..
// offsets[e+1] - 1; tile.b[] and the results without such rows are [E] matrices, this many elements apart.
//   forward, dx   the rows are the outputs i: tile.M is left to the device, results are [rows][..] too
//   dW            the rows are the reduction: tile.R is left to the device, A and B are both [rows][..]
struct GroupArgs {
  TileArgs tile;
  const int32_t* offsets;
  int32_t* ctrl;
  int32_t E, P;        // experts, rows that the matrices have
  int64_t stride;      // of the weights, or of dW
  int32_t mats;        // dW: 1 or 2 (tile.a[m], tile.epi.y[m])
};

// experts_bf16.hip, experts_f16.hip
hipError_t launch_experts_forward_bf16(const GroupArgs& a, int epi_kind, hipStream_t st);
hipError_t launch_experts_forward_f16(const GroupArgs& a, int epi_kind, hipStream_t st);
// dx.tile.nseg or dw.mats 0: not wanted
hipError_t launch_experts_backward_bf16(const GroupArgs& dx, const GroupArgs& dw, hipStream_t st);
hipError_t launch_experts_backward_f16(const GroupArgs& dx, const GroupArgs& dw, hipStream_t st);

}  // namespace moe
