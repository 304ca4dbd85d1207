// Host-side checks that the operators on caller-strided matrices share.
#pragma once

#include "kernels.hpp"

namespace moe {

inline size_t dense_align(size_t v) { return (v + 255) & ~(size_t)255; }
inline int dense_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

inline int check_tokens(int32_t T) {
  if (T < 1) return MOE_EINVAL;
  return T > MOE_DENSE_MAX_TOKENS ? MOE_EUNSUPPORTED : MOE_OK;
}

// Collects the checks of a call's matrices: element-aligned, rows that do not overlap, strides in range.
struct Mats {
  int rc = MOE_OK;
  void fail(int code) {
    if (rc == MOE_OK) rc = code;
  }
  void need(const void* p, int64_t ld, int64_t len, int elem = 2) {
    if (!p) fail(MOE_EINVAL);
    else opt(p, ld, len, elem);
  }
  void opt(const void* p, int64_t ld, int64_t len, int elem = 2) {
    if (!p) return;
    if ((uintptr_t)p % elem || ld < len) fail(MOE_EINVAL);
    else if (ld > MOE_DENSE_MAX_LD) fail(MOE_EUNSUPPORTED);
  }
  void vec(const void* p) { opt(p, 1, 1); }
};

}  // namespace moe
