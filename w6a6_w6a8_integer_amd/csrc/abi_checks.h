// abi_checks.h -- host-side argument checks shared by the C ABI files.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/flexq.h"

namespace flexq {

struct Range {
  uintptr_t lo, hi;
};

inline Range range_of(const void* p, uint64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + (uintptr_t)bytes};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline flexq_status launched(hipError_t e) {
  return e == hipSuccess ? FLEXQ_SUCCESS : FLEXQ_ERROR_LAUNCH;
}

}  // namespace flexq

#define FLEXQ_TRY(expr)                 \
  do {                                  \
    const flexq_status s_ = (expr);     \
    if (s_ != FLEXQ_SUCCESS) return s_; \
  } while (0)
