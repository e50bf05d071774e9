// Host-side helpers shared by the files of the C ABI (sbl_api.hip, sbl_api_step.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sbl {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool ranges_overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a && b && a0 < b0 + (uintptr_t)nb && b0 < a0 + (uintptr_t)na;
}

// SBL_OK, or SBL_ERR_LAUNCH with the error kept for sbl_last_hip_error()
int launch_status(hipError_t e);

}  // namespace sbl
