// Host-side helpers shared by the files of the C ABI (sbl_api.hip, sbl_api_step.hip) and by launches.
#pragma once

#include <atomic>

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sbl {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool ranges_overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a && b && a0 < b0 + (uintptr_t)nb && b0 < a0 + (uintptr_t)na;
}

// The dynamic LDS that a kernel may ask for, raised past its default once on each GPU: the limit
// belongs to the kernel on one device.  One object for each kernel; any threads may share it.
class LdsLimit {
 public:
  hipError_t raise(const void* kernel, int bytes) {
    int device = 0;
    hipError_t e = hipGetDevice(&device);
    if (e != hipSuccess) return e;
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if (done_.load(std::memory_order_relaxed) & bit) return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess) done_.fetch_or(bit, std::memory_order_relaxed);
    else (void)hipGetLastError();                // reported here, not by the next call's launch as well
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// SBL_OK, or SBL_ERR_LAUNCH with the error kept for sbl_last_hip_error()
int launch_status(hipError_t e);

}  // namespace sbl
