// A kernel's limit of dynamic LDS.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace qn {

// The limit is an attribute of the kernel on a device: set on the current one ahead of the
// kernel's first launch there (asked of the runtime before every launch it would be host time
// of every call; once a process, launches on the other devices would be without it).  One
// object a kernel; an error is not kept.
class LdsLimit {
 public:
  hipError_t operator()(const void* kernel, size_t bytes) {
    int dev = 0;
    const hipError_t got = hipGetDevice(&dev);
    if (got != hipSuccess) return got;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;  // (past 64 devices: every time)
    if (done_.load(std::memory_order_acquire) & bit) return hipSuccess;
    const hipError_t set =
        hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (set == hipSuccess) done_.fetch_or(bit, std::memory_order_release);
    return set;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace qn
