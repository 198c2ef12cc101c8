// qblk_lds.h -- kernels with more dynamic LDS than a launch gets unasked (internal, host).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace qblk {

// Lets `kernel` use `bytes` of dynamic LDS on the current device.  The limit is an
// attribute of the kernel on one device, so it is set once on each; `done` (one for each
// kernel) remembers where.
inline hipError_t allow_lds(std::atomic<uint64_t>& done, const void* kernel, int bytes) {
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  const hipError_t set = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (set == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return set;
}

}  // namespace qblk
