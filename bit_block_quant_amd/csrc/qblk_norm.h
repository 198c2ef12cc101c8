// qblk_norm.h -- arguments of the norm kernel (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qblk {

struct NormArgs {
  const void* x;
  const void* residual;  // or nullptr
  const void* weight;
  void* total;  // with a residual
  void* y;      // or nullptr
  uint8_t* codes;
  void* scale;
  int64_t row0, end;  // rows of this launch
  float eps;
  int hidden, xt, wt, act;
};

hipError_t launch_rmsnorm(const NormArgs& a, int64_t n, hipStream_t s);

}  // namespace qblk
