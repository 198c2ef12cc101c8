// qblk_checks.h -- host-side argument checks shared by the C ABI sources.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qblk.h"

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
// Rows of one qblk_gemm / qblk_gemm_w4a8 call: the product kernels run up to
// 8 threads per row in one launch, which holds at most 2^32 - 1 threads.
constexpr int64_t kMaxGemmRows = int64_t(1) << 28;
constexpr int64_t kMaxBytes = int64_t(1) << 40;

int elems_of(int fmt) {
  switch (fmt) {
    case QBLK_Q4_0: return 32;
    case QBLK_W4G128: return 128;
    case QBLK_SB4:
    case QBLK_SB4_AFFINE:
    case QBLK_Q4_K: return 256;
    default: return 0;
  }
}

size_t bytes_of(int fmt) {
  switch (fmt) {
    case QBLK_Q4_0: return 18;
    case QBLK_SB4: return 138;
    case QBLK_SB4_AFFINE: return 148;
    case QBLK_Q4_K: return 144;
    case QBLK_W4G128: return 66;  // 64 code bytes + a 2-byte scale, in two planes
    default: return 0;
  }
}

bool dtype_ok(int t) { return t == QBLK_F32 || t == QBLK_F16 || t == QBLK_BF16; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shape of a packed rows x k matrix: sizes in range, k a multiple of the block.
qblk_status_t check_shape(int fmt, int64_t rows, int64_t k) {
  const int e = elems_of(fmt);
  if (e == 0) return QBLK_ERR_FORMAT;
  if (rows < 0 || k < 0 || rows > kMaxDim || k > kMaxDim || k % e != 0) return QBLK_ERR_SHAPE;
  if (rows > 0 && k > 0 && rows * (k / e) > kMaxBytes / static_cast<int64_t>(bytes_of(fmt)))
    return QBLK_ERR_SHAPE;
  return QBLK_OK;
}

qblk_status_t check_ptr(const void* p, bool needed) {
  if (!needed) return QBLK_OK;
  if (!p) return QBLK_ERR_NULL;
  if (!aligned16(p)) return QBLK_ERR_ALIGN;
  return QBLK_OK;
}

// fp32 scale arrays (one per token) are read element by element: 4-byte
// alignment, so that a slice of them starting at any token is accepted
qblk_status_t check_ptr4(const void* p, bool needed) {
  if (!needed) return QBLK_OK;
  if (!p) return QBLK_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return QBLK_ERR_ALIGN;
  return QBLK_OK;
}

qblk_status_t from_hip(hipError_t e) { return e == hipSuccess ? QBLK_OK : QBLK_ERR_LAUNCH; }

#define QBLK_TRY(expr)                 \
  do {                                 \
    const qblk_status_t st_ = (expr);  \
    if (st_ != QBLK_OK) return st_;    \
  } while (0)

}  // namespace
