// qblk_mx_abi.hip -- the C ABI of the microscaling formats, their products and
// the norm with quantized output (declared in include/qblk.h).  Argument checks
// on the host, then launches on the caller's stream.
#include "../../include/qblk.h"
#include "qblk_checks.h"
#include "qblk_launch.h"
#include "qblk_norm.h"

namespace {

constexpr int kBlock = 32;
// Rows of one product: a workgroup of 512 threads takes 16 of them, and a launch
// holds at most 2^32 - 1 threads.  Columns: a tile's rows are addressed by 32-bit
// offsets.
constexpr int64_t kMaxMxRows = int64_t(1) << 26, kMaxMxCols = int64_t(1) << 23;
// Columns of a norm's row: a row's values are counted in 32 bits.
constexpr int64_t kMaxNormCols = int64_t(1) << 24;

bool mx_elem(int act) { return act == QBLK_ACT_MXFP8 || act == QBLK_ACT_MXFP4; }

// A matrix of rows x k values in blocks of 32 columns, of at most 4 bytes a value.
qblk_status_t check_mx(int64_t rows, int64_t k) {
  if (rows < 0 || k < 0 || rows > kMaxDim || k > kMaxDim || k % kBlock != 0) return QBLK_ERR_SHAPE;
  if (rows > 0 && k > 0 && rows > kMaxBytes / 4 / k) return QBLK_ERR_SHAPE;
  return QBLK_OK;
}

qblk_status_t check_bytes(const void* p, bool needed) { return needed && !p ? QBLK_ERR_NULL : QBLK_OK; }

bool product_shape_ok(int64_t m, int64_t k, int64_t n) {
  return check_mx(m, k) == QBLK_OK && m <= kMaxMxRows && k <= kMaxMxCols && check_mx(n, k) == QBLK_OK &&
         (m == 0 || n <= kMaxBytes / 4 / m);
}

qblk_status_t check_room(const void* work, size_t have, int64_t need) {
  if (need == 0) return QBLK_OK;
  if (!work) return QBLK_ERR_NULL;
  if (!aligned16(work)) return QBLK_ERR_ALIGN;
  return have < static_cast<uint64_t>(need) ? QBLK_ERR_WORKSPACE : QBLK_OK;
}

int64_t bytes_of_type(int t) { return t == QBLK_F32 ? 4 : 2; }

}  // namespace

extern "C" {

qblk_status_t qblk_quantize_mx(const void* v, qblk_dtype_t vt, int64_t rows, int64_t k, qblk_act_t elem, void* codes,
                               uint8_t* scale, qblk_stream_t stream) {
  QBLK_TRY(check_mx(rows, k));
  if (!dtype_ok(vt)) return QBLK_ERR_DTYPE;
  if (!mx_elem(elem)) return QBLK_ERR_FORMAT;
  const bool work = rows > 0 && k > 0;
  QBLK_TRY(check_ptr(v, work));
  QBLK_TRY(check_ptr(codes, work));
  QBLK_TRY(check_bytes(scale, work));
  if (!work) return QBLK_OK;
  return from_hip(qblk::launch_quantize_mx(v, vt, rows, k, elem == QBLK_ACT_MXFP8, static_cast<uint8_t*>(codes), scale,
                                           static_cast<hipStream_t>(stream)));
}

qblk_status_t qblk_dequant_mx(const void* codes, const uint8_t* scale, qblk_act_t elem, int64_t rows, int64_t k,
                              void* out, qblk_dtype_t ot, qblk_stream_t stream) {
  QBLK_TRY(check_mx(rows, k));
  if (!dtype_ok(ot)) return QBLK_ERR_DTYPE;
  if (!mx_elem(elem)) return QBLK_ERR_FORMAT;
  const bool work = rows > 0 && k > 0;
  QBLK_TRY(check_ptr(codes, work));
  QBLK_TRY(check_bytes(scale, work));
  QBLK_TRY(check_ptr(out, work));
  if (!work) return QBLK_OK;
  return from_hip(qblk::launch_dequant_mx(static_cast<const uint8_t*>(codes), scale, rows, k, elem == QBLK_ACT_MXFP8, out,
                                          ot, static_cast<hipStream_t>(stream)));
}

size_t qblk_gemm_mxfp4_workspace(int64_t m, int64_t k, int64_t n, qblk_act_t act) {
  if (!product_shape_ok(m, k, n) || !mx_elem(act) || m == 0 || k == 0 || n == 0) return 0;
  return static_cast<size_t>(qblk::gemm_mxfp4_workspace(m, k, n, act == QBLK_ACT_MXFP8));
}

qblk_status_t qblk_gemm_mxfp4(const uint8_t* w, const uint8_t* wscale, int64_t m, int64_t k, const void* xq,
                              const uint8_t* xscale, qblk_act_t act, int64_t n, void* y, qblk_dtype_t yt,
                              void* workspace, size_t workspace_bytes, qblk_stream_t stream) {
  if (!product_shape_ok(m, k, n)) return QBLK_ERR_SHAPE;
  if (!dtype_ok(yt)) return QBLK_ERR_DTYPE;
  if (!mx_elem(act)) return QBLK_ERR_FORMAT;
  const bool out = m > 0 && n > 0, work = out && k > 0, f8 = act == QBLK_ACT_MXFP8;
  QBLK_TRY(check_ptr(w, work));
  QBLK_TRY(check_bytes(wscale, work));
  QBLK_TRY(check_ptr(xq, work));
  QBLK_TRY(check_bytes(xscale, work));
  QBLK_TRY(check_ptr(y, out));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!out) return QBLK_OK;
  if (k == 0) return from_hip(qblk::launch_zero_bytes(y, m * n * bytes_of_type(yt), s));
  QBLK_TRY(check_room(workspace, workspace_bytes, qblk::gemm_mxfp4_workspace(m, k, n, f8)));
  return from_hip(qblk::launch_gemm_mxfp4(w, wscale, m, k, static_cast<const uint8_t*>(xq), xscale, f8, n, y, yt, workspace, s));
}

size_t qblk_linear_mxfp4_workspace(int64_t m, int64_t k, int64_t n, qblk_act_t act) {
  if (!product_shape_ok(m, k, n) || !mx_elem(act) || m == 0 || k == 0 || n == 0) return 0;
  return static_cast<size_t>(qblk::linear_mxfp4_workspace(m, k, n, act == QBLK_ACT_MXFP8));
}

qblk_status_t qblk_linear_mxfp4(const uint8_t* w, const uint8_t* wscale, int64_t m, int64_t k, const void* x,
                                qblk_dtype_t xt, qblk_act_t act, int64_t n, void* y, qblk_dtype_t yt, void* workspace,
                                size_t workspace_bytes, qblk_stream_t stream) {
  if (!product_shape_ok(m, k, n)) return QBLK_ERR_SHAPE;
  if (!dtype_ok(xt) || !dtype_ok(yt)) return QBLK_ERR_DTYPE;
  if (!mx_elem(act)) return QBLK_ERR_FORMAT;
  const bool out = m > 0 && n > 0, work = out && k > 0, f8 = act == QBLK_ACT_MXFP8;
  QBLK_TRY(check_ptr(w, work));
  QBLK_TRY(check_bytes(wscale, work));
  QBLK_TRY(check_ptr(x, work));
  QBLK_TRY(check_ptr(y, out));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!out) return QBLK_OK;
  if (k == 0) return from_hip(qblk::launch_zero_bytes(y, m * n * bytes_of_type(yt), s));
  QBLK_TRY(check_room(workspace, workspace_bytes, qblk::linear_mxfp4_workspace(m, k, n, f8)));
  return from_hip(qblk::launch_linear_mxfp4(w, wscale, m, k, x, xt, f8, n, y, yt, workspace, s));
}

qblk_status_t qblk_rmsnorm(const qblk_rmsnorm_t* a, qblk_stream_t stream) {
  if (!a) return QBLK_ERR_NULL;
  int step = 8;
  if (a->act == QBLK_ACT_F8) step = 128;
  if (mx_elem(a->act)) step = kBlock;
  if (a->act < QBLK_ACT_NONE || a->act > QBLK_ACT_MXFP4) return QBLK_ERR_FORMAT;
  if (a->n < 0 || a->n > kMaxDim || a->hidden < 0 || a->hidden > kMaxNormCols || a->hidden % step != 0) return QBLK_ERR_SHAPE;
  if (a->n > 0 && a->hidden > 0 && a->n > kMaxBytes / 4 / a->hidden) return QBLK_ERR_SHAPE;
  if (!dtype_ok(a->xt) || !dtype_ok(a->wt)) return QBLK_ERR_DTYPE;
  if (!(a->eps >= 0.0f)) return QBLK_ERR_SHAPE;
  const bool work = a->n > 0 && a->hidden > 0;
  QBLK_TRY(check_ptr(a->x, work));
  QBLK_TRY(check_ptr(a->weight, work));
  if (a->residual) {
    QBLK_TRY(check_ptr(a->residual, work));
    QBLK_TRY(check_ptr(a->total, work));
  }
  if (a->act == QBLK_ACT_NONE) {
    QBLK_TRY(check_ptr(a->y, work));
  } else {
    if (a->y) QBLK_TRY(check_ptr(a->y, work));
    QBLK_TRY(check_ptr(a->codes, work));
    if (mx_elem(a->act))
      QBLK_TRY(check_bytes(a->scale, work));
    else
      QBLK_TRY(check_ptr4(a->scale, work));
  }
  if (a->act == QBLK_ACT_I8 && a->hidden == 0 && a->n > 0) {  // rows without columns: scales of 0
    QBLK_TRY(check_ptr4(a->scale, true));
    return from_hip(qblk::launch_zero_bytes(a->scale, a->n * 4, static_cast<hipStream_t>(stream)));
  }
  if (!work) return QBLK_OK;
  qblk::NormArgs k;
  k.x = a->x;
  k.residual = a->residual;
  k.weight = a->weight;
  k.total = a->residual ? a->total : nullptr;
  k.y = a->y;
  k.codes = static_cast<uint8_t*>(a->codes);
  k.scale = a->scale;
  k.row0 = k.end = 0;
  k.eps = a->eps;
  k.hidden = static_cast<int>(a->hidden);
  k.xt = a->xt;
  k.wt = a->wt;
  k.act = a->act;
  return from_hip(qblk::launch_rmsnorm(k, a->n, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
