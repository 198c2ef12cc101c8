// qblk_ffn_abi.hip -- the C ABI of the feed-forward operators (declared in
// include/qblk.h): the 8-bit products with a scale for each block of 128, the
// gated layer built from them and the mixture-of-experts layer.  Argument
// checks on the host, then launches on the caller's stream.
#include "../../include/qblk.h"
#include "qblk_checks.h"
#include "qblk_launch.h"
#include "qblk_moe.h"

namespace {

constexpr int kF8Group = 128;
// Rows of one 8-bit matrix: a workgroup of 512 threads takes 16 of them, and
// a launch holds at most 2^32 - 1 threads.
constexpr int64_t kMaxF8Rows = int64_t(1) << 26;
// Columns of a product: a tile's 256 rows are addressed by 32-bit offsets.
constexpr int64_t kMaxF8Cols = int64_t(1) << 24;

// An 8-bit matrix of rows x k codes (k a multiple of 128).
qblk_status_t check_f8(int64_t rows, int64_t k) {
  if (rows < 0 || k < 0 || rows > kMaxDim || k > kMaxDim || k % kF8Group != 0) return QBLK_ERR_SHAPE;
  if (rows > 0 && k > 0 && rows > kMaxBytes / k) return QBLK_ERR_SHAPE;
  return QBLK_OK;
}

// n rows of `per` values of at most 4 bytes stay below 2^40 bytes
qblk_status_t check_rows(int64_t n, int64_t per) {
  if (n < 0 || n > kMaxDim) return QBLK_ERR_SHAPE;
  if (n > 0 && per > 0 && n > kMaxBytes / 4 / per) return QBLK_ERR_SHAPE;
  return QBLK_OK;
}

qblk_status_t check_work(const void* work, size_t have, int64_t need) {
  if (need == 0) return QBLK_OK;
  if (!work) return QBLK_ERR_NULL;
  if (!aligned16(work)) return QBLK_ERR_ALIGN;
  return have < static_cast<uint64_t>(need) ? QBLK_ERR_WORKSPACE : QBLK_OK;
}

int64_t bytes_of_type(int t) { return t == QBLK_F32 ? 4 : 2; }

bool gemm_shape_ok(int64_t m, int64_t k, int64_t n) {
  return check_f8(m, k) == QBLK_OK && m <= kMaxF8Rows && k <= kMaxF8Cols && check_rows(n, k) == QBLK_OK &&
         check_rows(n, m) == QBLK_OK;
}

// hidden and inter of a gated layer: each is the columns of one matrix
bool ffn_shape_ok(int64_t hidden, int64_t inter, int64_t n) {
  return hidden >= 0 && inter >= 0 && inter <= kMaxF8Rows / 2 && gemm_shape_ok(2 * inter, hidden, n) &&
         gemm_shape_ok(hidden, inter, n);
}

qblk_status_t moe_shape(const qblk_moe_t& a) {
  const int e = elems_of(a.fmt);
  if (e == 0) return QBLK_ERR_FORMAT;
  if (a.fmt == QBLK_W4G128) return QBLK_ERR_UNSUPPORTED;  // its products take 8-bit activations
  if (a.n < 0 || a.n > kMaxDim || a.hidden < 0 || a.inter < 0 || a.hidden % e != 0 || a.inter % e != 0)
    return QBLK_ERR_SHAPE;
  if (a.hidden > qblk::kMoeMaxDim || a.inter > qblk::kMoeMaxDim) return QBLK_ERR_SHAPE;
  if (a.experts < 1 || a.experts > qblk::kMoeMaxExperts || a.top_k < 1 || a.top_k > qblk::kMoeMaxTopK ||
      a.top_k > a.experts)
    return QBLK_ERR_SHAPE;
  QBLK_TRY(check_shape(a.fmt, a.experts * 2 * a.inter, a.hidden));
  QBLK_TRY(check_shape(a.fmt, a.experts * a.hidden, a.inter));
  QBLK_TRY(check_rows(a.n, a.hidden));
  return QBLK_OK;
}

int64_t moe_work(const qblk_moe_t& a) {
  if (a.n == 0 || a.hidden == 0 || a.inter == 0) return 0;
  const int64_t all = a.n < qblk::kMoeMaxPairs ? a.n * a.top_k : qblk::kMoeMaxPairs;
  const int64_t pairs = all < qblk::kMoeMaxPairs ? all : qblk::kMoeMaxPairs;
  return qblk::moe_table_bytes() + pairs * a.inter * 4;
}

}  // namespace

extern "C" {

qblk_status_t qblk_quantize_f8(const void* w, qblk_dtype_t wt, int64_t rows, int64_t k, uint8_t* codes, float* scale,
                               qblk_stream_t stream) {
  QBLK_TRY(check_f8(rows, k));
  if (!dtype_ok(wt)) return QBLK_ERR_DTYPE;
  const bool work = rows > 0 && k > 0;
  QBLK_TRY(check_ptr(w, work));
  QBLK_TRY(check_ptr(codes, work));
  QBLK_TRY(check_ptr4(scale, work));
  if (!work) return QBLK_OK;
  return from_hip(qblk::launch_quantize_f8(w, wt, rows, k, codes, scale, static_cast<hipStream_t>(stream)));
}

qblk_status_t qblk_quantize_act_f8(const void* x, qblk_dtype_t xt, int64_t n, int64_t k, uint8_t* xq, float* scale,
                                   qblk_stream_t stream) {
  QBLK_TRY(check_f8(n, k));
  if (!dtype_ok(xt)) return QBLK_ERR_DTYPE;
  const bool work = n > 0 && k > 0;
  QBLK_TRY(check_ptr(x, work));
  QBLK_TRY(check_ptr(xq, work));
  QBLK_TRY(check_ptr4(scale, work));
  if (!work) return QBLK_OK;
  return from_hip(qblk::launch_quantize_act_f8(x, xt, n, k, xq, scale, static_cast<hipStream_t>(stream)));
}

size_t qblk_gemm_f8_workspace(int64_t m, int64_t k, int64_t n) {
  if (!gemm_shape_ok(m, k, n) || m == 0 || k == 0 || n == 0) return 0;
  return static_cast<size_t>(qblk::gemm_f8_workspace(m, k, n));
}

qblk_status_t qblk_gemm_f8(const uint8_t* w, const float* wscale, int64_t m, int64_t k, const uint8_t* xq,
                           const float* xscale, int64_t n, void* y, qblk_dtype_t yt, void* workspace,
                           size_t workspace_bytes, qblk_stream_t stream) {
  if (!gemm_shape_ok(m, k, n)) return QBLK_ERR_SHAPE;
  if (!dtype_ok(yt)) return QBLK_ERR_DTYPE;
  const bool out = m > 0 && n > 0, work = out && k > 0;
  QBLK_TRY(check_ptr(w, work));
  QBLK_TRY(check_ptr4(wscale, work));
  QBLK_TRY(check_ptr(xq, work));
  QBLK_TRY(check_ptr4(xscale, work));
  QBLK_TRY(check_ptr(y, out));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!out) return QBLK_OK;
  if (k == 0) return from_hip(qblk::launch_zero_bytes(y, m * n * bytes_of_type(yt), s));
  QBLK_TRY(check_work(workspace, workspace_bytes, qblk::gemm_f8_workspace(m, k, n)));
  return from_hip(qblk::launch_gemm_f8(w, wscale, m, k, xq, xscale, n, y, yt, workspace, s));
}

size_t qblk_linear_f8_workspace(int64_t m, int64_t k, int64_t n) {
  if (!gemm_shape_ok(m, k, n) || m == 0 || k == 0 || n == 0) return 0;
  return static_cast<size_t>(qblk::linear_f8_workspace(m, k, n));
}

qblk_status_t qblk_linear_f8(const uint8_t* w, const float* wscale, int64_t m, int64_t k, const void* x,
                             qblk_dtype_t xt, int64_t n, void* y, qblk_dtype_t yt, void* workspace,
                             size_t workspace_bytes, qblk_stream_t stream) {
  if (!gemm_shape_ok(m, k, n)) return QBLK_ERR_SHAPE;
  if (!dtype_ok(xt) || !dtype_ok(yt)) return QBLK_ERR_DTYPE;
  const bool out = m > 0 && n > 0, work = out && k > 0;
  QBLK_TRY(check_ptr(w, work));
  QBLK_TRY(check_ptr4(wscale, work));
  QBLK_TRY(check_ptr(x, work));
  QBLK_TRY(check_ptr(y, out));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!out) return QBLK_OK;
  if (k == 0) return from_hip(qblk::launch_zero_bytes(y, m * n * bytes_of_type(yt), s));
  QBLK_TRY(check_work(workspace, workspace_bytes, qblk::linear_f8_workspace(m, k, n)));
  return from_hip(qblk::launch_linear_f8(w, wscale, m, k, x, xt, n, y, yt, workspace, s));
}

size_t qblk_ffn_f8_workspace(int64_t hidden, int64_t inter, int64_t n) {
  if (!ffn_shape_ok(hidden, inter, n) || hidden == 0 || inter == 0 || n == 0) return 0;
  return static_cast<size_t>(qblk::ffn_f8_workspace(hidden, inter, n));
}

qblk_status_t qblk_ffn_f8(const uint8_t* w13, const float* s13, const uint8_t* w2, const float* s2, int64_t hidden,
                          int64_t inter, const void* x, qblk_dtype_t xt, int64_t n, void* y, qblk_dtype_t yt,
                          void* workspace, size_t workspace_bytes, qblk_stream_t stream) {
  if (!ffn_shape_ok(hidden, inter, n)) return QBLK_ERR_SHAPE;
  if (!dtype_ok(xt) || !dtype_ok(yt)) return QBLK_ERR_DTYPE;
  const bool out = hidden > 0 && n > 0, work = out && inter > 0;
  QBLK_TRY(check_ptr(w13, work));
  QBLK_TRY(check_ptr4(s13, work));
  QBLK_TRY(check_ptr(w2, work));
  QBLK_TRY(check_ptr4(s2, work));
  QBLK_TRY(check_ptr(x, work));
  QBLK_TRY(check_ptr(y, out));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!out) return QBLK_OK;
  if (inter == 0) return from_hip(qblk::launch_zero_bytes(y, hidden * n * bytes_of_type(yt), s));
  QBLK_TRY(check_work(workspace, workspace_bytes, qblk::ffn_f8_workspace(hidden, inter, n)));
  return from_hip(qblk::launch_ffn_f8(w13, s13, w2, s2, hidden, inter, x, xt, n, y, yt, workspace, s));
}

size_t qblk_moe_workspace(const qblk_moe_t* a) {
  if (!a || moe_shape(*a) != QBLK_OK) return 0;
  return static_cast<size_t>(moe_work(*a));
}

qblk_status_t qblk_moe(const qblk_moe_t* a, qblk_stream_t stream) {
  if (!a) return QBLK_ERR_NULL;
  QBLK_TRY(moe_shape(*a));
  if (!dtype_ok(a->xt) || !dtype_ok(a->yt)) return QBLK_ERR_DTYPE;
  if (a->xt == QBLK_F32) return QBLK_ERR_UNSUPPORTED;  // the matrix cores take 16-bit activations
  const bool out = a->n > 0 && a->hidden > 0, work = out && a->inter > 0;
  QBLK_TRY(check_ptr(a->x, work));
  QBLK_TRY(check_ptr(a->gate_up, work));
  QBLK_TRY(check_ptr(a->down, work));
  if (a->logits) QBLK_TRY(check_ptr4(a->logits, true));
  QBLK_TRY(check_ptr4(a->ids, a->n > 0));
  QBLK_TRY(check_ptr4(a->weights, a->n > 0));
  QBLK_TRY(check_ptr(a->y, out));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!out) return QBLK_OK;
  if (!work) return from_hip(qblk::launch_zero_bytes(a->y, a->n * a->hidden * bytes_of_type(a->yt), s));
  QBLK_TRY(check_work(a->workspace, a->workspace_bytes, moe_work(*a)));
  qblk::MoeArgs k;
  k.x = a->x;
  k.logits = a->logits;
  k.gate_up = static_cast<const uint8_t*>(a->gate_up);
  k.down = static_cast<const uint8_t*>(a->down);
  k.ids = a->ids;
  k.weights = a->weights;
  k.y = a->y;
  k.table = a->workspace;
  k.h = static_cast<uint8_t*>(a->workspace) + qblk::moe_table_bytes();
  k.up_row_bytes = a->hidden / elems_of(a->fmt) * static_cast<int64_t>(bytes_of(a->fmt));
  k.down_row_bytes = a->inter / elems_of(a->fmt) * static_cast<int64_t>(bytes_of(a->fmt));
  k.wscale = a->weight_scale;
  k.n = 0;
  k.hidden = static_cast<int>(a->hidden);
  k.inter = static_cast<int>(a->inter);
  k.experts = a->experts;
  k.top_k = a->top_k;
  k.renorm = a->renorm != 0;
  k.xt = a->xt;
  k.yt = a->yt;
  return from_hip(qblk::launch_moe(a->fmt, k, a->n, s));
}

}  // extern "C"
