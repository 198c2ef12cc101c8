// The argument checks of the feed-forward operators' C ABI, built for the host
// alone under AddressSanitizer and UndefinedBehaviorSanitizer, with stand-ins
// for the launchers that record the call (see abi_sanitize_main.cpp).
#include "../bit_block_quant_amd/csrc/qblk_ffn_abi.hip"

#include <stdio.h>

#include <string>

namespace {
std::string g_name;
int g_count = 0, g_fail = 0;
int64_t g_n = -1;
qblk::MoeArgs g_moe;
hipError_t rec(const char* name, int64_t n) {
  g_name = name;
  g_n = n;
  g_count++;
  return hipSuccess;
}
}  // namespace

namespace qblk {
hipError_t launch_quantize_f8(const void*, int, int64_t rows, int64_t, uint8_t*, float*, hipStream_t) {
  return rec("quantize_f8", rows);
}
hipError_t launch_quantize_act_f8(const void*, int, int64_t n, int64_t, uint8_t*, float*, hipStream_t) {
  return rec("quantize_act_f8", n);
}
int64_t gemm_f8_workspace(int64_t, int64_t, int64_t) { return 0; }
hipError_t launch_gemm_f8(const uint8_t*, const float*, int64_t, int64_t, const uint8_t*, const float*, int64_t n,
                          void*, int, void*, hipStream_t) {
  return rec("gemm_f8", n);
}
int64_t linear_f8_workspace(int64_t, int64_t, int64_t n) { return n > 1 ? 512 : 0; }
hipError_t launch_linear_f8(const uint8_t*, const float*, int64_t, int64_t, const void*, int, int64_t n, void*, int,
                            void*, hipStream_t) {
  return rec("linear_f8", n);
}
int64_t ffn_f8_workspace(int64_t, int64_t, int64_t) { return 512; }
hipError_t launch_ffn_f8(const uint8_t*, const float*, const uint8_t*, const float*, int64_t, int64_t, const void*,
                         int, int64_t n, void*, int, void*, hipStream_t) {
  return rec("ffn_f8", n);
}
hipError_t launch_zero_bytes(void*, int64_t bytes, hipStream_t) { return rec("zero", bytes); }
int64_t moe_table_bytes() { return 1024; }
hipError_t launch_moe(int, const MoeArgs& a, int64_t n, hipStream_t) {
  g_moe = a;
  return rec("moe", n);
}
}  // namespace qblk

#define EXPECT(cond)                                                           \
  do {                                                                         \
    if (!(cond)) {                                                             \
      fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      g_fail++;                                                                \
    }                                                                          \
  } while (0)
#define REJECTS(expr, st)            \
  do {                               \
    const int before_ = g_count;     \
    EXPECT((expr) == (st));          \
    EXPECT(g_count == before_);      \
  } while (0)
#define LAUNCHES(expr, nm, n)        \
  do {                               \
    const int before_ = g_count;     \
    EXPECT((expr) == QBLK_OK);       \
    EXPECT(g_count == before_ + 1);  \
    EXPECT(g_name == (nm));          \
    EXPECT(g_n == (n));              \
  } while (0)

int main() {
  alignas(64) static unsigned char buf[8192];
  uint8_t* const A = buf;
  float* const S = reinterpret_cast<float*>(buf + 1028);  // scales: 4-byte aligned only
  void* const B = buf + 2048;
  void* const Y = buf + 3072;
  void* const W = buf + 4096;
  void* const MIS = buf + 8;
  float* const MIS4 = reinterpret_cast<float*>(buf + 1030);
  const int64_t kMax = (int64_t(1) << 31) - 1;
  const qblk_dtype_t bad = static_cast<qblk_dtype_t>(3);
  void* const s = nullptr;
  uint8_t* const C = buf + 5120;

  // quantizers
  REJECTS(qblk_quantize_f8(nullptr, QBLK_F32, 2, 128, C, S, s), QBLK_ERR_NULL);
  REJECTS(qblk_quantize_f8(A, QBLK_F32, 2, 128, nullptr, S, s), QBLK_ERR_NULL);
  REJECTS(qblk_quantize_f8(A, QBLK_F32, 2, 128, C, nullptr, s), QBLK_ERR_NULL);
  REJECTS(qblk_quantize_f8(MIS, QBLK_F32, 2, 128, C, S, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_quantize_f8(A, QBLK_F32, 2, 128, C, MIS4, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_quantize_f8(A, bad, 2, 128, C, S, s), QBLK_ERR_DTYPE);
  REJECTS(qblk_quantize_f8(A, QBLK_F32, 2, 127, C, S, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_quantize_f8(A, QBLK_F32, -1, 128, C, S, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_quantize_f8(A, QBLK_F32, kMax, kMax / 128 * 128, C, S, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_quantize_f8(A, QBLK_F32, INT64_MAX, 128, C, S, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_quantize_f8(nullptr, QBLK_F32, 0, 128, nullptr, nullptr, s), QBLK_OK);
  LAUNCHES(qblk_quantize_f8(A, QBLK_BF16, 3, 256, C, S, s), "quantize_f8", 3);
  REJECTS(qblk_quantize_act_f8(A, QBLK_F16, 2, 64, C, S, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_quantize_act_f8(A, QBLK_F16, 2, -128, C, S, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_quantize_act_f8(nullptr, QBLK_F16, 5, 0, nullptr, nullptr, s), QBLK_OK);
  LAUNCHES(qblk_quantize_act_f8(A, QBLK_F16, 2, 128, C, S, s), "quantize_act_f8", 2);

  // products
  REJECTS(qblk_gemm_f8(A, S, 4, 100, C, S, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_gemm_f8(A, S, 4, 128, C, S, -2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_gemm_f8(A, S, (int64_t(1) << 26) + 1, 128, C, S, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_gemm_f8(A, S, 16, (int64_t(1) << 24) + 128, C, S, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_gemm_f8(A, S, int64_t(1) << 26, 128, C, S, kMax, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_gemm_f8(A, S, 4, 128, C, S, 2, Y, bad, nullptr, 0, s), QBLK_ERR_DTYPE);
  REJECTS(qblk_gemm_f8(nullptr, S, 4, 128, C, S, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_NULL);
  REJECTS(qblk_gemm_f8(A, nullptr, 4, 128, C, S, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_NULL);
  REJECTS(qblk_gemm_f8(A, S, 4, 128, nullptr, S, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_NULL);
  REJECTS(qblk_gemm_f8(A, S, 4, 128, C, S, 2, MIS, QBLK_F32, nullptr, 0, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_gemm_f8(A, S, 4, 128, buf + 1, S, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_gemm_f8(nullptr, nullptr, 4, 128, nullptr, nullptr, 0, nullptr, QBLK_F32, nullptr, 0, s), QBLK_OK);
  LAUNCHES(qblk_gemm_f8(nullptr, nullptr, 4, 0, nullptr, nullptr, 3, Y, QBLK_BF16, nullptr, 0, s), "zero", 24);
  LAUNCHES(qblk_gemm_f8(A, S, 4, 128, C, S, 2, Y, QBLK_F16, nullptr, 0, s), "gemm_f8", 2);
  EXPECT(qblk_gemm_f8_workspace(4, 100, 2) == 0 && qblk_gemm_f8_workspace(INT64_MIN, 128, 2) == 0);

  REJECTS(qblk_linear_f8(A, S, 4, 128, B, bad, 1, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_DTYPE);
  REJECTS(qblk_linear_f8(A, S, 4, 128, MIS, QBLK_F16, 1, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_linear_f8(A, S, 4, 128, B, QBLK_F16, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_NULL);
  REJECTS(qblk_linear_f8(A, S, 4, 128, B, QBLK_F16, 2, Y, QBLK_F32, MIS, 512, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_linear_f8(A, S, 4, 128, B, QBLK_F16, 2, Y, QBLK_F32, W, 511, s), QBLK_ERR_WORKSPACE);
  LAUNCHES(qblk_linear_f8(A, S, 4, 128, B, QBLK_F16, 2, Y, QBLK_F32, W, 512, s), "linear_f8", 2);
  LAUNCHES(qblk_linear_f8(A, S, 4, 128, B, QBLK_F16, 1, Y, QBLK_F32, nullptr, 0, s), "linear_f8", 1);
  EXPECT(qblk_linear_f8_workspace(4, 128, 2) == 512 && qblk_linear_f8_workspace(4, 128, 0) == 0);

  REJECTS(qblk_ffn_f8(A, S, A, S, 128, 100, B, QBLK_F16, 1, Y, QBLK_F16, W, 512, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_ffn_f8(A, S, A, S, 100, 128, B, QBLK_F16, 1, Y, QBLK_F16, W, 512, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_ffn_f8(A, S, A, S, 128, INT64_MAX / 128 * 128, B, QBLK_F16, 1, Y, QBLK_F16, W, 512, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_ffn_f8(A, S, nullptr, S, 128, 128, B, QBLK_F16, 1, Y, QBLK_F16, W, 512, s), QBLK_ERR_NULL);
  REJECTS(qblk_ffn_f8(A, S, A, S, 128, 128, B, QBLK_F16, 1, Y, QBLK_F16, W, 500, s), QBLK_ERR_WORKSPACE);
  REJECTS(qblk_ffn_f8(A, S, A, S, 128, 128, B, QBLK_F16, 1, nullptr, QBLK_F16, W, 512, s), QBLK_ERR_NULL);
  LAUNCHES(qblk_ffn_f8(A, S, A, S, 128, 128, B, QBLK_F16, 1, Y, QBLK_F16, W, 512, s), "ffn_f8", 1);
  LAUNCHES(qblk_ffn_f8(nullptr, nullptr, nullptr, nullptr, 128, 0, nullptr, QBLK_F16, 2, Y, QBLK_F16, nullptr, 0, s), "zero", 512);

  // mixture of experts
  qblk_moe_t m = {};
  m.fmt = QBLK_SB4;
  m.n = 3;
  m.hidden = 256;
  m.inter = 512;
  m.experts = 4;
  m.top_k = 2;
  m.x = B;
  m.xt = QBLK_F16;
  m.logits = S;
  m.renorm = 5;
  m.weight_scale = 2.5f;
  m.gate_up = A;
  m.down = A;
  m.ids = reinterpret_cast<int32_t*>(S);
  m.weights = S;
  m.y = Y;
  m.yt = QBLK_F32;
  m.workspace = W;
  m.workspace_bytes = qblk_moe_workspace(&m);
  EXPECT(m.workspace_bytes == 1024 + 6 * 512 * 4);
  LAUNCHES(qblk_moe(&m, s), "moe", 3);
  EXPECT(g_moe.renorm == 1 && g_moe.wscale == 2.5f && g_moe.up_row_bytes == 138 && g_moe.down_row_bytes == 276);
  EXPECT(static_cast<uint8_t*>(g_moe.h) == static_cast<uint8_t*>(W) + 1024);
  REJECTS(qblk_moe(nullptr, s), QBLK_ERR_NULL);
  EXPECT(qblk_moe_workspace(nullptr) == 0);
#define WITH(field, value, st)    \
  do {                            \
    qblk_moe_t c = m;             \
    c.field = value;              \
    REJECTS(qblk_moe(&c, s), st); \
  } while (0)
  WITH(fmt, 9, QBLK_ERR_FORMAT);
  WITH(fmt, -1, QBLK_ERR_FORMAT);
  WITH(fmt, QBLK_W4G128, QBLK_ERR_UNSUPPORTED);
  WITH(n, -1, QBLK_ERR_SHAPE);
  WITH(n, kMax + 1, QBLK_ERR_SHAPE);
  WITH(hidden, 255, QBLK_ERR_SHAPE);
  WITH(hidden, INT64_MAX / 256 * 256, QBLK_ERR_SHAPE);
  WITH(inter, -256, QBLK_ERR_SHAPE);
  WITH(inter, int64_t(1) << 40, QBLK_ERR_SHAPE);
  WITH(inter, (int64_t(1) << 19) + 256, QBLK_ERR_SHAPE);
  WITH(hidden, (int64_t(1) << 19) + 256, QBLK_ERR_SHAPE);
  WITH(experts, 0, QBLK_ERR_SHAPE);
  WITH(experts, 513, QBLK_ERR_SHAPE);
  WITH(top_k, 0, QBLK_ERR_SHAPE);
  WITH(top_k, 5, QBLK_ERR_SHAPE);
  WITH(top_k, 33, QBLK_ERR_SHAPE);
  WITH(xt, 3, QBLK_ERR_DTYPE);
  WITH(yt, -1, QBLK_ERR_DTYPE);
  WITH(xt, QBLK_F32, QBLK_ERR_UNSUPPORTED);
  WITH(x, nullptr, QBLK_ERR_NULL);
  WITH(x, MIS, QBLK_ERR_ALIGN);
  WITH(gate_up, nullptr, QBLK_ERR_NULL);
  WITH(down, MIS, QBLK_ERR_ALIGN);
  WITH(ids, nullptr, QBLK_ERR_NULL);
  WITH(weights, MIS4, QBLK_ERR_ALIGN);
  WITH(logits, MIS4, QBLK_ERR_ALIGN);
  WITH(y, nullptr, QBLK_ERR_NULL);
  WITH(workspace, nullptr, QBLK_ERR_NULL);
  WITH(workspace, MIS, QBLK_ERR_ALIGN);
  WITH(workspace_bytes, m.workspace_bytes - 1, QBLK_ERR_WORKSPACE);
  WITH(n, 0, QBLK_OK);
  WITH(hidden, 0, QBLK_OK);
  {
    qblk_moe_t c = m;
    c.inter = 0;
    c.workspace = nullptr;
    LAUNCHES(qblk_moe(&c, s), "zero", 3 * 256 * 4);
    c = m;
    c.logits = nullptr;  // ids and weights given
    LAUNCHES(qblk_moe(&c, s), "moe", 3);
    EXPECT(g_moe.logits == nullptr);
    c.n = 5000;  // more tokens than one piece: the workspace stops growing
    EXPECT(qblk_moe_workspace(&c) == 1024 + 1024 * 512 * 4);
  }
  if (g_fail == 0) printf("clean\n");
  return g_fail != 0;
}
