// The argument checks of the microscaling formats' and the norm's C ABI, built for
// the host alone under AddressSanitizer and UndefinedBehaviorSanitizer, with
// stand-ins for the launchers that record the call (see abi_sanitize_main.cpp).
#include "../bit_block_quant_amd/csrc/qblk_mx_abi.hip"

#include <stdio.h>

#include <string>

namespace {
std::string g_name;
int g_count = 0, g_fail = 0;
int64_t g_n = -1;
qblk::NormArgs g_norm;
hipError_t rec(const char* name, int64_t n) {
  g_name = name;
  g_n = n;
  g_count++;
  return hipSuccess;
}
}  // namespace

namespace qblk {
hipError_t launch_quantize_mx(const void*, int, int64_t rows, int64_t, bool f8, uint8_t*, uint8_t*, hipStream_t) {
  return rec(f8 ? "quantize8" : "quantize4", rows);
}
hipError_t launch_dequant_mx(const uint8_t*, const uint8_t*, int64_t rows, int64_t, bool f8, void*, int, hipStream_t) {
  return rec(f8 ? "dequant8" : "dequant4", rows);
}
int64_t gemm_mxfp4_workspace(int64_t, int64_t, int64_t n, bool) { return n > 64 ? 1024 : 0; }
hipError_t launch_gemm_mxfp4(const uint8_t*, const uint8_t*, int64_t, int64_t, const uint8_t*, const uint8_t*, bool f8,
                             int64_t n, void*, int, void*, hipStream_t) {
  return rec(f8 ? "gemm8" : "gemm4", n);
}
int64_t linear_mxfp4_workspace(int64_t, int64_t, int64_t n, bool) { return n > 1 ? 512 : 0; }
hipError_t launch_linear_mxfp4(const uint8_t*, const uint8_t*, int64_t, int64_t, const void*, int, bool f8, int64_t n,
                               void*, int, void*, hipStream_t) {
  return rec(f8 ? "linear8" : "linear4", n);
}
hipError_t launch_zero_bytes(void*, int64_t bytes, hipStream_t) { return rec("zero", bytes); }
hipError_t launch_rmsnorm(const NormArgs& a, int64_t n, hipStream_t) {
  g_norm = a;
  return rec("rmsnorm", n);
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
  uint8_t* const S = buf + 1025;  // scales of blocks: any byte
  float* const S4 = reinterpret_cast<float*>(buf + 1028);
  void* const B = buf + 2048;
  void* const Y = buf + 5120;
  void* const W = buf + 4096;
  void* const MIS = buf + 8;
  const int64_t kMax = (int64_t(1) << 31) - 1;
  const qblk_dtype_t bad = static_cast<qblk_dtype_t>(3);
  const qblk_act_t F4 = QBLK_ACT_MXFP4, F8 = QBLK_ACT_MXFP8;
  void* const s = nullptr;

  // quantizer and values
  REJECTS(qblk_quantize_mx(nullptr, QBLK_F32, 2, 32, F4, B, S, s), QBLK_ERR_NULL);
  REJECTS(qblk_quantize_mx(A, QBLK_F32, 2, 32, F4, nullptr, S, s), QBLK_ERR_NULL);
  REJECTS(qblk_quantize_mx(A, QBLK_F32, 2, 32, F4, B, nullptr, s), QBLK_ERR_NULL);
  REJECTS(qblk_quantize_mx(MIS, QBLK_F32, 2, 32, F4, B, S, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_quantize_mx(A, QBLK_F32, 2, 32, F4, MIS, S, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_quantize_mx(A, bad, 2, 32, F4, B, S, s), QBLK_ERR_DTYPE);
  REJECTS(qblk_quantize_mx(A, QBLK_F32, 2, 32, QBLK_ACT_F8, B, S, s), QBLK_ERR_FORMAT);
  REJECTS(qblk_quantize_mx(A, QBLK_F32, 2, 32, QBLK_ACT_I8, B, S, s), QBLK_ERR_FORMAT);
  REJECTS(qblk_quantize_mx(A, QBLK_F32, 2, 32, QBLK_ACT_NONE, B, S, s), QBLK_ERR_FORMAT);
  REJECTS(qblk_quantize_mx(A, QBLK_F32, 2, 33, F4, B, S, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_quantize_mx(A, QBLK_F32, -1, 32, F4, B, S, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_quantize_mx(A, QBLK_F32, 2, -32, F4, B, S, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_quantize_mx(A, QBLK_F32, kMax, kMax / 32 * 32, F4, B, S, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_quantize_mx(A, QBLK_F32, INT64_MAX, 32, F4, B, S, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_quantize_mx(nullptr, QBLK_F32, 0, 32, F4, nullptr, nullptr, s), QBLK_OK);
  REJECTS(qblk_quantize_mx(nullptr, QBLK_F32, 3, 0, F4, nullptr, nullptr, s), QBLK_OK);
  LAUNCHES(qblk_quantize_mx(A, QBLK_BF16, 3, 96, F4, B, S, s), "quantize4", 3);
  LAUNCHES(qblk_quantize_mx(A, QBLK_BF16, 4, 96, F8, B, S, s), "quantize8", 4);
  REJECTS(qblk_dequant_mx(nullptr, S, F4, 2, 32, Y, QBLK_F32, s), QBLK_ERR_NULL);
  REJECTS(qblk_dequant_mx(A, nullptr, F4, 2, 32, Y, QBLK_F32, s), QBLK_ERR_NULL);
  REJECTS(qblk_dequant_mx(A, S, F4, 2, 32, MIS, QBLK_F32, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_dequant_mx(MIS, S, F4, 2, 32, Y, QBLK_F32, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_dequant_mx(A, S, F4, 2, 32, Y, bad, s), QBLK_ERR_DTYPE);
  REJECTS(qblk_dequant_mx(A, S, QBLK_ACT_F8, 2, 128, Y, QBLK_F32, s), QBLK_ERR_FORMAT);
  REJECTS(qblk_dequant_mx(A, S, F4, 2, 16, Y, QBLK_F32, s), QBLK_ERR_SHAPE);
  LAUNCHES(qblk_dequant_mx(A, S, F8, 2, 32, Y, QBLK_F32, s), "dequant8", 2);

  // products
  REJECTS(qblk_gemm_mxfp4(A, S, 4, 100, B, S, F4, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_gemm_mxfp4(A, S, 4, 96, B, S, F4, -2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_gemm_mxfp4(A, S, (int64_t(1) << 26) + 1, 32, B, S, F4, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_gemm_mxfp4(A, S, 16, (int64_t(1) << 23) + 32, B, S, F4, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_gemm_mxfp4(A, S, int64_t(1) << 26, 32, B, S, F4, kMax, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_SHAPE);
  REJECTS(qblk_gemm_mxfp4(A, S, 4, 96, B, S, F4, 2, Y, bad, nullptr, 0, s), QBLK_ERR_DTYPE);
  REJECTS(qblk_gemm_mxfp4(A, S, 4, 96, B, S, QBLK_ACT_I8, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_FORMAT);
  REJECTS(qblk_gemm_mxfp4(nullptr, S, 4, 96, B, S, F4, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_NULL);
  REJECTS(qblk_gemm_mxfp4(A, nullptr, 4, 96, B, S, F4, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_NULL);
  REJECTS(qblk_gemm_mxfp4(A, S, 4, 96, nullptr, S, F4, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_NULL);
  REJECTS(qblk_gemm_mxfp4(A, S, 4, 96, B, nullptr, F4, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_NULL);
  REJECTS(qblk_gemm_mxfp4(A, S, 4, 96, B, S, F4, 2, MIS, QBLK_F32, nullptr, 0, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_gemm_mxfp4(buf + 1, S, 4, 96, B, S, F4, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_gemm_mxfp4(A, S, 4, 96, B, S, F4, 65, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_NULL);
  REJECTS(qblk_gemm_mxfp4(A, S, 4, 96, B, S, F4, 65, Y, QBLK_F32, MIS, 1024, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_gemm_mxfp4(A, S, 4, 96, B, S, F4, 65, Y, QBLK_F32, W, 1023, s), QBLK_ERR_WORKSPACE);
  REJECTS(qblk_gemm_mxfp4(nullptr, nullptr, 4, 96, nullptr, nullptr, F4, 0, nullptr, QBLK_F32, nullptr, 0, s), QBLK_OK);
  LAUNCHES(qblk_gemm_mxfp4(nullptr, nullptr, 4, 0, nullptr, nullptr, F4, 3, Y, QBLK_BF16, nullptr, 0, s), "zero", 24);
  LAUNCHES(qblk_gemm_mxfp4(A, S, 4, 96, B, S, F8, 2, Y, QBLK_F16, nullptr, 0, s), "gemm8", 2);
  LAUNCHES(qblk_gemm_mxfp4(A, S, 4, 96, B, S, F4, 65, Y, QBLK_F16, W, 1024, s), "gemm4", 65);
  EXPECT(qblk_gemm_mxfp4_workspace(4, 100, 2, F4) == 0 && qblk_gemm_mxfp4_workspace(INT64_MIN, 96, 2, F4) == 0);
  EXPECT(qblk_gemm_mxfp4_workspace(4, 96, 65, QBLK_ACT_F8) == 0 && qblk_gemm_mxfp4_workspace(4, 96, 65, F8) == 1024);
  REJECTS(qblk_linear_mxfp4(A, S, 4, 96, B, bad, F4, 1, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_DTYPE);
  REJECTS(qblk_linear_mxfp4(A, S, 4, 96, B, QBLK_F16, QBLK_ACT_F8, 1, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_FORMAT);
  REJECTS(qblk_linear_mxfp4(A, S, 4, 96, MIS, QBLK_F16, F4, 1, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_ALIGN);
  REJECTS(qblk_linear_mxfp4(A, S, 4, 96, B, QBLK_F16, F4, 2, Y, QBLK_F32, nullptr, 0, s), QBLK_ERR_NULL);
  REJECTS(qblk_linear_mxfp4(A, S, 4, 96, B, QBLK_F16, F4, 2, Y, QBLK_F32, W, 511, s), QBLK_ERR_WORKSPACE);
  LAUNCHES(qblk_linear_mxfp4(A, S, 4, 96, B, QBLK_F16, F4, 2, Y, QBLK_F32, W, 512, s), "linear4", 2);
  LAUNCHES(qblk_linear_mxfp4(A, S, 4, 96, B, QBLK_F16, F8, 1, Y, QBLK_F32, nullptr, 0, s), "linear8", 1);
  EXPECT(qblk_linear_mxfp4_workspace(4, 96, 2, F4) == 512 && qblk_linear_mxfp4_workspace(4, 96, 0, F4) == 0);

  // norm
  qblk_rmsnorm_t m = {};
  m.n = 3;
  m.hidden = 256;
  m.x = A;
  m.residual = B;
  m.xt = QBLK_BF16;
  m.weight = Y;
  m.wt = QBLK_F32;
  m.eps = 1e-6f;
  m.act = QBLK_ACT_F8;
  m.codes = W;
  m.scale = S4;
  m.total = A;
  LAUNCHES(qblk_rmsnorm(&m, s), "rmsnorm", 3);
  EXPECT(g_norm.total == A && g_norm.hidden == 256 && g_norm.y == nullptr && g_norm.act == QBLK_ACT_F8);
  REJECTS(qblk_rmsnorm(nullptr, s), QBLK_ERR_NULL);
#define WITH(field, value, st)        \
  do {                                \
    qblk_rmsnorm_t c = m;             \
    c.field = value;                  \
    REJECTS(qblk_rmsnorm(&c, s), st); \
  } while (0)
  WITH(n, -1, QBLK_ERR_SHAPE);
  WITH(n, kMax + 1, QBLK_ERR_SHAPE);
  WITH(hidden, 64, QBLK_ERR_SHAPE);
  WITH(hidden, -128, QBLK_ERR_SHAPE);
  WITH(hidden, (int64_t(1) << 24) + 128, QBLK_ERR_SHAPE);
  WITH(n, kMax, QBLK_ERR_SHAPE);  // 2^31 rows of 256 fp32 values pass 2^40 bytes
  WITH(act, -2, QBLK_ERR_FORMAT);
  WITH(act, 4, QBLK_ERR_FORMAT);
  WITH(act, QBLK_ACT_NONE, QBLK_ERR_NULL);  // no y
  WITH(xt, 3, QBLK_ERR_DTYPE);
  WITH(wt, -1, QBLK_ERR_DTYPE);
  WITH(eps, -1.0f, QBLK_ERR_SHAPE);
  WITH(eps, __builtin_nanf(""), QBLK_ERR_SHAPE);
  WITH(x, nullptr, QBLK_ERR_NULL);
  WITH(x, MIS, QBLK_ERR_ALIGN);
  WITH(residual, MIS, QBLK_ERR_ALIGN);
  WITH(weight, nullptr, QBLK_ERR_NULL);
  WITH(weight, MIS, QBLK_ERR_ALIGN);
  WITH(total, nullptr, QBLK_ERR_NULL);
  WITH(codes, nullptr, QBLK_ERR_NULL);
  WITH(codes, MIS, QBLK_ERR_ALIGN);
  WITH(scale, nullptr, QBLK_ERR_NULL);
  WITH(scale, S, QBLK_ERR_ALIGN);
  WITH(y, MIS, QBLK_ERR_ALIGN);
  WITH(n, 0, QBLK_OK);
  WITH(hidden, 0, QBLK_OK);
  {
    qblk_rmsnorm_t c = m;
    c.act = QBLK_ACT_MXFP4;
    c.hidden = 96;
    c.scale = S;  // bytes at any address
    c.residual = nullptr;
    c.total = MIS;  // not looked at
    LAUNCHES(qblk_rmsnorm(&c, s), "rmsnorm", 3);
    EXPECT(g_norm.total == nullptr);
    c.hidden = 48;
    REJECTS(qblk_rmsnorm(&c, s), QBLK_ERR_SHAPE);
    c.act = QBLK_ACT_NONE;
    c.y = Y;
    c.codes = c.scale = nullptr;
    LAUNCHES(qblk_rmsnorm(&c, s), "rmsnorm", 3);
    c.act = QBLK_ACT_I8;
    c.codes = W;
    c.scale = S4;
    LAUNCHES(qblk_rmsnorm(&c, s), "rmsnorm", 3);
    c.hidden = 52;
    REJECTS(qblk_rmsnorm(&c, s), QBLK_ERR_SHAPE);
    c.hidden = 0;  // rows without columns have a scale each
    LAUNCHES(qblk_rmsnorm(&c, s), "zero", 12);
    c.scale = nullptr;
    REJECTS(qblk_rmsnorm(&c, s), QBLK_ERR_NULL);
  }
  if (g_fail == 0) printf("clean\n");
  return g_fail != 0;
}
