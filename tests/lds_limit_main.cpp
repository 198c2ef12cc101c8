// The dynamic-LDS limit of a kernel (qblk_lds.h) with stand-ins for the runtime: set once on
// every device, and again where it failed.
#include "../bit_block_quant_amd/csrc/qblk_lds.h"

#include <stdio.h>

static int g_dev = 0, g_calls[80], g_fail = 0;
static hipError_t g_next = hipSuccess;

extern "C" hipError_t hipGetDevice(int* dev) {
  *dev = g_dev;
  return hipSuccess;
}
extern "C" hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) {
  g_calls[g_dev]++;
  return g_next;
}

#define EXPECT(cond)                                                         \
  do {                                                                       \
    if (!(cond)) {                                                           \
      fprintf(stderr, "line %d: check failed: %s\n", __LINE__, #cond); \
      g_fail++;                                                              \
    }                                                                        \
  } while (0)

int main() {
  static std::atomic<uint64_t> done{0}, other{0};
  for (int round = 0; round < 3; round++)
    for (g_dev = 0; g_dev < 64; g_dev++) EXPECT(qblk::allow_lds(done, "kernel", 1 << 17) == hipSuccess);
  for (int d = 0; d < 64; d++) EXPECT(g_calls[d] == 1);
  g_dev = 70;  // past what is remembered: asked for each time
  for (int round = 0; round < 2; round++) EXPECT(qblk::allow_lds(done, "kernel", 1 << 17) == hipSuccess);
  EXPECT(g_calls[70] == 2);
  g_dev = 1;  // another kernel's own limit; a failure is reported and not kept
  g_next = hipErrorInvalidValue;
  EXPECT(qblk::allow_lds(other, "other", 1) == hipErrorInvalidValue && g_calls[1] == 2);
  g_next = hipSuccess;
  EXPECT(qblk::allow_lds(other, "other", 1) == hipSuccess && g_calls[1] == 3);
  EXPECT(qblk::allow_lds(other, "other", 1) == hipSuccess && g_calls[1] == 3);
  printf("%s\n", g_fail ? "failed" : "clean");
  return g_fail != 0;
}
