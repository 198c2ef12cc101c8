// qblk_moe.h -- the mixture-of-experts layer's launcher (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qblk {

constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopK = 32;
// Pairs of a token and an expert that one pair of launches takes: their
// partial rows fit the 64 KB of LDS that k_moe_down uses.  More tokens run in
// pieces, in stream order.
constexpr int kMoeMaxPairs = 1024;
// Largest hidden and inter: the intermediate of those pairs is at most 2 GB,
// which k_moe_down addresses by 32-bit offsets.
constexpr int64_t kMoeMaxDim = int64_t(1) << 19;

struct MoeArgs {
  const void* x;
  const float* logits;  // nullptr: ids and weights are given
  const uint8_t* gate_up;
  const uint8_t* down;
  int32_t* ids;
  float* weights;
  void* y;
  void* table;  // workspace
  void* h;      // workspace: pairs of one piece x inter, 4 bytes each
  int64_t up_row_bytes, down_row_bytes;
  float wscale;
  int n, hidden, inter, experts, top_k, renorm, xt, yt;
};

int64_t moe_table_bytes();
// n tokens; a.n, and the pointers of later pieces, are set by the launcher
hipError_t launch_moe(int fmt, const MoeArgs& a, int64_t n, hipStream_t s);

}  // namespace qblk
