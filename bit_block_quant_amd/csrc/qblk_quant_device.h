// qblk_quant_device.h -- device code shared by the kernels that make 8-bit
// activations and by the products of them: loads of 8 values, maxima that keep a
// NaN, e4m3 codes of a group of 128, and the results' types.
#pragma once

#include "qblk_device.h"
#include "qblk_launch.h"

namespace qblk {
namespace {

typedef __bf16 bf16x2_n __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_n __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kGroup = 128;
constexpr float kF8Max = 448.0f;

// -------------------------------------------------------------- inputs
// 8 consecutive elements (16-byte aligned for the 16-bit types, 32 for fp32's two halves)
template <int XT>
__device__ __forceinline__ void load8(const void* x, int64_t at, float v[8]) {
  if constexpr (XT == QBLK_F32) {
    const float4_t* p = reinterpret_cast<const float4_t*>(static_cast<const float*>(x) + at);
    const float4_t a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + at);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (XT == QBLK_F16) {
        v[2 * i] = f16_bits_to_f32(a[i] & 0xffffu);
        v[2 * i + 1] = f16_bits_to_f32(a[i] >> 16);
      } else {
        v[2 * i] = bf16_bits_to_f32(a[i] & 0xffffu);
        v[2 * i + 1] = __builtin_bit_cast(float, a[i] & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + __builtin_expf(-g)) * u; }

// The larger, NaN if one is: a NaN among 128 values makes their scale NaN and so
// every result that they enter, where a maximum of numbers would pass over it.
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// max over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ float row16_max(float v) {
  v = max_nan(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, true)));
  v = max_nan(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, true)));
  v = max_nan(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xF, 0xF, true)));
  v = max_nan(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xF, 0xF, true)));
  return v;
}

// The e4m3 codes of N values (a multiple of 4) against one scale: the IEEE
// quotient v/s, clamped, rounded to nearest even by the conversion.  The
// quotients are formed from the correctly rounded reciprocal with two
// residual corrections (Markstein 1990: q' = q + (v - q s) r is the correctly
// rounded quotient when r is the rounded reciprocal and q is within an ulp;
// the first correction brings q there).  That needs the residuals to stay
// clear of under- and overflow, so a wave that holds a scale outside 2^+-60
// divides instead.
template <int N>
__device__ __forceinline__ void codes_f8(const float v[N], float s, uint32_t out[N / 4]) {
  float q[N];
  if (__builtin_amdgcn_ballot_w64(s != 0.0f && !(s >= 0x1p-60f && s <= 0x1p60f)) == 0) {
    const float d = s == 0.0f ? 1.0f : s;
    const float r = 1.0f / d;
#pragma unroll
    for (int i = 0; i < N; i++) {
      const float x = s == 0.0f ? 0.0f : v[i];
      float t = x * r;
      t = __builtin_fmaf(__builtin_fmaf(-t, d, x), r, t);
      q[i] = __builtin_fmaf(__builtin_fmaf(-t, d, x), r, t);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i++) q[i] = qdiv(v[i], s);
  }
#pragma unroll
  for (int i = 0; i < N; i++) q[i] = __builtin_elementwise_minimum(max_nan(q[i], -kF8Max), kF8Max);
#pragma unroll
  for (int i = 0; i < N / 4; i++) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
    out[i] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], w, true));
  }
}

// One group of 128 by the 16 lanes of a DPP row, 8 values each: the scale and
// this lane's 8 codes.
__device__ __forceinline__ float quant_group(const float v[8], uint32_t code[2]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) a = max_nan(a, __builtin_fabsf(v[i]));
  const float s = row16_max(a) / kF8Max;
  codes_f8<8>(v, s, code);
  return s;
}

// ------------------------------------------------------------ results
__device__ __forceinline__ u32x2 bits16(const float4_t& v, int yt) {
  uint32_t h[4];
#pragma unroll
  for (int e = 0; e < 4; e++) h[e] = yt == QBLK_F16 ? f32_to_f16_bits(v[e]) : f32_to_bf16_bits(v[e]);
  return u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
}

// (stores take any address: with a ragged number of rows the tokens' rows of y
// start at every value.  4096 x 5003 x 4096: 96 us, as for 5120 rows; with the
// values of an odd row count stored one by one a fifth more.)
typedef float float4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));

// floats from one token's partial sums to the next one's
__host__ __device__ __forceinline__ int64_t part_pitch(int64_t m) { return (m + 3) & ~int64_t(3); }

__device__ __forceinline__ void store_y(void* y, int64_t at, float v, int yt) {
  if (yt == QBLK_F32)
    static_cast<float*>(y)[at] = v;
  else
    static_cast<uint16_t*>(y)[at] = yt == QBLK_F16 ? f32_to_f16_bits(v) : f32_to_bf16_bits(v);
}

}  // namespace
}  // namespace qblk
