// qblk_mx_device.h -- device code of the OCP microscaling (MX) formats: 32
// neighbouring values of a row under one scale 2^e, kept as the byte e + 127
// (e8m0; 255: the whole block is NaN), the elements as e2m1 (MXFP4, two to a
// byte) or e4m3 (MXFP8).
//
//   e = floor(log2 max|v|) - 2 (e2m1: largest 6 = 1.5 * 2^2) or - 8 (e4m3: 448),
//   at least -127; element = v / 2^e to nearest even, at most the largest
//
// The quotients are exact: 2^-e is an fp32 number (at most 2^127), and what it
// makes underflow is far below half of the smallest element.
#pragma once

#include "qblk_quant_device.h"

namespace qblk {
namespace {

constexpr int kMxBlock = 32;
constexpr float kF4Max = 6.0f;

// the largest of 4 neighbouring lanes, in each of them (as bits: a NaN is above infinity)
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xF, 0xF, true));
  v = v > o ? v : o;
  o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xF, 0xF, true));
  return v > o ? v : o;
}

template <int N>
__device__ __forceinline__ uint32_t top_bits(const float v[N]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < N; i++) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
    a = a > b ? a : b;
  }
  return a;
}

// The scale's byte from the bits of the largest magnitude.
template <bool F8>
__device__ __forceinline__ uint32_t mx_scale(uint32_t top) {
  const uint32_t e = top >> 23, low = F8 ? 8u : 2u;
  return e == 255u ? 255u : (e > low ? e - low : 0u);
}

// The codes of N values (a multiple of 8) under the scale byte b: four bits each, or a byte.
template <bool F8, int N>
__device__ __forceinline__ void mx_codes(const float v[N], uint32_t b, uint32_t* out) {
  const float r = __builtin_bit_cast(float, (254u - (b < 254u ? b : 253u)) << 23);  // 2^-e
  float q[N];
#pragma unroll
  for (int i = 0; i < N; i++) q[i] = b == 255u ? 0.0f : __builtin_amdgcn_fmed3f(v[i] * r, F8 ? -kF8Max : -kF4Max, F8 ? kF8Max : kF4Max);
  if constexpr (F8) {
#pragma unroll
    for (int i = 0; i < N / 4; i++) {
      const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
      out[i] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], w, true));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 8; i++) {
      uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, q[8 * i], q[8 * i + 1], 1.0f, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[8 * i + 2], q[8 * i + 3], 1.0f, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[8 * i + 4], q[8 * i + 5], 1.0f, 2);
      out[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[8 * i + 6], q[8 * i + 7], 1.0f, 3);
    }
  }
}

// 8 elements with their scale as bf16
__device__ __forceinline__ bf16x8_n wide4(uint32_t c, float s) {
  const bf16x2_n p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0);
  const bf16x2_n p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1);
  const bf16x2_n p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2);
  const bf16x2_n p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3);
  return bf16x8_n{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}
__device__ __forceinline__ bf16x8_n wide8(uint32_t a, uint32_t b, float s) {
  const bf16x2_n p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, false);
  const bf16x2_n p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, true);
  const bf16x2_n p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, false);
  const bf16x2_n p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, true);
  return bf16x8_n{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

// Four values in 16 bits each, rounded to nearest even by the conversions (v_cvt_pk_bf16_f32
// for bf16: one operation for two values).
template <int YT>
__device__ __forceinline__ u32x2 pack16(const float4_t& v) {
  if constexpr (YT == QBLK_F16) {
    const half2_t a = {static_cast<half_t>(v.x), static_cast<half_t>(v.y)}, b = {static_cast<half_t>(v.z), static_cast<half_t>(v.w)};
    return u32x2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
  } else {
    const bf16x2_n a = {static_cast<__bf16>(v.x), static_cast<__bf16>(v.y)}, b = {static_cast<__bf16>(v.z), static_cast<__bf16>(v.w)};
    return u32x2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
  }
}

// The value of a scale's byte.
__device__ __forceinline__ float mx_scale_value(uint32_t b) {
  return b == 255u ? __builtin_nanf("") : b == 0u ? 0x1p-127f : __builtin_bit_cast(float, b << 23);
}

}  // namespace
}  // namespace qblk
