// qblk_norm.hip -- root-mean-square norm of the residual stream with the codes
// that the next product reads, on gfx950.
//
//   t = x + residual, rounded to x's type (what the next layer adds to)
//   y = t * (1 / sqrt(mean(t^2) + eps)) * weight            in fp32
//   codes and scales of y: e4m3 with an fp32 scale per 128 columns, int8 with one
//   per row, or MXFP8 / MXFP4, each by the rule of its own quantizer
//
// The codes are made from the fp32 y: rounding it to 16 bits first would move them.
#include "qblk_mx_device.h"
#include "qblk_norm.h"

namespace qblk {
namespace {

__device__ __forceinline__ void load_weight(const void* w, int wt, int64_t at, float v[8]) {
  if (wt == QBLK_F32)
    load8<QBLK_F32>(w, at, v);
  else if (wt == QBLK_F16)
    load8<QBLK_F16>(w, at, v);
  else
    load8<QBLK_BF16>(w, at, v);
}

// v rounded to the type, and stored there if `to` is given
template <int XT>
__device__ __forceinline__ void round_store(float v[8], void* to, int64_t at) {
  if constexpr (XT == QBLK_F32) {
    if (!to) return;
    float4_t* o = reinterpret_cast<float4_t*>(static_cast<float*>(to) + at);
    o[0] = float4_t{v[0], v[1], v[2], v[3]};
    o[1] = float4_t{v[4], v[5], v[6], v[7]};
  } else {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t a = XT == QBLK_F16 ? f32_to_f16_bits(v[2 * i]) : f32_to_bf16_bits(v[2 * i]);
      const uint32_t b = XT == QBLK_F16 ? f32_to_f16_bits(v[2 * i + 1]) : f32_to_bf16_bits(v[2 * i + 1]);
      h[i] = a | (b << 16);
      v[2 * i] = XT == QBLK_F16 ? f16_bits_to_f32(a) : bf16_bits_to_f32(a);
      v[2 * i + 1] = XT == QBLK_F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
    }
    if (to) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(to) + at) = u32x4{h[0], h[1], h[2], h[3]};
  }
}

// The sum (or, MAX, the largest) over `waves` waves' lanes, in every lane; `part`
// holds a float for each wave and is free again afterwards.
template <bool MAX>
__device__ __forceinline__ float row_total(float v, float* part, int waves, int wave) {
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    const float o = __shfl_xor(v, m, kWave);
    v = MAX ? max_nan(v, o) : v + o;
  }
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[wave] = v;
  __syncthreads();
  v = part[0];
  for (int i = 1; i < waves; i++) v = MAX ? max_nan(v, part[i]) : v + part[i];
  __syncthreads();
  return v;
}

// One row by TH threads, V units of 8 values each (unit t, t + TH, ...); rows
// of one wave: four to a workgroup.  Rows wider than 8 TH V values (LOOP) are read a
// second time for the output.
template <int XT, int TH, int V, bool LOOP>
__global__ __launch_bounds__(TH < 256 ? 256 : TH) void k_rmsnorm(NormArgs p) {
  __shared__ float part[TH / kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rows = TH < 256 ? 256 / TH : 1;
  const int64_t row = p.row0 + static_cast<int64_t>(blockIdx.x) * rows + (TH < 256 ? wave : 0);
  if (TH < 256 && row >= p.end) return;  // a wave's own row: no barrier in that form
  const int t = TH < 256 ? threadIdx.x & 63 : threadIdx.x;
  const int units = p.hidden / 8;
  const int64_t base = row * p.hidden;

  auto fetch = [&](int u, float v[8]) {
    load8<XT>(p.x, base + 8 * u, v);
    if (p.residual) {
      float o[8];
      load8<XT>(p.residual, base + 8 * u, o);
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] += o[i];
      round_store<XT>(v, p.total, base + 8 * u);
    }
  };
  auto squares = [](const float v[8]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) a = __builtin_fmaf(v[i], v[i], a);
    return a;
  };
  float v[V][8];
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < V; j++) {
    const int u = t + j * TH;
    if (u < units) {
      fetch(u, v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[j][i] = 0.0f;
    }
  }
#pragma unroll
  for (int j = 0; j < V; j++) sum += squares(v[j]);
  if constexpr (LOOP) {
    for (int u = t + V * TH; u < units; u += TH) {
      float o[8];
      fetch(u, o);
      sum += squares(o);
    }
  }
  sum = row_total<false>(sum, part, TH / kWave, wave);
  const float r = 1.0f / __builtin_sqrtf(sum / static_cast<float>(p.hidden) + p.eps);

  auto scaled = [&](int u, float a[8]) {
    float w[8];
    load_weight(p.weight, p.wt, 8 * static_cast<int64_t>(u), w);
#pragma unroll
    for (int i = 0; i < 8; i++) a[i] = a[i] * r * w[i];
  };
  const void* const again = p.residual ? p.total : p.x;  // LOOP: this thread's own stores, or x
  float top = 0.0f;
  if (p.act == QBLK_ACT_I8) {
#pragma unroll
    for (int j = 0; j < V; j++) {
      if (t + j * TH >= units) continue;
      float a[8];
#pragma unroll
      for (int i = 0; i < 8; i++) a[i] = v[j][i];
      scaled(t + j * TH, a);
#pragma unroll
      for (int i = 0; i < 8; i++) top = max_nan(top, __builtin_fabsf(a[i]));
    }
    if constexpr (LOOP) {
      for (int u = t + V * TH; u < units; u += TH) {
        float a[8];
        load8<XT>(again, base + 8 * u, a);
        scaled(u, a);
#pragma unroll
        for (int i = 0; i < 8; i++) top = max_nan(top, __builtin_fabsf(a[i]));
      }
    }
    top = row_total<true>(top, part, TH / kWave, wave) / 127.0f;
    if (t == 0) static_cast<float*>(p.scale)[row] = top;
  }
  // whole waves take part: groups of 16 lanes and quads are on or off together
  auto emit = [&](int u, float a[8], bool on) {
    if (on) {
      scaled(u, a);
    }
    uint32_t c[2];
    const int64_t at = base + 8 * u;
    switch (p.act) {
      case QBLK_ACT_F8: {
        const float s = quant_group(a, c);
        if (on) {
          *reinterpret_cast<u32x2*>(p.codes + at) = u32x2{c[0], c[1]};
          if ((t & 15) == 0) static_cast<float*>(p.scale)[at / kGroup] = s;
        }
        break;
      }
      case QBLK_ACT_MXFP8: {
        const uint32_t b = mx_scale<true>(quad_max(top_bits<8>(a)));
        mx_codes<true, 8>(a, b, c);
        if (on) {
          *reinterpret_cast<u32x2*>(p.codes + at) = u32x2{c[0], c[1]};
          if ((t & 3) == 0) static_cast<uint8_t*>(p.scale)[at / kMxBlock] = static_cast<uint8_t>(b);
        }
        break;
      }
      case QBLK_ACT_MXFP4: {
        const uint32_t b = mx_scale<false>(quad_max(top_bits<8>(a)));
        mx_codes<false, 8>(a, b, c);
        if (on) {
          *reinterpret_cast<uint32_t*>(p.codes + at / 2) = c[0];
          if ((t & 3) == 0) static_cast<uint8_t*>(p.scale)[at / kMxBlock] = static_cast<uint8_t>(b);
        }
        break;
      }
      case QBLK_ACT_I8: {
        int n[8];
        codes8(a, top, -127.0f, 127.0f, n);
#pragma unroll
        for (int i = 0; i < 2; i++)
          c[i] = (n[4 * i] & 255) | ((n[4 * i + 1] & 255) << 8) | ((n[4 * i + 2] & 255) << 16) | (static_cast<uint32_t>(n[4 * i + 3]) << 24);
        if (on) *reinterpret_cast<u32x2*>(p.codes + at) = u32x2{c[0], c[1]};
        break;
      }
    }
    if (on && p.y) round_store<XT>(a, p.y, at);
  };
#pragma unroll
  for (int j = 0; j < V; j++) emit(t + j * TH, v[j], t + j * TH < units);
  if constexpr (LOOP) {
    for (int u0 = V * TH; u0 < units; u0 += TH) {
      const int u = u0 + t;
      float a[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (u < units) load8<XT>(again, base + 8 * u, a);
      emit(u, a, u < units);
    }
  }
}

template <int XT, int TH, int V, bool LOOP>
hipError_t norm(const NormArgs& all, int64_t n, hipStream_t s) {
  constexpr int rows = TH < 256 ? 256 / TH : 1, threads = TH < 256 ? 256 : TH;
  return in_pieces(n, rows, threads, [&](int64_t r0, int64_t c) {
    NormArgs a = all;
    a.row0 = r0;
    a.end = r0 + c;
    k_rmsnorm<XT, TH, V, LOOP><<<dim3(static_cast<unsigned>((c + rows - 1) / rows)), threads, 0, s>>>(a);
    return hipGetLastError();
  });
}

template <int XT>
hipError_t norm_width(const NormArgs& a, int64_t n, hipStream_t s) {
  const int units = a.hidden / 8;
  if (units <= 64) return norm<XT, 64, 1, false>(a, n, s);
  if (units <= 256) return norm<XT, 256, 1, false>(a, n, s);
  if (units <= 512) return norm<XT, 256, 2, false>(a, n, s);
  if (units <= 1024) return norm<XT, 256, 4, false>(a, n, s);
  if (units <= 2048) return norm<XT, 1024, 2, false>(a, n, s);
  return norm<XT, 1024, 4, true>(a, n, s);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, int64_t n, hipStream_t s) {
  log_launch("rmsnorm n=%lld hidden=%d act=%d", (long long)n, a.hidden, a.act);
  switch (a.xt) {
    case QBLK_F32: return norm_width<QBLK_F32>(a, n, s);
    case QBLK_F16: return norm_width<QBLK_F16>(a, n, s);
    default: return norm_width<QBLK_BF16>(a, n, s);
  }
}

}  // namespace qblk
