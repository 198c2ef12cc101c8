// qblk_f8.hip -- 8-bit floating point (OCP e4m3) weights and activations with
// one fp32 scale per block of 128, and their products, on gfx950.
//
//   weights      W[r,c]  = sw[r/128, c/128] * qw[r,c]     (128 x 128 blocks)
//   activations  X[t,c]  = sx[t, c/128] * qx[t,c]         (1 x 128 groups)
//   scale        s = max|v| / 448 in fp32; code = e4m3(clamp(v / s, +-448)),
//                both divisions IEEE fp32; s = 0 gives code 0
//   product      Y[t,r] = sum_g sx[t,g] sw[r/128,g] (sum_{c in g} qw qx)
//
// A scale covers 128 columns on both sides, so the inner sum over a group is
// formed on the matrix cores from the bare codes and scaled once, in fp32.
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
template <int XT>
struct Src;  // element type of x as stored
template <>
struct Src<QBLK_F32> {
  typedef float type;
};
template <>
struct Src<QBLK_F16> {
  typedef uint16_t type;
};
template <>
struct Src<QBLK_BF16> {
  typedef uint16_t type;
};

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

// max over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ float row16_max(float v) {
  v = __builtin_fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, true)));
  v = __builtin_fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, true)));
  v = __builtin_fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xF, 0xF, true)));
  v = __builtin_fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xF, 0xF, true)));
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
  for (int i = 0; i < N; i++) q[i] = __builtin_amdgcn_fmed3f(q[i], -kF8Max, kF8Max);
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
  for (int i = 0; i < 8; i++) a = __builtin_fmaxf(a, __builtin_fabsf(v[i]));
  const float s = row16_max(a) / kF8Max;
  codes_f8<8>(v, s, code);
  return s;
}

// ------------------------------------------------------ activation codes
// HBM bound: 2 or 4 bytes read and 1 + 1/32 written per value; 16 lanes to a
// group, so a wave reads 1 KB (16-bit input) of consecutive values at once.
template <int XT>
__global__ __launch_bounds__(256) void k_quant_act_f8(const void* __restrict__ x, int64_t group0, int64_t groups,
                                                      uint8_t* __restrict__ xq, float* __restrict__ scale) {
  int64_t g = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  const bool on = g < groups;
  g = group0 + (on ? g : groups - 1);  // whole waves take part in the row reductions
  const int l = threadIdx.x & 15;
  float v[8];
  load8<XT>(x, g * kGroup + 8 * l, v);
  uint32_t code[2];
  const float s = quant_group(v, code);
  if (on) {
    *reinterpret_cast<u32x2*>(xq + g * kGroup + 8 * l) = u32x2{code[0], code[1]};
    if (l == 0) scale[g] = s;
  }
}

// ---------------------------------------------------------- weight codes
// One workgroup per 128 x 128 block; a thread holds 64 of its values in
// registers between the maximum and the codes, so the block is read once.
template <int XT>
__global__ __launch_bounds__(256) void k_quant_f8(const void* __restrict__ w, int64_t rows, int64_t k,
                                                  int64_t block0, uint8_t* __restrict__ codes,
                                                  float* __restrict__ scale) {
  __shared__ float part[4];
  const int64_t b = block0 + blockIdx.x;
  const int64_t per = k / kGroup;
  const int64_t br = b / per, bc = b - br * per;
  // 16 threads to a row, 16 rows at a time
  const int l = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  float v[8][8];
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const int64_t row = br * kGroup + 16 * j + r0;
    if (row < rows) {
      load8<XT>(w, row * k + bc * kGroup + 8 * l, v[j]);
#pragma unroll
      for (int i = 0; i < 8; i++) a = __builtin_fmaxf(a, __builtin_fabsf(v[j][i]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[j][i] = 0.0f;
    }
  }
  a = group_max<kWave>(a);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
  __syncthreads();
  a = __builtin_fmaxf(__builtin_fmaxf(part[0], part[1]), __builtin_fmaxf(part[2], part[3]));
  const float s = a / kF8Max;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const int64_t row = br * kGroup + 16 * j + r0;
    uint32_t c[2];
    codes_f8<8>(v[j], s, c);
    if (row < rows) *reinterpret_cast<u32x2*>(codes + row * k + bc * kGroup + 8 * l) = u32x2{c[0], c[1]};
  }
  if (threadIdx.x == 0) scale[b] = s;
}

// ------------------------------------------------------------- few tokens
// 8 e4m3 codes as bf16 (every e4m3 value is a bf16 value): two per conversion.
__device__ __forceinline__ bf16x8_n widen8(uint32_t a, uint32_t b) {
  const bf16x2_n p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const bf16x2_n p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const bf16x2_n p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const bf16x2_n p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return bf16x8_n{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

__device__ __forceinline__ void store_y(void* y, int64_t at, float v, int yt) {
  if (yt == QBLK_F32)
    static_cast<float*>(y)[at] = v;
  else
    static_cast<uint16_t*>(y)[at] = yt == QBLK_F16 ? f32_to_f16_bits(v) : f32_to_bf16_bits(v);
}

// Up to 16 T tokens, bound by the weight bytes.  A workgroup owns NR tiles of
// 16 rows for all its tokens and splits the columns over its waves (wave w
// takes groups w, w + WAVES, ...); the waves' fp32 partial sums meet in LDS in
// a fixed order.  The codes are widened to bf16 and multiplied on the bf16
// matrix cores, whose fp32 sums of such products are exact to fp32 rounding
// (the fp8 matrix instructions round a group's sum to about 2^-17 of
// sum|qw qx|); with so few tokens the widening and the matrix work hide
// behind the weight stream.
//
// A lane's 16-byte loads are 16 consecutive codes of one row (weights: row
// l & 15; tokens: token l & 15; quarter l >> 4 of a 64-code run), and the two
// operands meet in the same order, so no lane exchange is needed.
//
// GATE: the tiles are 16 gate rows and the 16 up rows i further on; the
// result is h = silu(gate) * up in fp32 (n x i).
// XSRC: kCodes = x given as codes and scales; else the element type of x,
// which the workgroup quantizes into LDS itself (one launch less; every
// workgroup repeats it, so only for few values, see launch_linear_f8).
constexpr int kCodes = 3;
constexpr int kDepth = 4;  // groups of a wave whose loads are in flight together

template <int T, int NR, int WAVES, bool GATE, int XSRC>
__global__ __launch_bounds__(WAVES* kWave) void k_f8_few(const uint8_t* __restrict__ w, const float* __restrict__ ws,
                                                         int m, int k, const void* __restrict__ xv,
                                                         const float* __restrict__ xs, int n, void* __restrict__ y,
                                                         int yt, int64_t up_row) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = k / kGroup;
  const int t0 = blockIdx.y * 16 * T;
  const int row0 = blockIdx.x * (GATE ? 16 : 16 * NR);
  const int r = lane & 15, q = lane >> 4;
  n -= t0;

  const uint8_t* wp[NR];
  const float* sp[NR];
#pragma unroll
  for (int a = 0; a < NR; a++) {
    const int64_t base = GATE ? row0 + a * up_row : row0 + 16 * a;
    const int64_t last = GATE ? base + 15 : m - 1;
    const int64_t row = base + r < last ? base + r : last;
    wp[a] = w + row * k + 16 * q;
    sp[a] = ws + (base < last ? base : last) / kGroup * G;
  }

  const uint8_t* xq = nullptr;
  int xstride = 0;
  if constexpr (XSRC != kCodes) {
    xstride = k + 16;
    float* sl = reinterpret_cast<float*>(lds);
    uint8_t* ql = lds + ((n < 16 * T ? n : 16 * T) * G * 4 + 15) / 16 * 16;
    const int nt = n < 16 * T ? n : 16 * T;
    for (int u = threadIdx.x >> 4; u < (nt * G + 3) / 4 * 4; u += WAVES * 4) {
      const bool on = u < nt * G;
      const int uu = on ? u : nt * G - 1;
      const int t = uu / G, g = uu - t * G;
      float v[8];
      load8<XSRC>(xv, static_cast<int64_t>(t0 + t) * k + g * kGroup + 8 * r, v);
      uint32_t c[2];
      const float s = quant_group(v, c);
      if (on) {
        *reinterpret_cast<u32x2*>(ql + t * xstride + g * kGroup + 8 * r) = u32x2{c[0], c[1]};
        if (r == 0) sl[uu] = s;
      }
    }
    __syncthreads();
    xq = ql;
  }

  const uint8_t* xp[T];
  const float* xsp[T];
#pragma unroll
  for (int t = 0; t < T; t++) {
    const int tok = 16 * t + r < n ? 16 * t + r : n - 1;
    if constexpr (XSRC == kCodes) {
      xp[t] = static_cast<const uint8_t*>(xv) + static_cast<int64_t>(t0 + tok) * k + 16 * q;
      xsp[t] = xs + static_cast<int64_t>(t0 + tok) * G;
    } else {
      xp[t] = xq + tok * xstride + 16 * q;
      xsp[t] = reinterpret_cast<const float*>(lds) + tok * G;
    }
  }

  float4_t acc[NR][T];
#pragma unroll
  for (int a = 0; a < NR; a++)
#pragma unroll
    for (int t = 0; t < T; t++) acc[a][t] = float4_t{0, 0, 0, 0};

  for (int g0 = wave; g0 < G; g0 += WAVES * kDepth) {
    u32x4 wr[kDepth][NR][2];
    float sw[kDepth][NR];
#pragma unroll
    for (int d = 0; d < kDepth; d++) {
      const int g = g0 + d * WAVES < G ? g0 + d * WAVES : G - 1;
#pragma unroll
      for (int a = 0; a < NR; a++) {
        wr[d][a][0] = *reinterpret_cast<const u32x4*>(wp[a] + g * kGroup);
        wr[d][a][1] = *reinterpret_cast<const u32x4*>(wp[a] + g * kGroup + 64);
        sw[d][a] = sp[a][g];
      }
    }
#pragma unroll
    for (int d = 0; d < kDepth; d++) {
      const bool on = g0 + d * WAVES < G;
      const int g = on ? g0 + d * WAVES : G - 1;
#pragma unroll
      for (int t = 0; t < T; t++) {
        const u32x4 x0 = *reinterpret_cast<const u32x4*>(xp[t] + g * kGroup);
        const u32x4 x1 = *reinterpret_cast<const u32x4*>(xp[t] + g * kGroup + 64);
        const float sx = on ? xsp[t][g] : 0.0f;
        const bf16x8_n b0 = widen8(x0.x, x0.y), b1 = widen8(x0.z, x0.w);
        const bf16x8_n b2 = widen8(x1.x, x1.y), b3 = widen8(x1.z, x1.w);
#pragma unroll
        for (int a = 0; a < NR; a++) {
          const u32x4 w0 = wr[d][a][0], w1 = wr[d][a][1];
          float4_t p = {0, 0, 0, 0};
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w0.x, w0.y), b0, p, 0, 0, 0);
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w0.z, w0.w), b1, p, 0, 0, 0);
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w1.x, w1.y), b2, p, 0, 0, 0);
          p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w1.z, w1.w), b3, p, 0, 0, 0);
          const float s = sx * sw[d][a];
#pragma unroll
          for (int i = 0; i < 4; i++) acc[a][t][i] = __builtin_fmaf(p[i], s, acc[a][t][i]);
        }
      }
    }
  }

  // lane (r, q) holds rows 4q..4q+3 of each tile for token r of each 16
  if constexpr (XSRC != kCodes) __syncthreads();  // the codes in LDS are read
  float4_t* red = reinterpret_cast<float4_t*>(lds);
#pragma unroll
  for (int a = 0; a < NR; a++)
#pragma unroll
    for (int t = 0; t < T; t++) red[((wave * NR + a) * T + t) * 64 + lane] = acc[a][t];
  __syncthreads();
  const float* rf = reinterpret_cast<const float*>(lds);
  const int tiles = GATE ? 1 : NR;
  for (int o = threadIdx.x; o < tiles * T * 256; o += WAVES * kWave) {
    const int rr = o & 15, tok = (o >> 4) % (16 * T), a = o / (256 * T);
    const int at = ((a * T + (tok >> 4)) * 64 + (rr >> 2) * 16 + (tok & 15)) * 4 + (rr & 3);
    float sum = 0.0f, up = 0.0f;
#pragma unroll
    for (int v = 0; v < WAVES; v++) {
      sum += rf[v * NR * T * 256 + at];
      if constexpr (GATE) up += rf[(v * NR + 1) * T * 256 + at];
    }
    if (tok >= n) continue;
    const int row = row0 + 16 * a + rr;
    if constexpr (GATE)
      static_cast<float*>(y)[static_cast<int64_t>(t0 + tok) * up_row + row] = silu_mul(sum, up);
    else if (row < m)
      store_y(y, static_cast<int64_t>(t0 + tok) * m + row, sum, yt);
  }
}

// ------------------------------------------------------------ many tokens
// Bound by the matrix cores.  A workgroup of 8 waves owns 256 rows x 64 NT
// tokens; a group of 128 columns is one stage in LDS (32 KB + 8 NT KB, two
// stages) and one K=128 fp8 matrix instruction per 16 x 16 tile, whose result
// is scaled by sx[t,g] * sw[r,g] into the fp32 accumulators: four multiply-adds
// per lane beside 32 matrix-core cycles.  Waves are 2 (rows) x 4 (tokens);
// wave row a holds rows 64a..64a+63 of the tile's first and second 128-row
// halves, so that for GATE, where the halves are 128 gate rows and their 128
// up rows, a lane holds both factors of silu(gate) * up.
//
// Rounding.  The fp8 instructions add fp32, except that they bring each 8
// neighbouring products to the largest one's exponent with about 16 bits:
// 1e-5 of the result in the 2-norm on normal data (measured), up to 2^-13 of
// the largest product in a group of 8 that spans many binades.  That is far
// below half a unit of a 16-bit result, but not of an fp32 one; and where the
// result is quantized again (the gated layer) it moves 1e-4 of the codes to
// the neighbouring one, which 11 bits of result show (relative error 1.0e-3
// instead of 2.6e-4) and 8 hardly (2.2e-3, 1.7e-3).  EXACT widens the codes
// to bf16 and multiplies those, at half the rate: products and sums are then
// exact to fp32 rounding.  It is taken for fp32 results and for the first
// product of a gated layer with an fp16 or fp32 result.
//
// LDS layout: 128 bytes per row, the row's 16-byte chunk c at c ^ (row & 7),
// so that the 16 rows of an operand read hit 8 different chunk columns.  The
// stages are filled by loads straight to LDS, which write 64 x 16 consecutive
// bytes: the exchange of chunks is made on the global address.
typedef int int8v __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void glob_void;

constexpr int kTileRows = 256;

template <int NT>
struct Stage {
  uint8_t a[kTileRows * kGroup];
  uint8_t b[64 * NT * kGroup];
};
// The scales of 4 groups: every token's, and (in the first 8) the two row
// halves'; as the copies to LDS leave them, 64 consecutive floats each.
template <int NT>
struct Scales {
  float x[64 * NT][4];
  float w[64];
};
// Stages in LDS: what a copy has to reach memory and come back is a stage's
// work with two of them.  The smaller tiles work that much shorter on one, and
// have room for three.
template <int NT>
constexpr int kStages = NT == 4 ? 2 : 3;
template <int NT>
struct TileLds {
  Stage<NT> st[kStages<NT>];
  Scales<NT> sc[2];
};

// A group's operands of a 16-row tile: lane (row r, quarter q) gives the row's
// chunks q and q + 4 (both sides in the same order).  EXACT: widened to bf16.
template <bool EXACT>
struct Frag;
template <>
struct Frag<false> {
  int8v v;
  __device__ __forceinline__ void load(const uint8_t* base, int row, int q) {
    const int key = (row >> 1) & 7;
    const u32x4 lo = *reinterpret_cast<const u32x4*>(base + row * kGroup + ((q ^ key) << 4));
    const u32x4 hi = *reinterpret_cast<const u32x4*>(base + row * kGroup + (((q + 4) ^ key) << 4));
    v = int8v{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
              static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
  }
};
template <>
struct Frag<true> {
  bf16x8_n v[4];
  __device__ __forceinline__ void load(const uint8_t* base, int row, int q) {
    const int key = (row >> 1) & 7;
    const u32x4 lo = *reinterpret_cast<const u32x4*>(base + row * kGroup + ((q ^ key) << 4));
    const u32x4 hi = *reinterpret_cast<const u32x4*>(base + row * kGroup + (((q + 4) ^ key) << 4));
    v[0] = widen8(lo.x, lo.y);
    v[1] = widen8(lo.z, lo.w);
    v[2] = widen8(hi.x, hi.y);
    v[3] = widen8(hi.z, hi.w);
  }
};
__device__ __forceinline__ float4_t group_product(const Frag<false>& a, const Frag<false>& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, float4_t{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ float4_t group_product(const Frag<true>& a, const Frag<true>& b) {
  float4_t c = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; i++) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

struct TileArgs {
  const uint8_t* w;
  const float* ws;
  const uint8_t* xq;
  const float* xs;
  void* y;        // n x m (GATE: codes of h, n x up)
  float* hs;      // GATE: scales of h
  float* part;    // split K: partial sums, [split][n][m]
  int m, k, n, yt, up, row_tiles, tok_tiles, groups_per_split;
};

template <int NT, bool GATE, bool SPLIT, bool EXACT>
__global__ __launch_bounds__(512, 2) void k_f8_tile(TileArgs p) {
  extern __shared__ __align__(16) uint8_t lds[];
  Stage<NT>* const st = reinterpret_cast<TileLds<NT>*>(lds)->st;
  Scales<NT>* const scl = reinterpret_cast<TileLds<NT>*>(lds)->sc;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int G = p.k / kGroup;

  // Workgroups go to the 8 XCDs in turn; each XCD takes a run of consecutive
  // tiles (token tiles fastest), so that its L2 holds the few row tiles and
  // the token tiles that its 32 CUs work on together.
  const int tiles = p.row_tiles * p.tok_tiles;
  const int b = blockIdx.x, xcd = b & 7;
  const int tile = xcd * (tiles >> 3) + (xcd < (tiles & 7) ? xcd : (tiles & 7)) + (b >> 3);
  const int band = tile / (8 * p.row_tiles), in_band = tile - band * 8 * p.row_tiles;
  const int wide = p.tok_tiles - 8 * band < 8 ? p.tok_tiles - 8 * band : 8;
  const int rt = in_band / wide, tt = 8 * band + in_band - rt * wide;
  const int row0 = rt * (GATE ? 128 : kTileRows), t0 = tt * 64 * NT;
  const int g0 = SPLIT ? blockIdx.y * p.groups_per_split : 0;
  const int g1 = SPLIT ? (g0 + p.groups_per_split < G ? g0 + p.groups_per_split : G) : G;

  // What this lane copies per stage: a 16-byte chunk of 4 rows of A and NT of
  // B, as 32-bit offsets from the tile's first row (of the up half for GATE).
  // Rows past the matrix repeat its last one; their results are not stored.
  const int64_t second = GATE ? static_cast<int64_t>(p.up) + row0 : row0;
  const uint8_t* abase[2] = {p.w + static_cast<int64_t>(row0) * p.k, p.w + second * p.k};
  const uint8_t* bbase = p.xq + static_cast<int64_t>(t0) * p.k;
  uint32_t ao[4], bo[NT];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int row = 64 * i + 8 * wave + (lane >> 3);
    int at = GATE ? row & 127 : row;
    if (!GATE && at > p.m - 1 - row0) at = p.m - 1 - row0;
    ao[i] = static_cast<uint32_t>(at) * static_cast<uint32_t>(p.k) + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
  }
#pragma unroll
  for (int i = 0; i < NT; i++) {
    const int row = 64 * i + 8 * wave + (lane >> 3);
    const int at = t0 + row < p.n ? row : p.n - 1 - t0;
    bo[i] = static_cast<uint32_t>(at) * static_cast<uint32_t>(p.k) + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
  }
  // chunk i of 4 + NT: the rows of A, then those of B
  auto copy = [&](Stage<NT>& s, int g, int i) {
    const int64_t at = static_cast<int64_t>(g) * kGroup;
    if (i < 4)
      __builtin_amdgcn_global_load_lds((glob_void*)((i < 2 ? abase[0] : abase[1]) + at + ao[i & 3]),
                                       (lds_void*)(s.a + (64 * i + 8 * wave) * kGroup), 16, 0, 0);
    else if (i < 4 + NT)
      __builtin_amdgcn_global_load_lds((glob_void*)(bbase + at + bo[i - 4]),
                                       (lds_void*)(s.b + (64 * (i - 4) + 8 * wave) * kGroup), 16, 0, 0);
  };

  const int wm = wave & 1, wn = wave >> 1;
  // Scales, 4 groups at a time (the 16 bytes of a token that lie together),
  // copied to LDS like the codes: read from memory a group at a time they were
  // as many accesses as the codes.
  const float* swp;
  {
    const int h = (lane >> 2) & 1;
    int64_t row = GATE ? row0 + static_cast<int64_t>(h) * p.up : row0 + 128 * h;
    if (row > p.m - 1) row = p.m - 1;
    swp = p.ws + row / kGroup * G;
  }
  auto copy_scales = [&](Scales<NT>& s, int g) {
    const int gg = g + (lane & 3) < g1 ? g + (lane & 3) : g1 - 1;
#pragma unroll
    for (int u = 0; u < (NT + 1) / 2; u++) {
      const int first = ((wave + 8 * u) & (4 * NT - 1)) * 16;
      int tok = t0 + first + (lane >> 2);
      if (tok > p.n - 1) tok = p.n - 1;
      __builtin_amdgcn_global_load_lds((glob_void*)(p.xs + static_cast<int64_t>(tok) * G + gg), (lds_void*)(s.x[first]), 4, 0, 0);
    }
    if (wave == 0) __builtin_amdgcn_global_load_lds((glob_void*)(swp + gg), (lds_void*)(s.w), 4, 0, 0);
  };

  float4_t acc[8][NT];
#pragma unroll
  for (int i = 0; i < 8; i++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[i][j] = float4_t{0, 0, 0, 0};

  // Software pipeline.  Within a stage: while the matrix cores work on row
  // tile i, its successor's operand is read from LDS and tile i - 1 is scaled.
  // Across stages: at the last row tile every operand of the stage is in
  // registers, so one barrier there frees its buffer for the copies two
  // stages on and shows the next stage's, whose first operands are read
  // behind the last matrix instructions.
  Frag<EXACT> bf[NT], af[2];
  float4_t c[2][NT];
  float sc[2][NT];
  auto arow = [&](int i) { return (i >> 2) * 128 + wm * 64 + (i & 3) * 16 + r; };
  auto scale = [&](int i, int j) {
#pragma unroll
    for (int e = 0; e < 4; e++) acc[i][j][e] = __builtin_fmaf(c[i & 1][j][e], sc[i >> 2][j], acc[i][j][e]);
  };
  copy_scales(scl[0], g0);
#pragma unroll
  for (int i = 0; i < 4 + NT; i++) copy(st[0], g0, i);
  if constexpr (kStages<NT> == 3) {
#pragma unroll
    for (int i = 0; i < 4 + NT; i++) copy(st[1], g0 + 1 < g1 ? g0 + 1 : g0, i);
  }
  __syncthreads();
  constexpr int kAhead = kStages<NT> - 1;  // stages whose copies are on their way
  auto group_at = [&](int step) { return g0 + step < g1 ? g0 + step : g1 - 1; };
  copy(st[kAhead], group_at(kAhead), 0);
  copy(st[kAhead], group_at(kAhead), 1);
  af[0].load(st[0].a, arow(0), q);
#pragma unroll
  for (int j = 0; j < NT; j++) bf[j].load(st[0].b, (wn * NT + j) * 16 + r, q);
  int now = 0;
  for (int g = g0; g < g1; g++) {
    const int step = g - g0;
    Stage<NT>& cur = st[now];
    Stage<NT>& nxt = st[now + 1 < kStages<NT> ? now + 1 : 0];
    Stage<NT>& far = st[now > 0 ? now - 1 : kStages<NT> - 1];  // the one before, filled kAhead stages on
    const int gf = group_at(step + kAhead), gc = group_at(step + kAhead + 1);
    now = now + 1 < kStages<NT> ? now + 1 : 0;
    {
      const Scales<NT>& l = scl[(step >> 2) & 1];
      const float w0 = l.w[step & 3], w1 = l.w[4 + (step & 3)];
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const float x = l.x[(wn * NT + j) * 16 + r][step & 3];
        sc[0][j] = x * w0;
        sc[1][j] = x * w1;
      }
    }
    if ((step & 3) == 0) copy_scales(scl[((step >> 2) + 1) & 1], g + 4 < g1 ? g + 4 : g1 - 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      if (i + 1 < 8) {
        af[(i + 1) & 1].load(cur.a, arow(i + 1), q);
      } else if constexpr (kStages<NT> == 2) {
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
      } else {
        // as __syncthreads, but leaving the newest 4 + NT loads under way: the
        // copies of the stage after next (all older ones are the next stage's)
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_s_waitcnt(0x0070 | (4 + NT));  // vmcnt(4 + NT) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int j = 0; j < NT; j++) {
        c[i & 1][j] = group_product(af[i & 1], bf[j]);
        if (i > 0) scale(i - 1, j);
        if (i + 1 == 8) bf[j].load(nxt.b, (wn * NT + j) * 16 + r, q);
      }
      // Each matrix instruction with the four multiply-adds of a finished tile
      // behind it; the LDS reads after the first (before it they would be
      // waited for together with the operand it needs).  The copies are spread
      // over four row tiles: issued at once they hold up the waves' issue.
      if (i + 1 < 8) {
        if (i < 3) {
          copy(far, gf, 2 * i + 2);
          copy(far, gf, 2 * i + 3);
        }
#pragma unroll
        for (int j = 0; j < NT && !EXACT; j++) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          if (j == 0) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
          if (j < 2) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
      } else {
        af[0].load(nxt.a, arow(0), q);
        copy(cur, gc, 0);
        copy(cur, gc, 1);
#pragma unroll
        for (int j = 0; j < NT && !EXACT; j++) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < NT; j++) scale(7, j);
  }
  __syncthreads();  // the last copies have landed: LDS may be used again, and left

  if constexpr (GATE) {
    // h = silu(gate) * up; a group of 128 columns is the tile's rows: its
    // maximum over this lane's 16, the four quarters and the two wave rows
    float top[NT];
#pragma unroll
    for (int j = 0; j < NT; j++) {
      float a = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          acc[i][j][e] = silu_mul(acc[i][j][e], acc[i + 4][j][e]);
          a = __builtin_fmaxf(a, __builtin_fabsf(acc[i][j][e]));
        }
      a = __builtin_fmaxf(a, __shfl_xor(a, 16, kWave));
      top[j] = __builtin_fmaxf(a, __shfl_xor(a, 32, kWave));
    }
    float* m2 = reinterpret_cast<float*>(lds);  // [2][64 NT]
    __syncthreads();
    if (q == 0) {
#pragma unroll
      for (int j = 0; j < NT; j++) m2[wm * 64 * NT + (wn * NT + j) * 16 + r] = top[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const int in = (wn * NT + j) * 16 + r, tok = t0 + in;
      const float s = __builtin_fmaxf(m2[in], m2[64 * NT + in]) / kF8Max;
      float v[16];
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) v[4 * i + e] = acc[i][j][e];
      codes_f8<16>(v, s, c);
      if (tok < p.n) {
        uint8_t* out = static_cast<uint8_t*>(p.y) + static_cast<int64_t>(tok) * p.up + row0 + wm * 64 + 4 * q;
#pragma unroll
        for (int i = 0; i < 4; i++) *reinterpret_cast<uint32_t*>(out + 16 * i) = c[i];
        if (wm == 0 && q == 0) p.hs[static_cast<int64_t>(tok) * (p.up / kGroup) + row0 / kGroup] = s;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const int tok = t0 + (wn * NT + j) * 16 + r;
      if (tok >= p.n) continue;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int row = row0 + (i >> 2) * 128 + wm * 64 + (i & 3) * 16 + 4 * q;
        if (row >= p.m) continue;
        const int64_t at = static_cast<int64_t>(tok) * p.m + row;
        const bool whole = row + 4 <= p.m && (p.m & 3) == 0;  // 4 consecutive values, aligned
        if (SPLIT || p.yt == QBLK_F32) {
          float* y = SPLIT ? p.part + static_cast<int64_t>(blockIdx.y) * p.n * p.m : static_cast<float*>(p.y);
          if (whole) {
            *reinterpret_cast<float4_t*>(y + at) = acc[i][j];
          } else {
#pragma unroll
            for (int e = 0; e < 4; e++)
              if (row + e < p.m) y[at + e] = acc[i][j][e];
          }
        } else {
          uint16_t h[4];
#pragma unroll
          for (int e = 0; e < 4; e++) h[e] = p.yt == QBLK_F16 ? f32_to_f16_bits(acc[i][j][e]) : f32_to_bf16_bits(acc[i][j][e]);
          uint16_t* y = static_cast<uint16_t*>(p.y) + at;
          if (whole) {
            *reinterpret_cast<u32x2*>(y) = u32x2{h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16)};
          } else {
#pragma unroll
            for (int e = 0; e < 4; e++)
              if (row + e < p.m) y[e] = h[e];
          }
        }
      }
    }
  }
}

// y = the sum of the splits' partial products, in their order
__global__ __launch_bounds__(256) void k_f8_join(const float* __restrict__ part, int64_t first, int64_t count,
                                                 int64_t stride, int splits, void* __restrict__ y, int yt) {
  int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= count) return;
  i += first;
  float v = 0.0f;
  for (int s = 0; s < splits; s++) v += part[s * stride + i];
  store_y(y, i, v, yt);
}

// LDS of k_f8_few: the waves' partial sums, or the quantized x before them
constexpr int kFewWaves = 8;
size_t few_lds(int T, int NR, bool codes, int n, int k) {
  const size_t red = static_cast<size_t>(kFewWaves) * NR * T * 1024;
  const int nt = n < 16 * T ? n : 16 * T;
  const size_t xq = codes ? 0 : (static_cast<size_t>(nt) * (k / kGroup) * 4 + 15) / 16 * 16 + static_cast<size_t>(nt) * (k + 16);
  return red > xq ? red : xq;
}

template <int T, int NR, bool GATE, int XSRC>
hipError_t few(const uint8_t* w, const float* ws, int64_t m, int64_t k, const void* x, const float* xs, int64_t n,
               void* y, int yt, int64_t up_row, hipStream_t s) {
  const int per = GATE ? 16 : 16 * NR;
  const int64_t rows = GATE ? up_row : m;
  const dim3 grid(static_cast<unsigned>((rows + per - 1) / per), static_cast<unsigned>((n + 16 * T - 1) / (16 * T)));
  const size_t lds = few_lds(T, NR, XSRC == kCodes, static_cast<int>(n), static_cast<int>(k));
  log_launch("f8 few%s rows=%lld k=%lld n=%lld T=%d NR=%d x=%d lds=%zu", GATE ? " gate" : "", (long long)m,
             (long long)k, (long long)n, T, NR, XSRC, lds);
  k_f8_few<T, NR, kFewWaves, GATE, XSRC><<<grid, kFewWaves * kWave, lds, s>>>(
      w, ws, static_cast<int>(m), static_cast<int>(k), x, xs, static_cast<int>(n), y, yt, up_row);
  return hipGetLastError();
}

template <bool GATE>
hipError_t few_codes(const uint8_t* w, const float* ws, int64_t m, int64_t k, const uint8_t* xq, const float* xs,
                     int64_t n, void* y, int yt, int64_t up_row, hipStream_t s) {
  constexpr int NR = GATE ? 2 : 1;
  if (n <= 16) return few<1, NR, GATE, kCodes>(w, ws, m, k, xq, xs, n, y, yt, up_row, s);
  if (n <= 32) return few<2, NR, GATE, kCodes>(w, ws, m, k, xq, xs, n, y, yt, up_row, s);
  return few<4, NR, GATE, kCodes>(w, ws, m, k, xq, xs, n, y, yt, up_row, s);
}

template <bool GATE>
hipError_t few_values(const uint8_t* w, const float* ws, int64_t m, int64_t k, const void* x, int xt, int64_t n,
                      void* y, int yt, int64_t up_row, hipStream_t s) {
  constexpr int NR = GATE ? 2 : 1;
  switch (xt) {
    case QBLK_F32: return few<1, NR, GATE, QBLK_F32>(w, ws, m, k, x, nullptr, n, y, yt, up_row, s);
    case QBLK_F16: return few<1, NR, GATE, QBLK_F16>(w, ws, m, k, x, nullptr, n, y, yt, up_row, s);
    default: return few<1, NR, GATE, QBLK_BF16>(w, ws, m, k, x, nullptr, n, y, yt, up_row, s);
  }
}

// The tile kernel's shape for a product: tokens per tile and splits of K.
struct Plan {
  int nt, splits, per;  // 64 nt tokens; groups per split
};

Plan tile_plan(int64_t m, int64_t k, int64_t n, bool gate, bool exact) {
  const int64_t rt = (m + kTileRows - 1) / kTileRows, G = k / kGroup;
  const int cus = cu_count();
  Plan best{1, 1, static_cast<int>(G)};
  double cost = 1e30;
  for (int nt = 1; nt <= (exact ? 2 : 4); nt *= 2) {
    const int64_t tiles = rt * ((n + 64 * nt - 1) / (64 * nt));
    for (int sp = 1; sp <= 8; sp *= 2) {
      if (sp > 1 && (gate || G / sp < 4)) break;
      const int64_t per = (G + sp - 1) / sp;
      const int64_t rounds = (tiles * sp + cus - 1) / cus;
      // us: a stage of a tile (matrix cores, or the copies where nt is small), a tile's start and end, the partial sums
      const double stage = nt == 4 ? 1.9 : nt == 2 ? (exact ? 1.6 : 1.1) : 0.8;
      const double c = rounds * (per * stage + 4.0) + (sp > 1 ? 3.0 + 2.0 * sp * n * m * 4 / 4.0e6 : 0.0);
      if (c < cost) {
        cost = c;
        best = Plan{nt, sp, static_cast<int>(per)};
      }
    }
  }
  best.splits = static_cast<int>((G + best.per - 1) / best.per);
  return best;
}

template <int NT, bool GATE, bool SPLIT, bool EXACT>
hipError_t tile_go(const TileArgs& a, int splits, hipStream_t s) {
  constexpr size_t lds = sizeof(TileLds<NT>);
  static const hipError_t allowed = hipFuncSetAttribute(reinterpret_cast<const void*>(k_f8_tile<NT, GATE, SPLIT, EXACT>),
                                                        hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (allowed != hipSuccess) return allowed;
  k_f8_tile<NT, GATE, SPLIT, EXACT><<<dim3(static_cast<unsigned>(a.row_tiles * a.tok_tiles), static_cast<unsigned>(splits)),
                                     512, lds, s>>>(a);
  return hipGetLastError();
}

template <bool GATE, bool SPLIT>
hipError_t tile_nt(int nt, bool exact, const TileArgs& a, int splits, hipStream_t s) {
  if (exact) return nt == 1 ? tile_go<1, GATE, SPLIT, true>(a, splits, s) : tile_go<2, GATE, SPLIT, true>(a, splits, s);
  switch (nt) {
    case 1: return tile_go<1, GATE, SPLIT, false>(a, splits, s);
    case 2: return tile_go<2, GATE, SPLIT, false>(a, splits, s);
    default: return tile_go<4, GATE, SPLIT, false>(a, splits, s);
  }
}

// Y (or, for `up` > 0, the codes and scales of H) by the tile kernel
hipError_t tile_product(const uint8_t* w, const float* ws, int64_t m, int64_t k, const uint8_t* xq, const float* xs,
                        int64_t n, void* y, int yt, int64_t up, float* hs, bool exact, void* work, hipStream_t s) {
  const Plan plan = tile_plan(m, k, n, up > 0, exact);
  TileArgs a{w, ws, xq, xs, y, hs, static_cast<float*>(work), static_cast<int>(m), static_cast<int>(k), static_cast<int>(n), yt,
             static_cast<int>(up), static_cast<int>((m + kTileRows - 1) / kTileRows),
             static_cast<int>((n + 64 * plan.nt - 1) / (64 * plan.nt)), plan.per};
  log_launch("f8 tile%s%s m=%lld k=%lld n=%lld tokens=%d splits=%d", up > 0 ? " gate" : "", exact ? " exact" : "",
             (long long)m, (long long)k, (long long)n, 64 * plan.nt, plan.splits);
  if (up > 0) return tile_nt<true, false>(plan.nt, exact, a, 1, s);
  if (plan.splits == 1) return tile_nt<false, false>(plan.nt, exact, a, 1, s);
  const hipError_t e = tile_nt<false, true>(plan.nt, exact, a, plan.splits, s);
  if (e != hipSuccess) return e;
  return in_pieces(m * n, 256, 256, [&](int64_t first, int64_t c) {
    k_f8_join<<<dim3(static_cast<unsigned>((c + 255) / 256)), 256, 0, s>>>(a.part, first, c, m * n, plan.splits, y, yt);
    return hipGetLastError();
  });
}

// Products up to this many tokens run k_f8_few.
constexpr int64_t kFewTokens = 64;

// Whether a product quantizes its x inside every workgroup.
bool fused_quant(int64_t n, int64_t k) { return n <= 4 && n * k <= 32768; }

// y = 0 (an empty sum), any element type
__global__ __launch_bounds__(256) void k_zero(uint8_t* __restrict__ y, int64_t bytes) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at < bytes) y[at] = 0;
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
int64_t code_bytes(int64_t n, int64_t k) { return align256(n * k) + align256(n * (k / kGroup) * 4); }

}  // namespace

hipError_t launch_quantize_act_f8(const void* x, int xt, int64_t n, int64_t k, uint8_t* xq, float* scale,
                                  hipStream_t s) {
  const int64_t groups = n * (k / kGroup);
  log_launch("quantize_act_f8 n=%lld k=%lld", (long long)n, (long long)k);
  return in_pieces(groups, 16, 256, [&](int64_t g0, int64_t c) {
    const dim3 grid(static_cast<unsigned>((c + 15) / 16));
    switch (xt) {
      case QBLK_F32: k_quant_act_f8<QBLK_F32><<<grid, 256, 0, s>>>(x, g0, c, xq, scale); break;
      case QBLK_F16: k_quant_act_f8<QBLK_F16><<<grid, 256, 0, s>>>(x, g0, c, xq, scale); break;
      default: k_quant_act_f8<QBLK_BF16><<<grid, 256, 0, s>>>(x, g0, c, xq, scale); break;
    }
    return hipGetLastError();
  });
}

hipError_t launch_quantize_f8(const void* w, int wt, int64_t rows, int64_t k, uint8_t* codes, float* scale,
                              hipStream_t s) {
  const int64_t blocks = (rows + kGroup - 1) / kGroup * (k / kGroup);
  log_launch("quantize_f8 rows=%lld k=%lld", (long long)rows, (long long)k);
  return in_pieces(blocks, 1, 256, [&](int64_t b0, int64_t c) {
    const dim3 grid(static_cast<unsigned>(c));
    switch (wt) {
      case QBLK_F32: k_quant_f8<QBLK_F32><<<grid, 256, 0, s>>>(w, rows, k, b0, codes, scale); break;
      case QBLK_F16: k_quant_f8<QBLK_F16><<<grid, 256, 0, s>>>(w, rows, k, b0, codes, scale); break;
      default: k_quant_f8<QBLK_BF16><<<grid, 256, 0, s>>>(w, rows, k, b0, codes, scale); break;
    }
    return hipGetLastError();
  });
}

hipError_t launch_zero_bytes(void* y, int64_t bytes, hipStream_t s) {
  return in_pieces(bytes, 256, 256, [&](int64_t b0, int64_t c) {
    k_zero<<<dim3(static_cast<unsigned>((c + 255) / 256)), 256, 0, s>>>(static_cast<uint8_t*>(y) + b0, c);
    return hipGetLastError();
  });
}

// (for either kind of result: the one that splits more decides)
int64_t gemm_f8_workspace(int64_t m, int64_t k, int64_t n) {
  if (n <= kFewTokens) return 0;
  const int a = tile_plan(m, k, n, false, false).splits, b = tile_plan(m, k, n, false, true).splits;
  const int most = a > b ? a : b;
  return most > 1 ? align256(most * n * m * 4) : 0;
}

hipError_t launch_gemm_f8(const uint8_t* w, const float* ws, int64_t m, int64_t k, const uint8_t* xq,
                          const float* xs, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  if (n <= kFewTokens) return few_codes<false>(w, ws, m, k, xq, xs, n, y, yt, 0, s);
  return tile_product(w, ws, m, k, xq, xs, n, y, yt, 0, nullptr, yt == QBLK_F32, work, s);
}

int64_t linear_f8_workspace(int64_t m, int64_t k, int64_t n) {
  if (fused_quant(n, k)) return 0;
  return code_bytes(n, k) + gemm_f8_workspace(m, k, n);
}

hipError_t launch_linear_f8(const uint8_t* w, const float* ws, int64_t m, int64_t k, const void* x, int xt,
                            int64_t n, void* y, int yt, void* work, hipStream_t s) {
  if (fused_quant(n, k)) return few_values<false>(w, ws, m, k, x, xt, n, y, yt, 0, s);
  uint8_t* xq = static_cast<uint8_t*>(work);
  float* xs = reinterpret_cast<float*>(xq + align256(n * k));
  const hipError_t e = launch_quantize_act_f8(x, xt, n, k, xq, xs, s);
  if (e != hipSuccess) return e;
  return launch_gemm_f8(w, ws, m, k, xq, xs, n, y, yt, xq + code_bytes(n, k), s);
}

// ffn workspace: few tokens: h in fp32, then what its two products need, one
// after the other; else the codes of x, those of h, and the second product's
int64_t ffn_f8_workspace(int64_t h, int64_t i, int64_t n) {
  if (n > kFewTokens) return code_bytes(n, h) + code_bytes(n, i) + gemm_f8_workspace(h, i, n);
  const int64_t up = fused_quant(n, h) ? 0 : code_bytes(n, h);
  const int64_t down = linear_f8_workspace(h, i, n);
  return align256(n * i * 4) + (up > down ? up : down);
}

hipError_t launch_ffn_f8(const uint8_t* w13, const float* s13, const uint8_t* w2, const float* s2, int64_t h,
                         int64_t i, const void* x, int xt, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  hipError_t e;
  if (n > kFewTokens) {
    uint8_t* xq = static_cast<uint8_t*>(work);
    float* xs = reinterpret_cast<float*>(xq + align256(n * h));
    uint8_t* hq = xq + code_bytes(n, h);
    float* hs = reinterpret_cast<float*>(hq + align256(n * i));
    e = launch_quantize_act_f8(x, xt, n, h, xq, xs, s);
    // (the codes of h turn on the last bits of the first product: see k_f8_tile)
    if (e == hipSuccess) e = tile_product(w13, s13, 2 * i, h, xq, xs, n, hq, 0, i, hs, yt != QBLK_BF16, nullptr, s);
    if (e != hipSuccess) return e;
    return launch_gemm_f8(w2, s2, h, i, hq, hs, n, y, yt, hq + code_bytes(n, i), s);
  }
  float* mid = static_cast<float*>(work);
  uint8_t* rest = static_cast<uint8_t*>(work) + align256(n * i * 4);
  if (fused_quant(n, h)) {
    e = few_values<true>(w13, s13, 2 * i, h, x, xt, n, mid, QBLK_F32, i, s);
  } else {
    float* xs = reinterpret_cast<float*>(rest + align256(n * h));
    e = launch_quantize_act_f8(x, xt, n, h, rest, xs, s);
    if (e != hipSuccess) return e;
    e = few_codes<true>(w13, s13, 2 * i, h, rest, xs, n, mid, QBLK_F32, i, s);
  }
  if (e != hipSuccess) return e;
  return launch_linear_f8(w2, s2, h, i, mid, QBLK_F32, n, y, yt, rest, s);
}

}  // namespace qblk
