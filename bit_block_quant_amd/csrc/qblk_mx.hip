// qblk_mx.hip -- OCP microscaling formats on gfx950: quantizers, the values that
// codes stand for, and products with MXFP4 weights.
//
//   W[r,c] = 2^ew[r,c/32] * qw[r,c]      e2m1, two to a byte (the even column low)
//   X[t,c] = 2^ex[t,c/32] * qx[t,c]      e2m1 likewise, or e4m3
//   Y[t,r] = sum_b 2^(ex[t,b] + ew[r,b]) sum_{c in b} qw qx
//
// The matrix cores take both scales with the codes: in a K = 128 instruction a
// lane holds 32 columns, which is one block, and its scales.
#include "qblk_mx_device.h"
#include "qblk_mx_tile.h"

namespace qblk {
namespace {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));

// ------------------------------------------------------------ quantizers
// HBM bound: 2 or 4 bytes read and 17/32 or 33/32 written per value.  A lane takes
// 8 values, four lanes a block; a workgroup kQuantUnits times 256 lanes' worth,
// every load before the first use.
constexpr int kQuantUnits = 4;

template <int XT, bool F8>
__global__ __launch_bounds__(256) void k_quant_mx(const void* __restrict__ x, int64_t first, int64_t units,
                                                  uint8_t* __restrict__ codes, uint8_t* __restrict__ scale, int per, int padded) {
  // unit = 8 values; whole quads are on or off together.  padded > 0: rows of `per`
  // units go to rows of `padded` bytes, zeros behind them.
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * (256 * kQuantUnits) + threadIdx.x;
  float v[kQuantUnits][8];
#pragma unroll
  for (int i = 0; i < kQuantUnits; i++) {
    const int64_t u = u0 + 256 * i;
    if (u < units) {
      load8<XT>(x, (first + u) * 8, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) v[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < kQuantUnits; i++) {
    const int64_t u = u0 + 256 * i;
    const uint32_t b = mx_scale<F8>(quad_max(top_bits<8>(v[i])));
    uint32_t c[2];
    mx_codes<F8, 8>(v[i], b, c);
    if (u >= units) continue;
    constexpr int kBytes = F8 ? 8 : 4;
    int64_t at = (first + u) * kBytes;
    if (padded > 0) {
      const int64_t t = (first + u) / per;
      const int in = static_cast<int>(first + u - t * per);
      at = t * padded + in * kBytes;
      if (in < 4)  // the row's first block clears what is behind its last
        for (int b = per * kBytes + in * 4 * kBytes; b < padded; b += 16 * kBytes) {
#pragma unroll
          for (int o = 0; o < 4 * kBytes; o += 16) *reinterpret_cast<u32x4*>(codes + t * padded + b + o) = u32x4{0, 0, 0, 0};
        }
    }
    if constexpr (F8)
      *reinterpret_cast<u32x2*>(codes + at) = u32x2{c[0], c[1]};
    else
      *reinterpret_cast<uint32_t*>(codes + at) = c[0];
    if ((threadIdx.x & 3) == 0) scale[(first + u) / 4] = static_cast<uint8_t>(b);
  }
}

// ------------------------------------------------------------- the values
// HBM bound.  A lane takes 8 values: element times scale in fp32 (exact, but for
// underflow), rounded once to the result's type.
template <int OT, bool F8>
__global__ __launch_bounds__(256) void k_dequant_mx(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scale,
                                                    int64_t first, int64_t units, void* __restrict__ out) {
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * (256 * kQuantUnits) + threadIdx.x;
  uint32_t c[kQuantUnits][2], b[kQuantUnits];
#pragma unroll
  for (int i = 0; i < kQuantUnits; i++) {
    const int64_t u = first + (u0 + 256 * i < units ? u0 + 256 * i : units - 1);
    if constexpr (F8) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(codes + u * 8);
      c[i][0] = w.x;
      c[i][1] = w.y;
    } else {
      c[i][0] = *reinterpret_cast<const uint32_t*>(codes + u * 4);
    }
    b[i] = scale[u / 4];
  }
#pragma unroll
  for (int i = 0; i < kQuantUnits; i++) {
    if (u0 + 256 * i >= units) continue;
    const int64_t at = (first + u0 + 256 * i) * 8;
    const float s = mx_scale_value(b[i]);
    typedef float f2 __attribute__((ext_vector_type(2)));
    f2 p[4];
    if constexpr (F8) {
      p[0] = __builtin_amdgcn_cvt_pk_f32_fp8(c[i][0], false);
      p[1] = __builtin_amdgcn_cvt_pk_f32_fp8(c[i][0], true);
      p[2] = __builtin_amdgcn_cvt_pk_f32_fp8(c[i][1], false);
      p[3] = __builtin_amdgcn_cvt_pk_f32_fp8(c[i][1], true);
    } else {
      p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i][0], 1.0f, 0);
      p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i][0], 1.0f, 1);
      p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i][0], 1.0f, 2);
      p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i][0], 1.0f, 3);
    }
    const float4_t lo = {p[0].x * s, p[0].y * s, p[1].x * s, p[1].y * s};
    const float4_t hi = {p[2].x * s, p[2].y * s, p[3].x * s, p[3].y * s};
    if constexpr (OT == QBLK_F32) {
      float4_t* o = reinterpret_cast<float4_t*>(static_cast<float*>(out) + at);
      o[0] = lo;
      o[1] = hi;
    } else {
      const u32x2 a = bits16(lo, OT), d = bits16(hi, OT);
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + at) = u32x4{a.x, a.y, d.x, d.y};
    }
  }
}

// ------------------------------------------------------------- few tokens
// A workgroup owns NR tiles of 16 rows for 16 T tokens and splits the columns
// over its waves, 256 columns (a group: 128 bytes of a row of W) at a time: wave w
// takes groups w, w + WAVES, ...; the waves' fp32 sums meet in LDS in a fixed
// order.  A load takes 8 rows' 128 bytes, 8 neighbouring lanes a row, and the rows
// change lanes through LDS of the wave's own.  A wave has its next two groups in
// flight, in registers.
//
// EXACT: e4m3 activations with fp32 results.  The e4m3 instructions bring 8
// neighbouring columns' products to the largest one's exponent and drop what is
// below 2^-13 of it, which an fp32 result shows; both operands are widened to
// bf16 with their scales instead (an element times its scale is a bf16 number) and
// multiplied there, where sums are exact to fp32 rounding.  (e2m1 by e2m1: the
// products of a block are whole multiples of 1/4 up to 36 of one scale, and the
// scaled instructions' sums were found equal to fp32 sums of them.)
constexpr int kCols = 256;                  // of a group
constexpr int kGroupBlocks = kCols / kMxBlock;

constexpr int few_region(int T, int NR, bool F8) {
  return T * NR * 1024 > (F8 ? 4096 : 2048) ? T * NR * 1024 : (F8 ? 4096 : 2048);
}

template <int T, int NR, bool F8>
struct FewSet {
  u32x4 w[NR][2], x[T][F8 ? 4 : 2];
  uint64_t sw[NR], sx[T];
};

// 8 bytes of a row's scales from block 8 g on; past the row's end zeros (2^-127)
__device__ __forceinline__ uint64_t scales8(const uint8_t* row, int g, int nb) {
  if (nb >= kGroupBlocks) {
    const int at = g * kGroupBlocks, from = at < nb - kGroupBlocks ? at : nb - kGroupBlocks;
    const u32x2_a1 v = *reinterpret_cast<const u32x2_a1*>(row + from);
    return ((static_cast<uint64_t>(v.y) << 32) | v.x) >> (8 * (at - from));
  }
  uint64_t v = 0;
  for (int j = 0; j < nb; j++) v |= static_cast<uint64_t>(row[j]) << (8 * j);
  return v;
}

__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ int8v regs4(const u32x4& v) {
  return int8v{static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w), 0, 0, 0, 0};
}
__device__ __forceinline__ int8v regs8(const u32x4& a, const u32x4& b) {
  return int8v{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w),
               static_cast<int>(b.x), static_cast<int>(b.y), static_cast<int>(b.z), static_cast<int>(b.w)};
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

struct FewArgs {
  const uint8_t* w;
  const uint8_t* ws;
  const uint8_t* xq;
  const uint8_t* xs;
  void* y;
  int64_t xrow;  // bytes from one token's codes to the next one's
  int m, k, n, yt;
};

template <int T, int NR, int WAVES, bool F8, bool EXACT>
__global__ __launch_bounds__(WAVES* kWave) void k_mx_few(FewArgs p) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int kRegion = few_region(T, NR, F8);
  using Set = FewSet<T, NR, F8>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nb = p.k / kMxBlock, G = (nb + kGroupBlocks - 1) / kGroupBlocks;
  const int row0 = blockIdx.x * 16 * NR, tok0 = blockIdx.y * 16 * T;
  const int r = lane & 15, q = lane >> 4;
  uint8_t* const region = lds + wave * kRegion;
  const int64_t wrow = static_cast<int64_t>(nb) * 16;

  // Rows and tokens past the last repeat it; their results are not stored.
  auto row_at = [&](int row) { return row < p.m ? row : p.m - 1; };
  auto tok_at = [&](int tok) { return tok < p.n ? tok : p.n - 1; };
  auto load = [&](Set& s, int step) {
    int g = wave + step * WAVES;
    if (g > G - 1) g = G - 1;
    // blocks past the row's end repeat its last; x is cleared there
    const int block = g * kGroupBlocks + (lane & 7) < nb ? g * kGroupBlocks + (lane & 7) : nb - 1;
#pragma unroll
    for (int a = 0; a < NR; a++) {
#pragma unroll
      for (int u = 0; u < 2; u++)
        s.w[a][u] = *reinterpret_cast<const u32x4*>(p.w + row_at(row0 + 16 * a + 8 * u + (lane >> 3)) * wrow + block * 16);
      s.sw[a] = scales8(p.ws + static_cast<int64_t>(row_at(row0 + 16 * a + r)) * nb, g, nb);
    }
#pragma unroll
    for (int t = 0; t < T; t++) {
      if constexpr (F8) {
        const int at = g * kCols + 16 * (lane & 15) < p.k ? g * kCols + 16 * (lane & 15) : p.k - 16;
#pragma unroll
        for (int u = 0; u < 4; u++)
          s.x[t][u] = *reinterpret_cast<const u32x4*>(p.xq + tok_at(tok0 + 16 * t + 4 * u + (lane >> 4)) * p.xrow + at);
      } else {
#pragma unroll
        for (int u = 0; u < 2; u++)
          s.x[t][u] = *reinterpret_cast<const u32x4*>(p.xq + tok_at(tok0 + 16 * t + 8 * u + (lane >> 3)) * p.xrow + block * 16);
      }
      s.sx[t] = scales8(p.xs + static_cast<int64_t>(tok_at(tok0 + 16 * t + r)) * nb, g, nb);
    }
  };
  // rows of 128 bytes, by 8 lanes each -> row r, chunks q and q + 4
  auto turn = [&](const u32x4 v[2], u32x4 out[2]) {
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const int row = 8 * u + (lane >> 3);
      *reinterpret_cast<u32x4*>(region + row * 128 + (((lane & 7) ^ ((row >> 1) & 7)) << 4)) = v[u];
    }
    wave_fence();
    const int key = (r >> 1) & 7;
    out[0] = *reinterpret_cast<const u32x4*>(region + r * 128 + ((q ^ key) << 4));
    out[1] = *reinterpret_cast<const u32x4*>(region + r * 128 + (((q + 4) ^ key) << 4));
    wave_fence();
  };
  // rows of 256 bytes, by 16 lanes each -> row r, of either 128 bytes what a lane's
  // operand holds: chunks q and q + 4 (the instruction's order), or its block (EXACT)
  auto turn8 = [&](const u32x4 v[4], u32x4 out[2][2]) {
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const int row = 4 * u + (lane >> 4);
      *reinterpret_cast<u32x4*>(region + row * 256 + (((lane & 15) ^ row) << 4)) = v[u];
    }
    wave_fence();
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int c = 8 * j + (EXACT ? 2 * q + h : q + 4 * h);
        out[j][h] = *reinterpret_cast<const u32x4*>(region + r * 256 + ((c ^ r) << 4));
      }
    wave_fence();
  };

  Set A, B;
  load(A, 0);
  load(B, 1);
  float4_t acc[NR][T];
#pragma unroll
  for (int a = 0; a < NR; a++)
#pragma unroll
    for (int t = 0; t < T; t++) acc[a][t] = float4_t{0, 0, 0, 0};

  auto use = [&](const Set& s, int step) {
    const int g = wave + step * WAVES;
    if (g >= G) return;
    u32x4 wv[NR][2];
    uint32_t sw[NR][2];
#pragma unroll
    for (int a = 0; a < NR; a++) {
      turn(s.w[a], wv[a]);
      sw[a][0] = static_cast<uint32_t>(s.sw[a]) >> (8 * q);
      sw[a][1] = static_cast<uint32_t>(s.sw[a] >> 32) >> (8 * q);
    }
    const int left = nb - g * kGroupBlocks;  // blocks of this group
#pragma unroll
    for (int t = 0; t < T; t++) {
      u32x4 xv[2][2];
      if constexpr (F8) {
        turn8(s.x[t], xv);
      } else {
        u32x4 c[2];
        turn(s.x[t], c);
        xv[0][0] = c[0];
        xv[1][0] = c[1];
      }
      if (left < kGroupBlocks) {
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
          for (int h = 0; h < (F8 ? 2 : 1); h++) {
            const int b = 4 * j + (F8 && !EXACT ? (q >> 1) + 2 * h : q);
            if (b >= left) xv[j][h] = u32x4{0, 0, 0, 0};
          }
      }
      const uint32_t sx[2] = {static_cast<uint32_t>(s.sx[t]) >> (8 * q), static_cast<uint32_t>(s.sx[t] >> 32) >> (8 * q)};
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int a = 0; a < NR; a++) {
          if constexpr (EXACT) {
            const float fw = __builtin_bit_cast(float, (sw[a][j] & 255u) << 23), fx = __builtin_bit_cast(float, (sx[j] & 255u) << 23);
#pragma unroll
            for (int h = 0; h < 2; h++) {
              acc[a][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide4(wv[a][j][2 * h], fw), wide8(xv[j][h].x, xv[j][h].y, fx), acc[a][t], 0, 0, 0);
              acc[a][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide4(wv[a][j][2 * h + 1], fw), wide8(xv[j][h].z, xv[j][h].w, fx), acc[a][t], 0, 0, 0);
            }
          } else if constexpr (F8) {
            acc[a][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(regs4(wv[a][j]), regs8(xv[j][0], xv[j][1]), acc[a][t], 4, 0, 0,
                                                                         static_cast<int>(sw[a][j]), 0, static_cast<int>(sx[j]));
          } else {
            acc[a][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(regs4(wv[a][j]), regs4(xv[j][0]), acc[a][t], 4, 4, 0,
                                                                         static_cast<int>(sw[a][j]), 0, static_cast<int>(sx[j]));
          }
        }
    }
  };

  const int steps = (G + WAVES - 1) / WAVES;
  for (int step = 0; step < steps; step += 2) {
    use(A, step);
    load(A, step + 2);
    use(B, step + 1);
    load(B, step + 3);
  }

  // lane (r, q) holds rows 4q..4q+3 of each tile for token r of each 16
  float4_t* red = reinterpret_cast<float4_t*>(region);
#pragma unroll
  for (int a = 0; a < NR; a++)
#pragma unroll
    for (int t = 0; t < T; t++) red[(a * T + t) * 64 + lane] = acc[a][t];
  __syncthreads();
  const float* rf = reinterpret_cast<const float*>(lds);
  for (int o = threadIdx.x; o < NR * T * 256; o += WAVES * kWave) {
    const int rr = o & 15, tok = (o >> 4) % (16 * T), a = o / (256 * T);
    const int at = ((a * T + (tok >> 4)) * 64 + (rr >> 2) * 16 + (tok & 15)) * 4 + (rr & 3);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < WAVES; v++) sum += rf[v * (kRegion / 4) + at];
    const int row = row0 + 16 * a + rr;
    if (tok0 + tok < p.n && row < p.m) store_y(p.y, static_cast<int64_t>(tok0 + tok) * p.m + row, sum, p.yt);
  }
}

template <int T, int NR, int WAVES, bool F8, bool EXACT>
hipError_t few(const FewArgs& a, hipStream_t s) {
  const size_t lds = static_cast<size_t>(WAVES) * few_region(T, NR, F8);
  log_launch("mx few%s m=%d k=%d n=%d T=%d NR=%d waves=%d%s", F8 ? " f8" : " f4", a.m, a.k, a.n, T, NR, WAVES, EXACT ? " exact" : "");
  k_mx_few<T, NR, WAVES, F8, EXACT>
      <<<dim3(static_cast<unsigned>((a.m + 16 * NR - 1) / (16 * NR)), static_cast<unsigned>((a.n + 16 * T - 1) / (16 * T))), WAVES * kWave, lds, s>>>(a);
  return hipGetLastError();
}

template <int T>
hipError_t few_kind(const FewArgs& a, bool f8, hipStream_t s) {
  if (!f8) return few<T, 1, 8, false, false>(a, s);
  return a.yt == QBLK_F32 ? few<T, 1, 8, true, true>(a, s) : few<T, 1, 8, true, false>(a, s);
}

// in pieces of tokens: at most 65535 workgroups in the grid's second dimension
hipError_t few_product(const FewArgs& all, int64_t n, bool f8, hipStream_t s) {
  return in_pieces(n, 64, 1, [&](int64_t t0, int64_t c) {
    FewArgs a = all;
    a.xq += t0 * all.xrow;
    a.xs += t0 * (all.k / kMxBlock);
    a.y = static_cast<uint8_t*>(a.y) + t0 * a.m * (a.yt == QBLK_F32 ? 4 : 2);
    a.n = static_cast<int>(c);
    return c <= 16 ? few_kind<1>(a, f8, s) : c <= 32 ? few_kind<2>(a, f8, s) : few_kind<4>(a, f8, s);
  }, 65535);
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

// ------------------------------------------------------------- many tokens
// Bytes of a token's codes in whole stages of the tile kernel: 128 each.
int64_t padded_row(int64_t k, bool f8) { return ((f8 ? k : k / 2) + 127) / 128 * 128; }

struct Plan {
  int tokens, splits, per;  // tokens of a tile; stages per split, a multiple of 4
  double us;
};
Plan tile_plan(int64_t m, int64_t k, int64_t n, bool f8) {
  const int64_t rt = (m + kMxTileRows - 1) / kMxTileRows, G = padded_row(k, f8) / 128;
  Plan best{64, 1, static_cast<int>((G + 3) / 4 * 4), 1e30};
  for (int i = 0; i < 3; i++) {
    const int tokens = 64 << i;
    for (int sp = 1; sp <= 16; sp *= 2) {
      const int64_t per = ((G + sp - 1) / sp + 3) / 4 * 4, real = (G + per - 1) / per;
      if (sp > 1 && real < sp) break;
      const int64_t rounds = (rt * ((n + tokens - 1) / tokens) * real + cu_count() - 1) / cu_count();
      constexpr double stage[2][3] = {{0.6, 0.8, 1.2}, {0.4, 0.6, 1.0}};
      const double us = rounds * (per * stage[f8][i] + 4 + i) + (real > 1 ? 2.0 + 0.35e-6 * real * n * m * 4 : 0.0);
      if (us < best.us) best = Plan{tokens, static_cast<int>(real), static_cast<int>(per), us};
    }
  }
  return best;
}

bool use_few(int64_t m, int64_t k, int64_t n, bool f8) { return n <= 32; }

// Rows of x's codes copied into rows of whole stages, zeros behind them: 16 bytes a thread.
__global__ __launch_bounds__(256) void k_mx_pad(const uint8_t* __restrict__ x, int64_t first, int64_t count, int row, int padded,
                                                uint8_t* __restrict__ out) {
  int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= count) return;
  i += first;
  const int per = padded / 16;
  const int64_t t = i / per;
  const int c = 16 * static_cast<int>(i - t * per);
  *reinterpret_cast<u32x4*>(out + 16 * i) = c < row ? *reinterpret_cast<const u32x4*>(x + t * row + c) : u32x4{0, 0, 0, 0};
}

hipError_t pad(const uint8_t* x, int64_t n, int64_t row, int64_t padded, uint8_t* out, hipStream_t s) {
  return in_pieces(n * (padded / 16), 256, 256, [&](int64_t first, int64_t c) {
    k_mx_pad<<<dim3(static_cast<unsigned>((c + 255) / 256)), 256, 0, s>>>(x, first, c, static_cast<int>(row), static_cast<int>(padded), out);
    return hipGetLastError();
  });
}

hipError_t tile_product(const uint8_t* w, const uint8_t* ws, int64_t m, int64_t k, const uint8_t* xq, int64_t xrow,
                        const uint8_t* xs, bool f8, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  const Plan plan = tile_plan(m, k, n, f8);
  uint8_t* rest = static_cast<uint8_t*>(work);
  const int64_t row = padded_row(k, f8);
  if (xrow != row) {
    const hipError_t e = pad(xq, n, xrow, row, rest, s);
    if (e != hipSuccess) return e;
    xq = rest;
    rest += align256(n * row);
  }
  const int64_t rt = (m + kMxTileRows - 1) / kMxTileRows;
  MxTileArgs a{w, ws, xq, xs, y, reinterpret_cast<float*>(rest), row, static_cast<int>(m), static_cast<int>(k), static_cast<int>(n), yt,
               static_cast<int>(rt), static_cast<int>((n + plan.tokens - 1) / plan.tokens), 0, plan.per};
  log_launch("mx tile f%d m=%lld k=%lld n=%lld tokens=%d splits=%d", f8 ? 8 : 4, (long long)m, (long long)k, (long long)n, plan.tokens, plan.splits);
  if (plan.splits > 1) {
    const hipError_t e = mx_tile(plan.tokens, f8, a, plan.splits, s);
    return e == hipSuccess ? launch_join(a.part, m, n, plan.splits, y, yt, s) : e;
  }
  // in pieces of the tokens: a launch of 2^23 tiles would pass 32 bits of threads
  return in_pieces((n + plan.tokens - 1) / plan.tokens, 1, 512 * rt, [&](int64_t tt, int64_t count) {
    const int64_t t0 = tt * plan.tokens, left = n - t0;
    MxTileArgs b = a;
    b.xq += t0 * row;
    b.xs += t0 * (k / kMxBlock);
    b.y = static_cast<uint8_t*>(y) + t0 * m * (yt == QBLK_F32 ? 4 : 2);
    b.n = static_cast<int>(left < count * plan.tokens ? left : count * plan.tokens);
    b.tok_tiles = static_cast<int>(count);
    return mx_tile(plan.tokens, f8, b, 1, s);
  });
}

// Y from codes in rows of xrow bytes, by one kernel or the other
hipError_t product(const uint8_t* w, const uint8_t* ws, int64_t m, int64_t k, const uint8_t* xq, int64_t xrow,
                   const uint8_t* xs, bool f8, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  if (use_few(m, k, n, f8) || (f8 && yt == QBLK_F32))
    return few_product(FewArgs{w, ws, xq, xs, y, xrow, static_cast<int>(m), static_cast<int>(k), 0, yt}, n, f8, s);
  return tile_product(w, ws, m, k, xq, xrow, xs, f8, n, y, yt, work, s);
}

template <bool F8>
hipError_t quantize(const void* x, int xt, int64_t units, uint8_t* codes, uint8_t* scale, int per, int padded, hipStream_t s) {
  return in_pieces(units, 256 * kQuantUnits, 256, [&](int64_t u0, int64_t c) {
    const dim3 grid(static_cast<unsigned>((c + 256 * kQuantUnits - 1) / (256 * kQuantUnits)));
    switch (xt) {
      case QBLK_F32: k_quant_mx<QBLK_F32, F8><<<grid, 256, 0, s>>>(x, u0, c, codes, scale, per, padded); break;
      case QBLK_F16: k_quant_mx<QBLK_F16, F8><<<grid, 256, 0, s>>>(x, u0, c, codes, scale, per, padded); break;
      default: k_quant_mx<QBLK_BF16, F8><<<grid, 256, 0, s>>>(x, u0, c, codes, scale, per, padded); break;
    }
    return hipGetLastError();
  });
}

hipError_t quantize_rows(const void* v, int vt, int64_t rows, int64_t k, bool f8, int64_t row_bytes, uint8_t* codes, uint8_t* scale,
                         hipStream_t s) {
  const int per = static_cast<int>(k / 8), padded = row_bytes == (f8 ? k : k / 2) ? 0 : static_cast<int>(row_bytes);
  return f8 ? quantize<true>(v, vt, rows * per, codes, scale, per, padded, s) : quantize<false>(v, vt, rows * per, codes, scale, per, padded, s);
}

template <bool F8>
hipError_t dequant(const uint8_t* codes, const uint8_t* scale, int64_t units, void* out, int ot, hipStream_t s) {
  return in_pieces(units, 256 * kQuantUnits, 256, [&](int64_t u0, int64_t c) {
    const dim3 grid(static_cast<unsigned>((c + 256 * kQuantUnits - 1) / (256 * kQuantUnits)));
    switch (ot) {
      case QBLK_F32: k_dequant_mx<QBLK_F32, F8><<<grid, 256, 0, s>>>(codes, scale, u0, c, out); break;
      case QBLK_F16: k_dequant_mx<QBLK_F16, F8><<<grid, 256, 0, s>>>(codes, scale, u0, c, out); break;
      default: k_dequant_mx<QBLK_BF16, F8><<<grid, 256, 0, s>>>(codes, scale, u0, c, out); break;
    }
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_quantize_mx(const void* v, int vt, int64_t rows, int64_t k, bool f8, uint8_t* codes, uint8_t* scale,
                              hipStream_t s) {
  log_launch("quantize_mx%d rows=%lld k=%lld", f8 ? 8 : 4, (long long)rows, (long long)k);
  return quantize_rows(v, vt, rows, k, f8, f8 ? k : k / 2, codes, scale, s);
}

hipError_t launch_dequant_mx(const uint8_t* codes, const uint8_t* scale, int64_t rows, int64_t k, bool f8, void* out,
                             int ot, hipStream_t s) {
  log_launch("dequant_mx%d rows=%lld k=%lld", f8 ? 8 : 4, (long long)rows, (long long)k);
  return f8 ? dequant<true>(codes, scale, rows * (k / 8), out, ot, s) : dequant<false>(codes, scale, rows * (k / 8), out, ot, s);
}

int64_t gemm_mxfp4_workspace(int64_t m, int64_t k, int64_t n, bool f8) {
  if (use_few(m, k, n, f8)) return 0;
  const int splits = tile_plan(m, k, n, f8).splits;
  return (padded_row(k, f8) != (f8 ? k : k / 2) ? align256(n * padded_row(k, f8)) : 0) + (splits > 1 ? align256(splits * n * part_pitch(m) * 4) : 0);
}

hipError_t launch_gemm_mxfp4(const uint8_t* w, const uint8_t* ws, int64_t m, int64_t k, const uint8_t* xq,
                             const uint8_t* xs, bool f8, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  return product(w, ws, m, k, xq, f8 ? k : k / 2, xs, f8, n, y, yt, work, s);
}

// Codes of x in rows of whole stages where the tile kernel reads them.
int64_t linear_mxfp4_workspace(int64_t m, int64_t k, int64_t n, bool f8) {
  const bool few = use_few(m, k, n, f8);
  const int splits = few ? 1 : tile_plan(m, k, n, f8).splits;
  return align256(n * (few ? (f8 ? k : k / 2) : padded_row(k, f8))) + align256(n * (k / kMxBlock)) +
         (splits > 1 ? align256(splits * n * part_pitch(m) * 4) : 0);
}

hipError_t launch_linear_mxfp4(const uint8_t* w, const uint8_t* ws, int64_t m, int64_t k, const void* x, int xt,
                               bool f8, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  const bool few = use_few(m, k, n, f8);
  const int64_t row = few ? (f8 ? k : k / 2) : padded_row(k, f8);
  uint8_t* xq = static_cast<uint8_t*>(work);
  uint8_t* xs = xq + align256(n * row);
  const hipError_t e = quantize_rows(x, xt, n, k, f8, row, xq, xs, s);
  if (e != hipSuccess) return e;
  return product(w, ws, m, k, xq, row, xs, f8, n, y, yt, xs + align256(n * (k / kMxBlock)), s);
}

}  // namespace qblk
