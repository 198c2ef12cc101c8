// qblk_mx.hip -- OCP microscaling formats on gfx950: quantizers, the values that
// codes stand for, and products with MXFP4 weights.
//
//   W[r,c] = 2^ew[r,c/32] * qw[r,c]      e2m1, two to a byte (the even column low)
//   X[t,c] = 2^ex[t,c/32] * qx[t,c]      e2m1 likewise, or e4m3
//   Y[t,r] = sum_b 2^(ex[t,b] + ew[r,b]) sum_{c in b} qw qx
//
// The matrix cores take both scales with the codes: in a K = 128 instruction a
// lane holds 32 columns, which is one block, and its scales.
#include "qblk_lds.h"
#include "qblk_mx_device.h"
#include "qblk_mx_tile.h"

namespace qblk {
namespace {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));

// ------------------------------------------------------------ quantizers
// HBM bound: 2 or 4 bytes read and 17/32 or 33/32 written per value.  A lane takes
// 8 values, four lanes a block, each workgroup 2048 values (us, lanes of 8 and of 32: 64 x 4096 bf16
// 2.1, 2.8; 4096 x 11008 to e2m1 21.3, 24.4, 5.5 TB/s; 14336 x 4096 fp32 45.9, 49.1, 5.9 TB/s).
template <int XT, bool F8>
__global__ __launch_bounds__(256) void k_quant_mx(const void* __restrict__ x, int64_t first, int64_t units,
                                                  uint8_t* __restrict__ codes, uint8_t* __restrict__ scale, int per, int padded) {
  // unit = 8 values; whole quads are on or off together.  padded > 0: rows of `per`
  // units go to rows of `padded` bytes, zeros behind them.
  int64_t u = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (u >= units) return;
  u += first;
  float v[8];
  load8<XT>(x, u * 8, v);
  const uint32_t b = mx_scale<F8>(quad_max(top_bits<8>(v)));
  uint32_t c[2];
  mx_codes<F8, 8>(v, b, c);
  constexpr int kBytes = F8 ? 8 : 4;
  int64_t at = u * kBytes;
  if (padded > 0) {
    const int64_t t = u / per;
    const int in = static_cast<int>(u - t * per);
    at = t * padded + in * kBytes;
    if (in < 4)  // the row's first block clears what is behind its last
      for (int z = per * kBytes + in * 4 * kBytes; z < padded; z += 16 * kBytes) {
#pragma unroll
        for (int o = 0; o < 4 * kBytes; o += 16) *reinterpret_cast<u32x4*>(codes + t * padded + z + o) = u32x4{0, 0, 0, 0};
      }
  }
  if constexpr (F8)
    *reinterpret_cast<u32x2*>(codes + at) = u32x2{c[0], c[1]};
  else
    *reinterpret_cast<uint32_t*>(codes + at) = c[0];
  if ((threadIdx.x & 3) == 0) scale[u / 4] = static_cast<uint8_t>(b);
}

// ------------------------------------------------------------- the values
// HBM bound.  A lane takes 8 values: element times scale in fp32 (exact, but for
// underflow), rounded once to the result's type; UNITS times, every load before the first
// use (dequant_units).
template <int OT, bool F8, int UNITS>
__global__ __launch_bounds__(256) void k_dequant_mx(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scale,
                                                    int64_t first, int64_t units, void* __restrict__ out) {
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * (256 * UNITS) + threadIdx.x;
  uint32_t c[UNITS][2], b[UNITS];
#pragma unroll
  for (int i = 0; i < UNITS; i++) {
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
  for (int i = 0; i < UNITS; i++) {
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
// Bound by the weight bytes.  A workgroup of 8 or 16 waves owns a run of rows, 16 at a
// time, for all tokens, and splits the columns over its waves, 256 (a group: 128 bytes
// of a row of W) at a time: wave w takes groups w, w + WAVES, ...; the waves' fp32 sums
// meet in LDS in a fixed order.  x stays in LDS: each wave holds the columns it works on,
// so no wave waits for another before the sums.  The loads of W run on over the ends of
// the 16 rows, in registers: a load takes 8 rows' 128 bytes, 8 neighbouring lanes a row,
// and the rows change lanes through LDS of the wave's own.  A wave has one group in
// flight where 24 waves share a compute unit, two where 16 do (few_shape).  One token, weights
// from memory: 131072 x 4096 56 us, 5.1 TB/s; 22016 x 4096 11.7, 4.1 TB/s; 4096 x 4096 4.8 (a
// launch, x, weights and sums, one round trip each).
//
// EXACT: e4m3 activations with fp32 results.  The e4m3 instructions bring 8
// neighbouring columns' products to the largest one's exponent and drop what is
// below 2^-13 of it, which an fp32 result shows; both operands are widened to
// bf16 with their scales instead (an element times its scale is a bf16 number) and
// multiplied there, where sums are exact to fp32 rounding.  (e2m1 by e2m1: the
// products of a block are whole multiples of 1/4 up to 36 of one scale, and the scaled
// instructions' sums are those of fp32 additions of blocks: exact under one scale, else within 4
// units of 2^-24 of the sum of magnitudes over 4096 columns.)
// XSRC: kCodes, x as codes and scales; else the element type of x, which every
// workgroup quantizes itself (one launch less; for few values, see fused_quant).
constexpr int kCodes = 3;
constexpr int kCols = 256;                  // of a group
constexpr int kGroupBlocks = kCols / kMxBlock;
constexpr int64_t kFewLds = 160 * 1024;

struct FewSet {
  u32x4 w[2];
  uint64_t s;
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

struct FewArgs {
  const uint8_t* w;
  const uint8_t* ws;
  const void* x;  // codes, or values
  const uint8_t* xs;
  void* y;
  int64_t xrow;  // bytes from one token's codes to the next one's
  int m, k, n, yt;
  int rows;  // of a workgroup
};

// What a workgroup keeps in LDS: partial sums of two turns, tiles of W changing lanes, and
// x with its scales.
constexpr int few_sums(int T, int waves) { return 2 * waves * T * 1024; }
constexpr int few_steps(int k, int waves) { return ((k + kCols - 1) / kCols + waves - 1) / waves; }  // groups of a wave
constexpr int few_xrow(bool f8) { return f8 ? kCols : kCols / 2; }
constexpr int64_t few_lds(int T, int waves, int k, int64_t n, bool f8) {
  return few_sums(T, waves) + waves * 2048 + int64_t(waves) * few_steps(k, waves) * n * (few_xrow(f8) + kGroupBlocks);
}

template <int T, int WAVES, bool F8, bool EXACT, int XSRC>
__global__ __launch_bounds__(WAVES* kWave) void k_mx_few(FewArgs p) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int kXRow = few_xrow(F8), kSets = WAVES == 16 ? 2 : 1;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nb = p.k / kMxBlock, G = (nb + kGroupBlocks - 1) / kGroupBlocks;
  const int steps = few_steps(p.k, WAVES);
  const int begin = blockIdx.x * p.rows, end = p.m - begin < p.rows ? p.m : begin + p.rows;
  const int tiles = (end - begin + 15) / 16;
  const int r = lane & 15, q = lane >> 4;
  constexpr int kSums = few_sums(T, WAVES);
  uint8_t* const turn_at = lds + kSums + wave * 2048;
  uint8_t* const xl = lds + kSums + WAVES * 2048 + wave * steps * p.n * kXRow;
  uint8_t* const xsl = lds + kSums + WAVES * 2048 + WAVES * steps * p.n * kXRow + wave * steps * p.n * kGroupBlocks;
  const uint32_t wrow = static_cast<uint32_t>(nb) * 16;

  // The next group of this wave, `lstep` of the 16 rows `ltile`.  Rows past the last
  // repeat it (their results are not stored), blocks past the row's end its last (x is
  // zero there), and so does a wave without a group.
  const int total = tiles * steps;
  int ltile = 0, lstep = 0, loaded = 0;
  const uint32_t whole = static_cast<uint32_t>(lane >> 3) * wrow + 16 * (lane & 7), whole_s = static_cast<uint32_t>(r * nb);
  auto next_load = [&](FewSet& s) {
    if (loaded++ >= total) return;
    int g = wave + lstep * WAVES;
    if (g > G - 1) g = G - 1;
    const int row0 = begin + 16 * ltile, last = end - 1 - row0 < 15 ? end - 1 - row0 : 15, left = nb - g * kGroupBlocks;
    const uint8_t* base = p.w + static_cast<int64_t>(row0) * wrow + static_cast<int64_t>(g) * (kCols / 2);
    uint32_t at[2] = {whole, whole + 8 * wrow}, at_s = whole_s;
    if (last < 15 || left < kGroupBlocks) {
      const int chunk = (lane & 7) < left ? lane & 7 : left - 1;
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const int row = 8 * u + (lane >> 3) < last ? 8 * u + (lane >> 3) : last;
        at[u] = static_cast<uint32_t>(row) * wrow + 16 * chunk;
      }
      at_s = static_cast<uint32_t>((r < last ? r : last) * nb);
    }
#pragma unroll
    for (int u = 0; u < 2; u++) s.w[u] = *reinterpret_cast<const u32x4*>(base + at[u]);
    s.s = scales8(p.ws + static_cast<int64_t>(row0) * nb + at_s, g, nb);
    if (++lstep == steps) {
      lstep = 0;
      ltile++;
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  FewSet S[kSets];
  auto first_loads = [&]() {
#pragma unroll
    for (int i = 0; i < kSets; i++) next_load(S[i]);
  };

  // x: chunk c of token t's group lies at chunk c ^ t & 15 (of 8: c ^ t >> 1 & 7) of its row.
  auto x_place = [&](int step, int t, int c) {
    return xl + (step * p.n + t) * kXRow + ((F8 ? c ^ (t & 15) : c ^ ((t >> 1) & 7)) << 4);
  };
  // Some tokens' part of this wave's group `step` at a time, several in flight; the first
  // of W behind the first of x.
  int xstep = 0, xtok = 0;
  if constexpr (XSRC == kCodes) {
    constexpr int lanes = kXRow / 16, per = 64 / lanes, kAtOnce = 4;  // lanes of a token, tokens of a load
    const uint8_t* xq = static_cast<const uint8_t*>(p.x);
    const int c = lane % lanes;
    for (bool first = true; xstep < steps; first = false) {
      u32x4 v[kAtOnce];
      uint64_t sc[kAtOnce];
      int st[kAtOnce], tk[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; i++) {
        st[i] = xstep;
        tk[i] = xtok + lane / lanes;
        const int g = wave + xstep * WAVES, left = p.k - g * kCols;  // columns of this group
        const bool here = xstep < steps && tk[i] < p.n;
        v[i] = here && c * (F8 ? 16 : 32) < left ? *reinterpret_cast<const u32x4*>(xq + tk[i] * p.xrow + static_cast<int64_t>(g) * kXRow + 16 * c)
                                                 : u32x4{0, 0, 0, 0};
        sc[i] = here && c == 0 && left > 0 ? scales8(p.xs + static_cast<int64_t>(tk[i]) * nb, g, nb) : 0;
        xtok += per;
        if (xtok >= p.n) {
          xtok = 0;
          xstep++;
        }
      }
      if (first) first_loads();
#pragma unroll
      for (int i = 0; i < kAtOnce; i++) {
        if (st[i] >= steps || tk[i] >= p.n) continue;
        *reinterpret_cast<u32x4*>(x_place(st[i], tk[i], c)) = v[i];
        if (c == 0) *reinterpret_cast<uint64_t*>(xsl + (st[i] * p.n + tk[i]) * kGroupBlocks) = sc[i];
      }
    }
  } else {
    constexpr int kAtOnce = 2;  // a token's group by 32 lanes, 8 values each
    const int l = lane & 31;
    for (bool first = true; xstep < steps; first = false) {
      float v[kAtOnce][8];
      int st[kAtOnce], tk[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; i++) {
        int s2[2], t2[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          s2[h] = xstep;
          t2[h] = xtok;
          if (++xtok == p.n) {
            xtok = 0;
            xstep++;
          }
        }
        st[i] = lane < 32 ? s2[0] : s2[1];
        tk[i] = lane < 32 ? t2[0] : t2[1];
        const int col = (wave + st[i] * WAVES) * kCols + 8 * l;
        if (col < p.k) {  // (a group past the steps lies past the columns too)
          load8<XSRC>(p.x, static_cast<int64_t>(tk[i]) * p.k + col, v[i]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; e++) v[i][e] = 0.0f;
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (first) first_loads();
#pragma unroll
      for (int i = 0; i < kAtOnce; i++) {
        const uint32_t b = mx_scale<F8>(quad_max(top_bits<8>(v[i])));
        uint32_t c[2];
        mx_codes<F8, 8>(v[i], b, c);
        if (st[i] >= steps) continue;
        if constexpr (F8)
          *reinterpret_cast<u32x2*>(x_place(st[i], tk[i], l >> 1) + 8 * (l & 1)) = u32x2{c[0], c[1]};
        else
          *reinterpret_cast<uint32_t*>(x_place(st[i], tk[i], l >> 2) + 4 * (l & 3)) = c[0];
        if ((l & 3) == 0) xsl[(st[i] * p.n + tk[i]) * kGroupBlocks + (l >> 2)] = static_cast<uint8_t>(b);
      }
    }
  }
  wave_fence();

  float4_t acc[T];
#pragma unroll
  for (int t = 0; t < T; t++) acc[t] = float4_t{0, 0, 0, 0};
  int tile = 0, step = 0;

  auto use = [&](const FewSet& s) {
    const int g = wave + step * WAVES;
    // rows of 128 bytes, by 8 lanes each -> row r, chunks q and q + 4
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const int row = 8 * u + (lane >> 3);
      *reinterpret_cast<u32x4*>(turn_at + row * 128 + (((lane & 7) ^ ((row >> 1) & 7)) << 4)) = s.w[u];
    }
    wave_fence();
    u32x4 wv[2];
#pragma unroll
    for (int j = 0; j < 2; j++) wv[j] = *reinterpret_cast<const u32x4*>(turn_at + r * 128 + (((q + 4 * j) ^ ((r >> 1) & 7)) << 4));
    const uint32_t sw[2] = {static_cast<uint32_t>(s.s) >> (8 * q), static_cast<uint32_t>(s.s >> 32) >> (8 * q)};
    if (g < G) {
#pragma unroll
      for (int t = 0; t < T; t++) {
        const int tok = 16 * t + r < p.n ? 16 * t + r : p.n - 1;
        const u32x2 sc = *reinterpret_cast<const u32x2*>(xsl + (step * p.n + tok) * kGroupBlocks);
        const uint32_t sx[2] = {sc.x >> (8 * q), sc.y >> (8 * q)};
#pragma unroll
        for (int j = 0; j < 2; j++) {
          if constexpr (EXACT) {
            const float fw = __builtin_bit_cast(float, (sw[j] & 255u) << 23), fx = __builtin_bit_cast(float, (sx[j] & 255u) << 23);
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const u32x4 x = *reinterpret_cast<const u32x4*>(x_place(step, tok, 8 * j + 2 * q + h));
              acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide4(wv[j][2 * h], fw), wide8(x.x, x.y, fx), acc[t], 0, 0, 0);
              acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide4(wv[j][2 * h + 1], fw), wide8(x.z, x.w, fx), acc[t], 0, 0, 0);
            }
          } else if constexpr (F8) {  // the instruction's order of e4m3: 16 columns of each half of the 128
            const u32x4 x0 = *reinterpret_cast<const u32x4*>(x_place(step, tok, 8 * j + q));
            const u32x4 x1 = *reinterpret_cast<const u32x4*>(x_place(step, tok, 8 * j + q + 4));
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(regs4(wv[j]), regs8(x0, x1), acc[t], 4, 0, 0,
                                                                     static_cast<int>(sw[j]), 0, static_cast<int>(sx[j]));
          } else {
            const u32x4 x = *reinterpret_cast<const u32x4*>(x_place(step, tok, 4 * j + q));
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(regs4(wv[j]), regs4(x), acc[t], 4, 4, 0,
                                                                     static_cast<int>(sw[j]), 0, static_cast<int>(sx[j]));
          }
        }
      }
    }
    wave_fence();  // (the tile's place is written again)
    if (++step < steps) return;
    // The waves' sums, in turns of two places: one barrier a tile.  Lane (r, q) holds rows
    // 4 q .. 4 q + 3 for token r of each 16.
    step = 0;
    uint8_t* const sums = lds + (tile & 1) * (kSums / 2);
#pragma unroll
    for (int t = 0; t < T; t++) {
      *reinterpret_cast<float4_t*>(sums + ((wave * T + t) * 64 + lane) * 16) = acc[t];
      acc[t] = float4_t{0, 0, 0, 0};
    }
    // as __syncthreads, but the loads stay under way
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const float* rf = reinterpret_cast<const float*>(sums);
    for (int o = threadIdx.x; o < T * 256; o += WAVES * kWave) {
      const int rr = o & 15, tok = o >> 4;
      const int at = ((tok >> 4) * 64 + (rr >> 2) * 16 + (tok & 15)) * 4 + (rr & 3);
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < WAVES; v++) sum += rf[v * (T * 256) + at];
      const int row = begin + 16 * tile + rr;
      if (tok < p.n && row < end) store_y(p.y, static_cast<int64_t>(tok) * p.m + row, sum, p.yt);
    }
    tile++;
  };

  for (int it = 0; it < total; it += kSets) {
#pragma unroll
    for (int i = 0; i < kSets; i++) {
      if (it + i >= total) break;
      use(S[i]);
      next_load(S[i]);
    }
  }
}

// Waves of a workgroup, and workgroups that share a compute unit.  16 waves and two
// groups in flight each where there is one workgroup for a unit (x leaves no room for
// another, or the row tiles do not suffice) and groups for as many waves; else 8 waves,
// up to three workgroups.  Us, 8 and 16 waves, weights from memory: 4096 x 14336, one
// token 13.6, 10.6; 22016 x 4096, 16 tokens 21.6, 17.6; but 22016 x 4096, one token 12.3,
// 15.5; 11008 x 4096, one token 8.5, 9.4; 700 x 1024 3.0, 3.8.  Three workgroups and two:
// 14336 x 4096, 4 tokens 11.2, 9.9 (in turns 6 and 4), 22016 x 4096 12.2, 15 (6 and 6).
struct FewShape {
  int waves, per_cu;
};
template <int T>
FewShape few_shape(int64_t m, int k, int64_t n, bool f8) {
  const int64_t lds = few_lds(T, 8, k, n, f8), tiles = (m + 15) / 16;
  const int per_cu = T == 1 && lds <= 53 * 1024 ? 3 : lds <= 80 * 1024 ? 2 : 1;
  const bool room = few_lds(T, 16, k, n, f8) <= kFewLds, one = tiles <= cu_count() || per_cu == 1 || (per_cu == 2 && tiles <= 3 * cu_count());
  if (room && one && k > 8 * kCols) return FewShape{16, 1};
  // three workgroups' turns of 16 rows, or two's where those leave much less undone
  auto turns = [&](int64_t per) { return per * ((tiles + per * cu_count() - 1) / (per * cu_count())); };
  return FewShape{8, per_cu == 3 && tiles > 3 * cu_count() && 5 * turns(2) < 4 * turns(3) ? 2 : per_cu};
}

template <int T, int WAVES, bool F8, bool EXACT, int XSRC>
hipError_t few_go(FewArgs a, int per_cu, hipStream_t s) {
  const size_t lds = static_cast<size_t>(few_lds(T, WAVES, a.k, a.n, F8));
  static std::atomic<uint64_t> done{0};
  const hipError_t allowed = allow_lds(done, reinterpret_cast<const void*>(k_mx_few<T, WAVES, F8, EXACT, XSRC>), kFewLds);
  if (allowed != hipSuccess) return allowed;
  const int64_t most = static_cast<int64_t>(cu_count()) * per_cu, tiles = (static_cast<int64_t>(a.m) + 15) / 16;
  a.rows = static_cast<int>(tiles <= most ? 16 : (a.m + most - 1) / most);
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.m) + a.rows - 1) / a.rows);
  log_launch("mx few%s m=%d k=%d n=%d T=%d waves=%d rows=%d x=%d%s lds=%zu", F8 ? " f8" : " f4", a.m, a.k, a.n, T, WAVES, a.rows, XSRC,
             EXACT ? " exact" : "", lds);
  k_mx_few<T, WAVES, F8, EXACT, XSRC><<<dim3(grid), WAVES * kWave, lds, s>>>(a);
  return hipGetLastError();
}

template <int T, bool F8, bool EXACT, int XSRC>
hipError_t few(const FewArgs& a, hipStream_t s) {
  const FewShape f = few_shape<T>(a.m, a.k, a.n, F8);
  return f.waves == 16 ? few_go<T, 16, F8, EXACT, XSRC>(a, f.per_cu, s) : few_go<T, 8, F8, EXACT, XSRC>(a, f.per_cu, s);
}

template <int T, int XSRC>
hipError_t few_kind(const FewArgs& a, bool f8, hipStream_t s) {
  if (!f8) return few<T, false, false, XSRC>(a, s);
  return a.yt == QBLK_F32 ? few<T, true, true, XSRC>(a, s) : few<T, true, false, XSRC>(a, s);
}

// Tokens of one launch: what fits into LDS with x.
int64_t few_tokens(int64_t k, bool f8) {
  for (int T = f8 ? 1 : 2; T >= 1; T /= 2)
    if (few_lds(T, 8, static_cast<int>(k), 16 * T, f8) <= kFewLds) return 16 * T;
  int64_t n = 15;
  while (n > 0 && few_lds(1, 8, static_cast<int>(k), n, f8) > kFewLds) n--;
  return n;
}

// x as codes; at most few_tokens of them
hipError_t few_product(const FewArgs& a, bool f8, hipStream_t s) {
  return a.n <= 16 ? few_kind<1, kCodes>(a, f8, s) : few<2, false, false, kCodes>(a, s);  // (e2m1 only: use_few)
}

// Whether a product quantizes its x inside every workgroup: that saves a launch, but each
// of them does it again, up to 8 tokens where they are few (us, in two launches and in one,
// e4m3: 4096 x 4096, 1 token 6.6, 4.8, 4 tokens 6.6, 5.4, 8 tokens 7.6, 6.9; 2048 x 2048, 8
// tokens 5.7, 4.5, 16 tokens 6.7, 6.9; 22016 x 4096, 1 token 14.6, 11.7, 8 tokens 17.3, 18.9;
// 4096 x 14336, 4 tokens 12.3, 13.7).  Such an x always fits into LDS.
bool fused_quant(int64_t m, int64_t n, int64_t k) {
  return n * k <= 32768 && (n <= 4 || (n <= 8 && (m + 15) / 16 <= cu_count()));
}

hipError_t fused_product(const FewArgs& a, int xt, bool f8, hipStream_t s) {
  switch (xt) {
    case QBLK_F32: return few_kind<1, QBLK_F32>(a, f8, s);
    case QBLK_F16: return few_kind<1, QBLK_F16>(a, f8, s);
    default: return few_kind<1, QBLK_BF16>(a, f8, s);
  }
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

// ------------------------------------------------------------- many tokens
// Bytes of a token's codes in whole stages of the tile kernel: 128 each.
int64_t padded_row(int64_t k, bool f8) { return ((f8 ? k : k / 2) + 127) / 128 * 128; }

struct Plan {
  int shape, splits, per;  // of kMxTiles; stages per split, a multiple of 4
  double us;
};

constexpr int kShapes = sizeof(kMxTiles) / sizeof(kMxTiles[0]);
// 256 x 128 is e4m3's alone: of e2m1 it was the best at none of the products below.
constexpr bool has_shape(int shape, bool f8) { return f8 || shape != 1; }

// The time of a shape is estimated from what was measured for it, us: a stage of a
// workgroup that has a compute unit to itself or (the small tiles, `both`) shares it,
// the rest of a workgroup's time, and of a split its join.  Fitted to 2300 times of 90
// products of either kind (9 matrices, 20 to 3000 tokens, every shape, 1 to 16
// splits, weights from memory): the choice is 0.5% (e2m1) and 1.6% (e4m3) behind the best
// form on average, at worst 18% (11008 x 4096, 160 tokens: 22.5 us for 19.1).  More tokens lie
// outside the fit (14336 x 4096, 4096 tokens, e2m1: a round of 256 x 256 takes 36 us for an estimated 29).
double tile_us(int64_t tiles, int shape, int64_t per, int64_t splits, int64_t out, bool f8, int64_t cus) {
  constexpr double both[2][6] = {{1.68, 1.27, 0.72, 1.16, 0.91, 0.59}, {1.28, 0.76, 0.575, 0.85, 0.60, 0.46}};
  constexpr double alone[2][3] = {{0.61, 0.505, 0.39}, {0.505, 0.34, 0.29}};
  constexpr double ends[2][6] = {{2.4, 2.2, 3.45, 2.1, 1.7, 1.0}, {0.8, 1.7, 2.7, 1.1, 1.2, 0.7}};
  constexpr double launch[2] = {2.1, 2.9}, join[2] = {3.25, 2.9}, join_byte[2] = {0.37e-6, 0.38e-6};
  const int64_t rounds = (tiles * splits + cus - 1) / cus;
  const double one = per * (shape >= 3 ? alone[f8][shape - 3] : both[f8][shape]) + ends[f8][shape], two = per * both[f8][shape] + ends[f8][shape];
  const double work = shape >= 3 ? (rounds / 2) * two + (rounds % 2) * one : rounds * one;
  return launch[f8] + work + (splits > 1 ? join[f8] + join_byte[f8] * splits * out * 4 : 0.0);
}
int64_t tiles_of(int64_t m, int64_t n, int shape) {
  return ((m + kMxTiles[shape].rows - 1) / kMxTiles[shape].rows) * ((n + kMxTiles[shape].tokens - 1) / kMxTiles[shape].tokens);
}
Plan tile_plan(int64_t m, int64_t k, int64_t n, bool f8) {
  const int64_t G = padded_row(k, f8) / 128, cus = cu_count();
  Plan best{0, 1, static_cast<int>((G + 3) / 4 * 4), 1e30};
  for (int i = 0; i < kShapes; i++) {
    if (!has_shape(i, f8)) continue;
    const int64_t tiles = tiles_of(m, n, i);
    for (int want = 1; want <= 16; want++) {
      if (want > 1 && (tiles * want > 2 * cus || 4 * want >= G + 4)) break;  // (splits are for tiles that leave units idle)
      const int64_t per = ((G + want - 1) / want + 3) / 4 * 4;
      if ((want - 1) * per >= G) continue;  // as many as fewer splits
      const double us = tile_us(tiles, i, want == 1 ? G : per, want, n * m, f8, cus);
      if (us < best.us) best = Plan{i, want, static_cast<int>(per), us};
    }
  }
  return best;
}

// Exact sums of e4m3 activations: two shapes, whose stages take twice the time.
Plan exact_plan(int64_t m, int64_t k, int64_t n) {
  const int64_t G = padded_row(k, true) / 128, cus = cu_count();
  Plan best{1, 1, static_cast<int>((G + 3) / 4 * 4), 1e30};
  for (int i = 1; i < 5; i += 3)
    for (int want = 1; want <= 16; want++) {
      const int64_t tiles = tiles_of(m, n, i);
      if (want > 1 && (tiles * want > 2 * cus || 4 * want >= G + 4)) break;
      const int64_t per = ((G + want - 1) / want + 3) / 4 * 4;
      if ((want - 1) * per >= G) continue;
      const double us = tile_us(tiles, i, 2 * (want == 1 ? G : per), want, n * m, true, cus);
      if (us < best.us) best = Plan{i, want, static_cast<int>(per), us};
    }
  return best;
}
// The splits that room is kept for: of either kind of result.
int most_splits(int64_t m, int64_t k, int64_t n, bool f8) {
  const int a = tile_plan(m, k, n, f8).splits, b = f8 ? exact_plan(m, k, n).splits : 1;
  return a > b ? a : b;
}

// Where an unsplit product's tiles leave much of their last round of compute units
// empty: the row tiles that fill whole rounds with one shape, and a second launch of the
// other rows with another.
struct Cut {
  int64_t rows;  // of the first launch; 0: do not cut
  int shape, rest;
};
Cut tile_cut(const Plan& plan, int64_t m, int64_t k, int64_t n, bool f8) {
  Cut best{0, 0, 0};
  if (plan.splits > 1) return best;
  const int64_t G = padded_row(k, f8) / 128, cus = cu_count();
  double us = plan.us;
  for (int i = 0; i < 2; i++) {
    if (!has_shape(i, f8)) continue;
    const int64_t rt = (m + 255) / 256, wide = (n + kMxTiles[i].tokens - 1) / kMxTiles[i].tokens;
    const int64_t rows = rt * wide / cus * cus / wide;
    if (rows <= 0 || rows >= rt) continue;
    for (int rest = i; rest < kShapes; rest++) {
      if (!has_shape(rest, f8)) continue;
      const double c = tile_us(rows * wide, i, G, 1, 0, f8, cus) + tile_us(tiles_of(m - rows * 256, n, rest), rest, G, 1, 0, f8, cus);
      if (c < us) {
        us = c;
        best = Cut{rows * 256, i, rest};
      }
    }
  }
  return best;
}

// Whether a product runs k_mx_few: up to 16 tokens, where x leaves room for 16 waves (with
// 8 alone on a unit the loads in flight are too few) and the rows make few turns of 16 a
// workgroup; up to 28 tokens where there is one turn.  Us, few and tiles: 8192 x 8192,
// e4m3, 8 tokens 12.7, 13.9, 12 tokens (no room) 18.9, 14.1; 22016 x 4096, e2m1, 8 tokens
// 12.5, 13.5, 16 tokens 15.2, 14.0; 11008 x 4096, 16 tokens 9.5, 10.0; 128256 x 4096, 2
// tokens 55.9, 52.5, e4m3 56.4, 56.4, 8 tokens 62.1, 58.6; 4096 x 4096, e2m1, 28 tokens
// 6.8, 7.9, 32 8.2, 8.0; e4m3, 20 tokens 8.6, 8.8.  Exact sums, whose tiles take twice the
// time: wherever the codes fit (8192 x 8192, 8 tokens 14.4, 18.9, 12 tokens 20.7, 18.9; 128256
// x 4096, 8 tokens 68.5, 76.2; 4096 x 14336, 8 tokens 19.1, 19.3).
bool use_few(int64_t m, int64_t k, int64_t n, bool f8, bool exact) {
  if (n > few_tokens(k, f8)) return false;
  if (exact) return n <= 16;
  const int64_t turns = ((m + 15) / 16 + cu_count() - 1) / cu_count();
  if (few_lds(n > 16 ? 2 : 1, 16, static_cast<int>(k), n, f8) > kFewLds) return false;
  if (n > 16) return !f8 && n <= 28 && turns == 1;
  return turns <= (n > 8 ? 4 : 6) || (f8 && n <= 4);
}

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
  const bool exact = f8 && yt == QBLK_F32;
  const Plan plan = exact ? exact_plan(m, k, n) : tile_plan(m, k, n, f8);
  uint8_t* rest = static_cast<uint8_t*>(work);
  const int64_t row = padded_row(k, f8);
  if (xrow != row) {
    const hipError_t e = pad(xq, n, xrow, row, rest, s);
    if (e != hipSuccess) return e;
    xq = rest;
    rest += align256(n * row);
  }
  MxTileArgs a{w, ws, xq, xs, y, reinterpret_cast<float*>(rest), row, static_cast<int>(m), static_cast<int>(k), static_cast<int>(n), yt,
               0, 0, 0, plan.per};
  // the rows [first, first + rows), `first` a multiple of the shape's
  auto whole = [&](int shape, int64_t first, int64_t rows) {
    const MxTile tile = kMxTiles[shape];
    a.first_row_tile = static_cast<int>(first / tile.rows);
    a.row_tiles = static_cast<int>((rows + tile.rows - 1) / tile.rows);
    // in pieces of the tokens: a launch of 2^23 tiles would pass 32 bits of threads
    return in_pieces((n + tile.tokens - 1) / tile.tokens, 1, 512 * static_cast<int64_t>(a.row_tiles), [&](int64_t tt, int64_t count) {
      const int64_t t0 = tt * tile.tokens, left = n - t0;
      MxTileArgs b = a;
      b.xq += t0 * row;
      b.xs += t0 * (k / kMxBlock);
      b.y = static_cast<uint8_t*>(y) + t0 * m * (yt == QBLK_F32 ? 4 : 2);
      b.n = static_cast<int>(left < count * tile.tokens ? left : count * tile.tokens);
      b.tok_tiles = static_cast<int>(count);
      return exact ? mx_tile_exact(shape, b, 1, s) : mx_tile(shape, f8, b, 1, s);
    });
  };
  if (plan.splits == 1) {
    const Cut cut = exact ? Cut{0, 0, 0} : tile_cut(plan, m, k, n, f8);
    if (cut.rows == 0) return whole(plan.shape, 0, m);
    const hipError_t e = whole(cut.shape, 0, cut.rows);
    return e == hipSuccess ? whole(cut.rest, cut.rows, m - cut.rows) : e;
  }
  const MxTile tile = kMxTiles[plan.shape];
  a.row_tiles = static_cast<int>((m + tile.rows - 1) / tile.rows);
  a.tok_tiles = static_cast<int>((n + tile.tokens - 1) / tile.tokens);
  const hipError_t e = exact ? mx_tile_exact(plan.shape, a, plan.splits, s) : mx_tile(plan.shape, f8, a, plan.splits, s);
  return e == hipSuccess ? launch_join(a.part, m, n, plan.splits, y, yt, s) : e;
}

// Y from codes in rows of xrow bytes, by one kernel or the other
hipError_t product(const uint8_t* w, const uint8_t* ws, int64_t m, int64_t k, const uint8_t* xq, int64_t xrow,
                   const uint8_t* xs, bool f8, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  if (use_few(m, k, n, f8, f8 && yt == QBLK_F32))
    return few_product(FewArgs{w, ws, xq, xs, y, xrow, static_cast<int>(m), static_cast<int>(k), static_cast<int>(n), yt, 0}, f8, s);
  return tile_product(w, ws, m, k, xq, xrow, xs, f8, n, y, yt, work, s);
}

template <bool F8>
hipError_t quantize(const void* x, int xt, int64_t units, uint8_t* codes, uint8_t* scale, int per, int padded, hipStream_t s) {
  return in_pieces(units, 256, 256, [&](int64_t u0, int64_t c) {
    const dim3 grid(static_cast<unsigned>((c + 255) / 256));
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

template <int OT, bool F8, int UNITS>
hipError_t dequant_go(const uint8_t* codes, const uint8_t* scale, int64_t units, void* out, hipStream_t s) {
  return in_pieces(units, 256 * UNITS, 256, [&](int64_t u0, int64_t c) {
    k_dequant_mx<OT, F8, UNITS><<<dim3(static_cast<unsigned>((c + 256 * UNITS - 1) / (256 * UNITS))), 256, 0, s>>>(codes, scale, u0, c, out);
    return hipGetLastError();
  });
}
// Four units a lane for much that is written in 16 bits (us, one and four: 14336 x 4096 e2m1
// to bf16 35.2, 29.6, e4m3 34.1, 33.0; 4096 x 4096 8.8, 9.0; 64 x 4096 2.1, 3.1; to fp32
// 52.1, 62.8 and 53.7, 68.5, 5.1 TB/s).
template <int OT, bool F8>
hipError_t dequant_units(const uint8_t* codes, const uint8_t* scale, int64_t units, void* out, hipStream_t s) {
  if constexpr (OT != QBLK_F32)
    if (units > int64_t(1) << 21) return dequant_go<OT, F8, 4>(codes, scale, units, out, s);
  return dequant_go<OT, F8, 1>(codes, scale, units, out, s);
}
template <bool F8>
hipError_t dequant(const uint8_t* codes, const uint8_t* scale, int64_t units, void* out, int ot, hipStream_t s) {
  switch (ot) {
    case QBLK_F32: return dequant_units<QBLK_F32, F8>(codes, scale, units, out, s);
    case QBLK_F16: return dequant_units<QBLK_F16, F8>(codes, scale, units, out, s);
    default: return dequant_units<QBLK_BF16, F8>(codes, scale, units, out, s);
  }
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

// Room for either kind of result (what has exact sums runs k_mx_few wherever others do).
int64_t gemm_mxfp4_workspace(int64_t m, int64_t k, int64_t n, bool f8) {
  if (use_few(m, k, n, f8, false)) return 0;
  const int splits = most_splits(m, k, n, f8);
  return (padded_row(k, f8) != (f8 ? k : k / 2) ? align256(n * padded_row(k, f8)) : 0) + (splits > 1 ? align256(splits * n * part_pitch(m) * 4) : 0);
}

hipError_t launch_gemm_mxfp4(const uint8_t* w, const uint8_t* ws, int64_t m, int64_t k, const uint8_t* xq,
                             const uint8_t* xs, bool f8, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  return product(w, ws, m, k, xq, f8 ? k : k / 2, xs, f8, n, y, yt, work, s);
}

// Codes of x in rows of whole stages where the tile kernel reads them.
int64_t linear_mxfp4_workspace(int64_t m, int64_t k, int64_t n, bool f8) {
  if (fused_quant(m, n, k)) return 0;
  const bool few = use_few(m, k, n, f8, false);
  const int splits = few ? 1 : most_splits(m, k, n, f8);
  return align256(n * (few ? (f8 ? k : k / 2) : padded_row(k, f8))) + align256(n * (k / kMxBlock)) +
         (splits > 1 ? align256(splits * n * part_pitch(m) * 4) : 0);
}

hipError_t launch_linear_mxfp4(const uint8_t* w, const uint8_t* ws, int64_t m, int64_t k, const void* x, int xt,
                               bool f8, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  if (fused_quant(m, n, k))
    return fused_product(FewArgs{w, ws, x, nullptr, y, 0, static_cast<int>(m), static_cast<int>(k), static_cast<int>(n), yt, 0}, xt, f8, s);
  const bool few = use_few(m, k, n, f8, f8 && yt == QBLK_F32);
  const int64_t row = few ? (f8 ? k : k / 2) : padded_row(k, f8);
  uint8_t* xq = static_cast<uint8_t*>(work);
  uint8_t* xs = xq + align256(n * row);
  const hipError_t e = quantize_rows(x, xt, n, k, f8, row, xq, xs, s);
  if (e != hipSuccess) return e;
  return product(w, ws, m, k, xq, row, xs, f8, n, y, yt, xs + align256(n * (k / kMxBlock)), s);
}

}  // namespace qblk
