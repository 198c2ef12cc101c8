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
#include "qblk_lds.h"
#include "qblk_quant_device.h"

namespace qblk {
namespace {

// ------------------------------------------------------ activation codes
// HBM bound: 2 or 4 bytes read and 1 + 1/32 written per value; 16 lanes to a
// group, so a wave reads 1 KB (16-bit input) of consecutive values at once.
// 4096 x 4096 bf16: 10.9 us, 4.7 TB/s; 4096 x 11008 26.8, 5.05; up to some hundred
// groups 2.5 us, a launch.
// The scales go out token by token, or (per > 0, the groups of a token) group
// by group, as k_f8_few reads them with neighbouring lanes.
template <int XT>
__global__ __launch_bounds__(256) void k_quant_act_f8(const void* __restrict__ x, int64_t group0, int64_t groups,
                                                      uint8_t* __restrict__ xq, float* __restrict__ scale, int per,
                                                      int tokens) {
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
    if (l == 0) {
      int64_t at = g;
      if (per > 0) {  // few tokens: g fits 32 bits
        const uint32_t t = static_cast<uint32_t>(g) / static_cast<uint32_t>(per);
        at = static_cast<int64_t>(static_cast<uint32_t>(g) - t * per) * tokens + t;
      }
      scale[at] = s;
    }
  }
}

// ---------------------------------------------------------- weight codes
// One workgroup per 128 x 128 block; a thread holds 64 of its values in
// registers between the maximum and the codes, so the block is read once.  HBM
// bound: 4096 x 11008 bf16 34.6 us, 3.9 TB/s of the copy's 5.2, fp32 50.0, 4.5 (a
// block's stores wait for the last of its loads); 1000 x 1152 6 us.
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
      for (int i = 0; i < 8; i++) a = max_nan(a, __builtin_fabsf(v[j][i]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[j][i] = 0.0f;
    }
  }
  a = row16_max(a);
  a = max_nan(a, __shfl_xor(a, 16, kWave));
  a = max_nan(a, __shfl_xor(a, 32, kWave));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
  __syncthreads();
  a = max_nan(max_nan(part[0], part[1]), max_nan(part[2], part[3]));
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

// n <= 16 T tokens, bound by the weight bytes.  A workgroup owns NR tiles of
// 16 rows for all tokens and splits the columns over its waves (wave w
// takes groups w, w + WAVES, ...); the waves' fp32 partial sums meet in LDS in
// a fixed order.  The codes are widened to bf16 and multiplied on the bf16
// matrix cores, whose fp32 sums of such products are exact to fp32 rounding
// (those of the fp8 matrix instructions are not, see k_f8_tile); with so few
// tokens the widening and the matrix work hide behind the weight stream.
//
// A load takes 8 rows of a group's 128 codes, 8 neighbouring lanes a row: the
// vector cache counts an access per 64 bytes of neighbouring lanes, 16 for
// these against 64 where every lane reads its own row, which held 32 tokens to
// half the memory's rate.  The rows change lanes through 2 KB of LDS of the
// wave's own (its LDS operations stay in order, so the next tile may follow at
// once); both operands are read in the same order.  A wave has the operands of
// its next two groups in flight, in registers: each set is loaded again where
// it has just been used.
//
// Measured: 4096 x 11008, weights from memory, 13 tokens 15.0 us (3.0 TB/s of
// weights), 32 tokens 20.4; in the Infinity Cache 11.2 and 15.3 (13.5 and 20.4 before
// the rows were loaded by neighbouring lanes); gate and up of 11008 x 4096, one
// token, 20.4 us (4.4 TB/s).  What is left is the start and the end of a workgroup,
// which one or two rounds of workgroups do not hide, and of x codes through the
// vector cache two bytes for each byte of weights with 32 tokens, four with 64.
//
// GATE: the tiles are 16 gate rows and the 16 up rows i further on; the
// result is h = silu(gate) * up in fp32 (n x i).
// XSRC: kCodes = x given as codes and scales (token t's of group g at
// t * xs_tok + g * xs_group); else the element type of x, which the workgroup
// quantizes into LDS itself (one launch less; every workgroup repeats it, so
// only for few values, see launch_linear_f8).
constexpr int kCodes = 3;

// What a wave keeps in LDS: an operand's tile while it changes lanes, then its
// partial sums.
constexpr int few_region(int T, int NR) { return T * NR < 2 ? 2048 : T * NR * 1024; }

template <int T, int NR, int XT>  // XT = T where x comes as codes, else 1 (unused)
struct FewSet {
  u32x4 w[NR][2], x[XT][2];
  float sw[NR], sx[XT];
};

template <int T, int NR, int WAVES, bool GATE, int XSRC>
__global__ __launch_bounds__(WAVES* kWave) void k_f8_few(const uint8_t* __restrict__ w, const float* __restrict__ ws,
                                                         int m, int k, const void* __restrict__ xv,
                                                         const float* __restrict__ xs, int xs_tok, int xs_group,
                                                         int n, void* __restrict__ y, int yt, int64_t up_row) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr bool CODES = XSRC == kCodes;
  constexpr int kRegion = few_region(T, NR);
  using Set = FewSet<T, NR, CODES ? T : 1>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = k / kGroup;
  const int row0 = blockIdx.x * (GATE ? 16 : 16 * NR);
  const int r = lane & 15, q = lane >> 4;
  uint8_t* const region = lds + wave * kRegion;

  // Rows and tokens past the last repeat it; their results are not stored.
  int zero;  // in a vector register, so that the scales come with the codes and in their order
  asm("v_mov_b32 %0, 0" : "=v"(zero));
  const uint8_t* wb[NR];
  const float* sp[NR];
  uint32_t wo[NR][2], xo[CODES ? T : 1][2], xso[CODES ? T : 1];
#pragma unroll
  for (int a = 0; a < NR; a++) {
    const int64_t base = GATE ? row0 + a * up_row : row0 + 16 * a;
    const int64_t first = GATE || base < m ? base : m - 1;
    const int last = GATE || m - first > 15 ? 15 : static_cast<int>(m - 1 - first);
    wb[a] = w + first * k;
    sp[a] = ws + first / kGroup * G;
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const int row = 8 * u + (lane >> 3) < last ? 8 * u + (lane >> 3) : last;
      wo[a][u] = static_cast<uint32_t>(row) * static_cast<uint32_t>(k) + 16 * (lane & 7);
    }
  }
  const uint8_t* xb = static_cast<const uint8_t*>(xv);
  if constexpr (CODES) {
#pragma unroll
    for (int t = 0; t < T; t++) {
#pragma unroll
      for (int u = 0; u < 2; u++) {
        const int tok = 16 * t + 8 * u + (lane >> 3);
        xo[t][u] = static_cast<uint32_t>(tok < n ? tok : n - 1) * static_cast<uint32_t>(k) + 16 * (lane & 7);
      }
      xso[t] = static_cast<uint32_t>(16 * t + r < n ? 16 * t + r : n - 1) * static_cast<uint32_t>(xs_tok);
    }
  }
  auto load = [&](Set& s, int step) {
    int g = wave + step * WAVES;
    if (g > G - 1) g = G - 1;
    const int64_t at = static_cast<int64_t>(g) * kGroup;
#pragma unroll
    for (int a = 0; a < NR; a++) {
#pragma unroll
      for (int u = 0; u < 2; u++) s.w[a][u] = *reinterpret_cast<const u32x4*>(wb[a] + at + wo[a][u]);
      s.sw[a] = sp[a][g + zero];
    }
    if constexpr (CODES) {
#pragma unroll
      for (int t = 0; t < T; t++) {
#pragma unroll
        for (int u = 0; u < 2; u++) s.x[t][u] = *reinterpret_cast<const u32x4*>(xb + at + xo[t][u]);
        s.sx[t] = xs[static_cast<int64_t>(g) * xs_group + xso[t]];
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // row l >> 3 (and 8 further), chunk l & 7 -> row r, chunks q and q + 4
  auto turn = [&](const u32x4 v[2], u32x4 out[2]) {
#pragma unroll
    for (int u = 0; u < 2; u++) {
      const int row = 8 * u + (lane >> 3);
      *reinterpret_cast<u32x4*>(region + row * kGroup + (((lane & 7) ^ ((row >> 1) & 7)) << 4)) = v[u];
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const int key = (r >> 1) & 7;
    out[0] = *reinterpret_cast<const u32x4*>(region + r * kGroup + ((q ^ key) << 4));
    out[1] = *reinterpret_cast<const u32x4*>(region + r * kGroup + (((q + 4) ^ key) << 4));
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };

  Set A, B;
  const uint8_t* xq = nullptr;
  const float* sl = nullptr;
  const int xstride = k + 16;
  if constexpr (!CODES) {
    float* const scales = reinterpret_cast<float*>(lds + WAVES * kRegion);
    uint8_t* const codes = lds + WAVES * kRegion + (n * G * 4 + 15) / 16 * 16;
    xq = codes;
    sl = scales;
    const int units = n * G;
    for (int u0 = 0; u0 < units; u0 += WAVES * 8) {  // two groups a row of 16 lanes
      float v[2][8];
      int unit[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        unit[i] = u0 + i * WAVES * 4 + (threadIdx.x >> 4);
        const int uu = unit[i] < units ? unit[i] : units - 1;
        load8<XSRC>(xv, uu * kGroup + 8 * r, v[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (u0 == 0) {
        load(A, 0);
        load(B, 1);
      }
#pragma unroll
      for (int i = 0; i < 2; i++) {
        uint32_t c[2];
        const float s = quant_group(v[i], c);
        if (unit[i] < units) {
          const int t = unit[i] / G, g = unit[i] - t * G;
          *reinterpret_cast<u32x2*>(codes + t * xstride + g * kGroup + 8 * r) = u32x2{c[0], c[1]};
          if (r == 0) scales[unit[i]] = s;
        }
      }
    }
    __syncthreads();
  } else {
    load(A, 0);
    load(B, 1);
  }

  float4_t acc[NR][T];
#pragma unroll
  for (int a = 0; a < NR; a++)
#pragma unroll
    for (int t = 0; t < T; t++) acc[a][t] = float4_t{0, 0, 0, 0};

  auto use = [&](const Set& s, int step) {
    const bool on = wave + step * WAVES < G;
    const int g = on ? wave + step * WAVES : G - 1;
    bf16x8_n wv[NR][4];
#pragma unroll
    for (int a = 0; a < NR; a++) {
      u32x4 c[2];
      turn(s.w[a], c);
#pragma unroll
      for (int j = 0; j < 2; j++) {
        wv[a][2 * j] = widen8(c[j].x, c[j].y);
        wv[a][2 * j + 1] = widen8(c[j].z, c[j].w);
      }
    }
#pragma unroll
    for (int t = 0; t < T; t++) {
      u32x4 c[2];
      float sx;
      if constexpr (CODES) {
        turn(s.x[t], c);
        sx = s.sx[t];
      } else {
        const int tok = 16 * t + r < n ? 16 * t + r : n - 1;
        const uint8_t* at = xq + tok * xstride + g * kGroup + 16 * q;
        c[0] = *reinterpret_cast<const u32x4*>(at);
        c[1] = *reinterpret_cast<const u32x4*>(at + 64);
        sx = sl[tok * G + g];
      }
      bf16x8_n xw[4];
#pragma unroll
      for (int j = 0; j < 2; j++) {
        xw[2 * j] = widen8(c[j].x, c[j].y);
        xw[2 * j + 1] = widen8(c[j].z, c[j].w);
      }
#pragma unroll
      for (int a = 0; a < NR; a++) {
        float4_t p = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; j++) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[a][j], xw[j], p, 0, 0, 0);
        const float sc = on ? sx * s.sw[a] : 0.0f;  // a group past the last repeats that one
#pragma unroll
        for (int i = 0; i < 4; i++) acc[a][t][i] = __builtin_fmaf(p[i], sc, acc[a][t][i]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
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
  const int tiles = GATE ? 1 : NR;
  for (int o = threadIdx.x; o < tiles * T * 256; o += WAVES * kWave) {
    const int rr = o & 15, tok = (o >> 4) % (16 * T), a = o / (256 * T);
    const int at = ((a * T + (tok >> 4)) * 64 + (rr >> 2) * 16 + (tok & 15)) * 4 + (rr & 3);
    float sum = 0.0f, up = 0.0f;
#pragma unroll
    for (int v = 0; v < WAVES; v++) {
      sum += rf[v * (kRegion / 4) + at];
      if constexpr (GATE) up += rf[v * (kRegion / 4) + T * 256 + at];
    }
    if (tok >= n) continue;
    const int row = row0 + 16 * a + rr;
    if constexpr (GATE)
      static_cast<float*>(y)[tok * up_row + row] = silu_mul(sum, up);
    else if (row < m)
      store_y(y, static_cast<int64_t>(tok) * m + row, sum, yt);
  }
}

// ------------------------------------------------------------ many tokens
// Bound by the matrix cores.  A workgroup of 8 waves owns 256 rows x 64 NT
// tokens; a group of 128 columns is one stage in LDS (32 KB + 8 NT KB, see
// kStages) and one K=128 fp8 matrix instruction per 16 x 16 tile, whose result
// is scaled by sx[t,g] * sw[r,g] into the fp32 accumulators: four multiply-adds
// per lane beside 32 matrix-core cycles.  Waves are 2 (rows) x 4 (tokens);
// wave row a holds rows 64a..64a+63 of the tile's first and second 128-row
// halves, so that for GATE, where the halves are 128 gate rows and their 128
// up rows, a lane holds both factors of silu(gate) * up.
//
// Measured (the product alone, in a graph, operands from memory): m = n = k = 8192
// 454 us, 2.4 PFLOP/s; 4096 x 14336 x 4096 233 us, 2.1; 1501 x 4096 x 11008 86 us, 1.6
// (74 with the operands in the Infinity Cache); 128 x 4096 x 4096 18.2 us.  Exact sums:
// 4096 x 14336 x 4096 457 us, 1.05 PFLOP/s, 1501 x 4096 x 11008 144.  Of 8192^3 the
// kernel without its copies takes 80%, without its products 85%.
//
// Rounding.  The fp8 instructions add fp32, except that they bring the products of
// 8 neighbouring columns to the largest one's exponent and drop what lies below
// 2^-13 of it (beside a product of 2^16 one of 8 counts and one of 4 does not; in
// the next 8 columns one of 2^-7 does).  A product has 8 significant bits: those
// within 2^-6 of the largest lose nothing, any other less than 2^-13 of it, so a
// result is off by at most 7 * 2^-13 of the largest product of each 8 columns (49 of
// 65536, 2^-10.4, seen).  In the 2-norm, 2048 x 4096 with 300 tokens: 1.4e-5 of the
// result on normal data, 7.2e-5 with 1% of the channels 1000 times the others,
// beside 2.0e-4 of rounding to f16 and 1.65e-3 to bf16.  An fp32 result would show
// it; and where the result is quantized again (the gated layer, 2048/4096) it moves
// codes to the neighbouring one, which is 9.8e-4 to 2.3e-3 of that layer's result on
// the same data: f16 shows it (1.0e-3 to 2.3e-3 instead of 2.1e-4 to 2.2e-4), bf16
// less (1.9e-3 to 2.9e-3 instead of 1.66e-3).  EXACT widens the codes to bf16 and
// multiplies those, at half the rate: products and sums are then exact to fp32
// rounding.  It is taken for fp32 results and for the first
// product of a gated layer with an fp16 or fp32 result.
//
// LDS layout.  The stages are filled by loads straight to LDS, which write what
// 64 lanes load to 64 x 16 consecutive bytes: 8 whole rows of 128 bytes.  The
// banks are spread by where the loads' KBs lie, 32 bytes apart, each with every
// eighth row of 64: row 16 t + r is row 2 t + (r >> 3 ^ r >> 2 & 1) of KB r & 7.
// The 16 rows of an operand then start at 8 of the 16 columns of banks, and the
// two quarters that one phase of a read takes (8 rows of each) lie next to one
// another; every operand is at a constant distance from a lane's place.  (The 16-
// byte chunks of a row exchanged instead: as few conflicts, 1-3% slower at 4096
// tokens.)
typedef int int8v __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void glob_void;

constexpr int kTileRows = 256;

// 64 rows of a stage: see above.
constexpr int kSlice = 8 * kGroup + 32, kBlock64 = 8 * kSlice;
template <int NT>
struct Stage {
  uint8_t a[kTileRows / 64 * kBlock64];
  uint8_t b[NT * kBlock64];
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

// A group's operands of 16-row tile `tile`: lane (row r, quarter q), whose place
// in a tile is `at`, gives the row's chunks q and q + 4 (both sides in the same
// order).  EXACT: widened to bf16.
template <bool EXACT>
struct Frag;
template <>
struct Frag<false> {
  int8v v;
  __device__ __forceinline__ void load(const uint8_t* base, int tile, int at) {
    const uint8_t* p = base + (tile >> 2) * kBlock64 + (tile & 3) * 2 * kGroup + at;
    const u32x4 lo = *reinterpret_cast<const u32x4*>(p);
    const u32x4 hi = *reinterpret_cast<const u32x4*>(p + kGroup / 2);
    v = int8v{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
              static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
  }
};
template <>
struct Frag<true> {
  bf16x8_n v[4];
  __device__ __forceinline__ void load(const uint8_t* base, int tile, int at) {
    const uint8_t* p = base + (tile >> 2) * kBlock64 + (tile & 3) * 2 * kGroup + at;
    const u32x4 lo = *reinterpret_cast<const u32x4*>(p);
    const u32x4 hi = *reinterpret_cast<const u32x4*>(p + kGroup / 2);
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
  float* part;    // split K: partial sums, [split][n][part_pitch(m)]
  int m, k, n, yt, up, row_tiles, tok_tiles, groups_per_split, first_row_tile;
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
  const int in_rt = in_band / wide, tt = 8 * band + in_band - in_rt * wide, rt = p.first_row_tile + in_rt;
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
  // this lane's row of 64
  const int row64 = 16 * (lane >> 4) + 8 * (((lane >> 3) ^ (wave >> 2)) & 1) + wave;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int row = 64 * i + row64;
    int at = GATE ? row & 127 : row;
    if (!GATE && at > p.m - 1 - row0) at = p.m - 1 - row0;
    ao[i] = static_cast<uint32_t>(at) * static_cast<uint32_t>(p.k) + ((lane & 7) << 4);
  }
#pragma unroll
  for (int i = 0; i < NT; i++) {
    const int row = 64 * i + row64;
    const int at = t0 + row < p.n ? row : p.n - 1 - t0;
    bo[i] = static_cast<uint32_t>(at) * static_cast<uint32_t>(p.k) + ((lane & 7) << 4);
  }
  // chunk i of 4 + NT: the rows of A, then those of B
  auto copy = [&](Stage<NT>& s, int g, int i) {
    const int64_t at = static_cast<int64_t>(g) * kGroup;
    if (i < 4)
      __builtin_amdgcn_global_load_lds((glob_void*)((i < 2 ? abase[0] : abase[1]) + at + ao[i & 3]),
                                       (lds_void*)(s.a + i * kBlock64 + wave * kSlice), 16, 0, 0);
    else if (i < 4 + NT)
      __builtin_amdgcn_global_load_lds((glob_void*)(bbase + at + bo[i - 4]),
                                       (lds_void*)(s.b + (i - 4) * kBlock64 + wave * kSlice), 16, 0, 0);
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
  // tile i, the operand of tile i + 2 is read from LDS and tile i - 1 is scaled.
  // Across stages: before the last two row tiles every operand of the stage is
  // in registers, so one barrier there frees its buffer for the copies of a
  // later stage and shows the next stage's, whose first operands are read
  // behind the matrix instructions of those two.
  Frag<EXACT> bf[NT], af[4];
  float4_t c[2][NT];
  float sc[2][NT];
  auto atile = [&](int i) { return (i >> 2) * 8 + wm * 4 + (i & 3); };
  const int place = (r & 7) * kSlice + (((r >> 3) ^ (r >> 2)) & 1) * kGroup + 16 * q;
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
  constexpr int kEarly = kStages<NT> == 2 ? 4 : 2;  // copies that go out behind the barrier
  auto group_at = [&](int step) { return g0 + step < g1 ? g0 + step : g1 - 1; };
#pragma unroll
  for (int e = 0; e < kEarly; e++) copy(st[kAhead], group_at(kAhead), e);
  af[0].load(st[0].a, atile(0), place);
  af[1].load(st[0].a, atile(1), place);
#pragma unroll
  for (int j = 0; j < NT; j++) bf[j].load(st[0].b, wn * NT + j, place);
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
      if (i < 6) {
        af[(i + 2) & 3].load(cur.a, atile(i + 2), place);
      } else if (i == 6) {
        if constexpr (kStages<NT> == 2) {
          __syncthreads();
        } else {
          // as __syncthreads, but leaving the newest 4 + NT loads under way: the
          // copies of the stage after next (all older ones are the next stage's)
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
          __builtin_amdgcn_s_waitcnt(0x0070 | (4 + NT));  // vmcnt(4 + NT) lgkmcnt(0)
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
        __builtin_amdgcn_sched_barrier(0);
        af[0].load(nxt.a, atile(0), place);
#pragma unroll
        for (int e = 0; e < kEarly / 2; e++) copy(cur, gc, e);
      } else {
        af[1].load(nxt.a, atile(1), place);
#pragma unroll
        for (int e = kEarly / 2; e < kEarly; e++) copy(cur, gc, e);
      }
#pragma unroll
      for (int j = 0; j < NT; j++) {
        c[i & 1][j] = group_product(af[i & 3], bf[j]);
        if (i > 0) scale(i - 1, j);
        if (i == 7) bf[j].load(nxt.b, wn * NT + j, place);
      }
      // Each matrix instruction with the four multiply-adds of a finished tile
      // behind it; the LDS reads after the first (before it they would be
      // waited for together with the operand it needs).  The copies are spread,
      // two a row tile: all at once they hold up the waves' issue (m = n = k =
      // 8192: 454 us; four a tile 512, one a tile 492), and with three stages
      // the first ones one a tile (m = 4096, k = 11008, n = 1501, operands in the
      // Infinity Cache: 72 and 74 us).
      if (i < 3) {
        copy(far, gf, kEarly + 2 * i);
        copy(far, gf, kEarly + 2 * i + 1);
      }
#pragma unroll
      for (int j = 0; j < NT && !EXACT; j++) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (j == 0 || i == 7) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        if (j < 2) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
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
          a = max_nan(a, __builtin_fabsf(acc[i][j][e]));
        }
      a = max_nan(a, __shfl_xor(a, 16, kWave));
      top[j] = max_nan(a, __shfl_xor(a, 32, kWave));
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
      const float s = max_nan(m2[in], m2[64 * NT + in]) / kF8Max;
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
        if constexpr (SPLIT) {  // rows of partial sums lie 16-byte aligned
          float* part = p.part + (static_cast<int64_t>(blockIdx.y) * p.n + tok) * part_pitch(p.m) + row;
          *reinterpret_cast<float4_t*>(part) = acc[i][j];
          continue;
        }
        const int64_t at = static_cast<int64_t>(tok) * p.m + row;
        const bool whole = row + 4 <= p.m;
        if (p.yt == QBLK_F32) {
          float* y = static_cast<float*>(p.y);
          if (whole) {
            *reinterpret_cast<float4_a4*>(y + at) = acc[i][j];
          } else {
#pragma unroll
            for (int e = 0; e < 4; e++)
              if (row + e < p.m) y[at + e] = acc[i][j][e];
          }
        } else {
          const u32x2 h = bits16(acc[i][j], p.yt);
          uint16_t* y = static_cast<uint16_t*>(p.y) + at;
          if (whole) {
            *reinterpret_cast<u32x2_a2*>(y) = h;
          } else {
#pragma unroll
            for (int e = 0; e < 4; e++)
              if (row + e < p.m) y[e] = static_cast<uint16_t>(h[e >> 1] >> (16 * (e & 1)));
          }
        }
      }
    }
  }
}

// y = the sum of the splits' partial products, in their order: a thread takes 4
// rows of a token.  Bound by the partial sums' bytes: 4 splits of 333 x 5003 in
// 6.2 us, 4.8 TB/s with y.
__global__ __launch_bounds__(256) void k_f8_join(const float* __restrict__ part, int64_t first, int64_t count, int m,
                                                 int64_t stride, int splits, void* __restrict__ y, int yt) {
  int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= count) return;
  i += first;
  const uint32_t chunks = static_cast<uint32_t>(part_pitch(m) / 4);
  const int64_t tok = i / chunks;
  const int row = 4 * static_cast<int>(i - tok * chunks);
  const float* p = part + 4 * i;
  float4_t v = *reinterpret_cast<const float4_t*>(p);
  for (int s = 1; s < splits; s++) {
    const float4_t o = *reinterpret_cast<const float4_t*>(p + s * stride);
#pragma unroll
    for (int e = 0; e < 4; e++) v[e] += o[e];
  }
  const int64_t at = tok * m + row;
  if (row + 4 <= m) {
    if (yt == QBLK_F32)
      *reinterpret_cast<float4_a4*>(static_cast<float*>(y) + at) = v;
    else
      *reinterpret_cast<u32x2_a2*>(static_cast<uint16_t*>(y) + at) = bits16(v, yt);
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (row + e < m) store_y(y, at + e, v[e], yt);
  }
}

// The codes and scales of H = silu(gate) * up from the splits' partial products
// of the rows [gate; up]: 16 lanes to a group of 128, like k_quant_act_f8.
// Group g's scale of token t goes to t * s_tok + g * s_group.
__global__ __launch_bounds__(256) void k_f8_join_gate(const float* __restrict__ part, int64_t stride, int splits,
                                                      int inter, int64_t groups, uint8_t* __restrict__ hq,
                                                      float* __restrict__ hs, int64_t s_tok, int64_t s_group) {
  const int64_t all = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  const bool on = all < groups;
  const int64_t u = on ? all : groups - 1;  // whole waves take part in the row reductions
  const int per = inter / kGroup, l = threadIdx.x & 15;
  const int64_t t = u / per;
  const int g = static_cast<int>(u - t * per);
  const float* p = part + t * 2 * inter + g * kGroup + 8 * l;
  float gate[8], up[8];
#pragma unroll
  for (int i = 0; i < 8; i++) gate[i] = up[i] = 0.0f;
  for (int s = 0; s < splits; s++, p += stride) {
    float a[8], b[8];
    load8<QBLK_F32>(p, 0, a);
    load8<QBLK_F32>(p, inter, b);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      gate[i] += a[i];
      up[i] += b[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; i++) gate[i] = silu_mul(gate[i], up[i]);
  uint32_t code[2];
  const float s = quant_group(gate, code);
  if (on) {
    *reinterpret_cast<u32x2*>(hq + u * kGroup + 8 * l) = u32x2{code[0], code[1]};
    if (l == 0) hs[t * s_tok + g * s_group] = s;
  }
}

// What a few-tokens product takes besides its matrix: x as values, or as codes
// with scales at the given strides.
struct FewX {
  const void* x;
  int xt;
  const float* xs;
  int64_t xs_tok, xs_group;
};

template <int T, int NR, int WAVES, bool GATE, int XSRC>
hipError_t few(const uint8_t* w, const float* ws, int64_t m, int64_t k, const FewX& x, int64_t n, void* y, int yt,
               int64_t up_row, hipStream_t s) {
  const int per = GATE ? 16 : 16 * NR;
  const int64_t rows = GATE ? up_row : m;
  const dim3 grid(static_cast<unsigned>((rows + per - 1) / per));
  const size_t G = static_cast<size_t>(k / kGroup);
  const size_t lds = static_cast<size_t>(WAVES) * few_region(T, NR) +
                     (XSRC == kCodes ? 0 : (n * G * 4 + 15) / 16 * 16 + n * (static_cast<size_t>(k) + 16));
  static std::atomic<uint64_t> done{0};
  const hipError_t allowed = allow_lds(done, reinterpret_cast<const void*>(k_f8_few<T, NR, WAVES, GATE, XSRC>), 128 * 1024);
  if (allowed != hipSuccess) return allowed;
  log_launch("f8 few%s rows=%lld k=%lld n=%lld T=%d NR=%d waves=%d x=%d lds=%zu", GATE ? " gate" : "", (long long)m,
             (long long)k, (long long)n, T, NR, WAVES, XSRC, lds);
  k_f8_few<T, NR, WAVES, GATE, XSRC><<<grid, WAVES * kWave, lds, s>>>(
      w, ws, static_cast<int>(m), static_cast<int>(k), x.x, x.xs, static_cast<int>(x.xs_tok),
      static_cast<int>(x.xs_group), static_cast<int>(n), y, yt, up_row);
  return hipGetLastError();
}

template <int NR, int WAVES, bool GATE>
hipError_t few_src(const uint8_t* w, const float* ws, int64_t m, int64_t k, const FewX& x, int64_t n, void* y, int yt,
                   int64_t up_row, hipStream_t s) {
  switch (x.xt) {
    case QBLK_F32: return few<1, NR, WAVES, GATE, QBLK_F32>(w, ws, m, k, x, n, y, yt, up_row, s);
    case QBLK_F16: return few<1, NR, WAVES, GATE, QBLK_F16>(w, ws, m, k, x, n, y, yt, up_row, s);
    case QBLK_BF16: return few<1, NR, WAVES, GATE, QBLK_BF16>(w, ws, m, k, x, n, y, yt, up_row, s);
  }
  if (n <= 16) return few<1, NR, WAVES, GATE, kCodes>(w, ws, m, k, x, n, y, yt, up_row, s);
  if (n <= 32) return few<2, NR, WAVES, GATE, kCodes>(w, ws, m, k, x, n, y, yt, up_row, s);
  // (16 waves have 128 registers each, too few for these tokens' sets)
  return few<4, NR, 8, GATE, kCodes>(w, ws, m, k, x, n, y, yt, up_row, s);
}

// Y = W X^T (or, for up_row > 0, H) by k_f8_few.  With no more row tiles than
// compute units one workgroup is all that a unit gets: 16 waves then, if 8 had
// more than four groups each or more than one round of x to quantize (m = 4096,
// us, 16 and 8 waves: k = 11008, n = 1: 13.2 and 14.6; k = 4096, n = 4: 6.5 and
// 7.4; but n = 1: 6.3 and 5.8).  With more rows 8 (m = 22016, k = 4096, n = 4
// as codes: 23.0, with 16 28.6).
hipError_t few_product(const uint8_t* w, const float* ws, int64_t m, int64_t k, const FewX& x, int64_t n, void* y,
                       int yt, int64_t up_row, hipStream_t s) {
  if (up_row > 0) return few_src<2, 8, true>(w, ws, m, k, x, n, y, yt, up_row, s);
  const int64_t G = k / kGroup;
  if ((m + 15) / 16 <= cu_count() && (G > 32 || (x.xt != kCodes && n * G > 64)))
    return few_src<1, 16, false>(w, ws, m, k, x, n, y, yt, 0, s);
  return few_src<1, 8, false>(w, ws, m, k, x, n, y, yt, 0, s);
}

// The tile kernel's shape for a product: tokens per tile and splits of K.
struct Plan {
  int nt, splits, per;  // 64 nt tokens; groups per split
  double us;            // the estimate by which it was taken
};

// The time of each shape is estimated from what was measured for the kernel's
// variants (us: a stage of a tile, then the rest of a tile's time, for 64, 128
// and 256 tokens) and the least taken.  (A gated product's split tiles leave gate
// and up apart in the partial sums, and the join forms h.)  A split is worth its
// join where tiles leave compute units without work: m = k = 4096, n = 128:
// 64-token tiles unsplit 29.0 us, split by 4 18.2; n = 1024: 28.9 against 59.8.  Wide
// tiles pay with many tokens: m = 14336, k = 4096, n = 4096: 64 tokens 390 us, 128
// 278, 256 249; n = 512: 58, 40, 65.  Over 108 products (6 matrices, 20 to 4096
// tokens, both kinds of sums, weights from memory) the choice is more than 3% behind
// the best form four times, 14% at worst (m = k = 4096, n = 100), and level with it
// on average.
double tile_us(int64_t row_tiles, int64_t n, int nt, int64_t splits, int64_t groups, bool exact) {
  constexpr double stage[2][3] = {{0.66, 0.8, 1.5}, {1.15, 1.6, 0}}, ends[2][3] = {{5, 8, 9}, {5, 7, 0}};
  const int64_t rounds = (row_tiles * ((n + 64 * nt - 1) / (64 * nt)) * splits + cu_count() - 1) / cu_count();
  return rounds * (groups * stage[exact][nt >> 1] + ends[exact][nt >> 1]);
}
Plan tile_plan(int64_t m, int64_t k, int64_t n, bool exact) {
  const int64_t rt = (m + kTileRows - 1) / kTileRows, G = k / kGroup;
  Plan best{1, 1, static_cast<int>(G), 1e30};
  for (int nt = 1; nt <= (exact ? 2 : 4); nt *= 2)
    for (int sp = 1; sp <= 8; sp *= 2) {
      if (sp > 1 && G / sp < 4) break;
      const int64_t per = (G + sp - 1) / sp;
      const double c = tile_us(rt, n, nt, sp, per, exact) + (sp > 1 ? 2.0 + 0.35e-6 * sp * n * m * 4 : 0.0);
      if (c < best.us) best = Plan{nt, sp, static_cast<int>(per), c};
    }
  best.splits = static_cast<int>((G + best.per - 1) / best.per);
  return best;
}

// Where an unsplit product's tiles leave most of their last round of compute
// units empty: the row tiles that fill whole rounds with `nt`, and a second
// launch of the rest with narrower tiles (`rest_nt`).  Us, cut and whole: m =
// 22016, k = 4096, n = 1501 (516 wide tiles) 158 and 178; m = 5003, k = 11008, n =
// 4096 227 and 260; m = 14336, k = 4096, n = 4096 235 and 249; exact sums, m = 22016,
// k = 4096, n = 512 108 and 121.
struct Cut {
  int64_t rows;  // row tiles of the first launch; 0: do not cut
  int nt, rest_nt;
};
Cut tile_cut(const Plan& plan, int64_t m, int64_t k, int64_t n, bool exact) {
  Cut best{0, 0, 0};
  if (plan.splits > 1) return best;
  const int64_t rt = (m + kTileRows - 1) / kTileRows, G = k / kGroup;
  double us = plan.us;
  for (int nt = 1; nt <= (exact ? 2 : 4); nt *= 2) {
    const int64_t wide = (n + 64 * nt - 1) / (64 * nt), rounds = rt * wide / cu_count(), rows = rounds * cu_count() / wide;
    if (rows <= 0 || rows >= rt) continue;
    for (int rest = 1; rest <= nt; rest *= 2) {
      const double c = tile_us(rows, n, nt, 1, G, exact) + tile_us(rt - rows, n, rest, 1, G, exact) + 3.0;
      if (c < us) {
        us = c;
        best = Cut{rows, nt, rest};
      }
    }
  }
  return best;
}

template <int NT, bool GATE, bool SPLIT, bool EXACT>
hipError_t tile_go(const TileArgs& a, int splits, hipStream_t s) {
  constexpr size_t lds = sizeof(TileLds<NT>);
  static std::atomic<uint64_t> done{0};
  const hipError_t allowed = allow_lds(done, reinterpret_cast<const void*>(k_f8_tile<NT, GATE, SPLIT, EXACT>), lds);
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

// Where the scales of codes go or are: token t's of group g at t * tok + g * group.
struct ScaleAt {
  int64_t tok, group;
};

// Y (or, for `up` > 0, the codes and scales of H) by the tile kernel
hipError_t tile_product(const uint8_t* w, const float* ws, int64_t m, int64_t k, const uint8_t* xq, const float* xs,
                        int64_t n, void* y, int yt, int64_t up, float* hs, ScaleAt at, bool exact, void* work,
                        hipStream_t s) {
  const Plan plan = tile_plan(m, k, n, exact);
  const bool split = plan.splits > 1;
  TileArgs a{w, ws, xq, xs, y, hs, static_cast<float*>(work), static_cast<int>(m), static_cast<int>(k), static_cast<int>(n), yt,
             static_cast<int>(split ? 0 : up), static_cast<int>((m + kTileRows - 1) / kTileRows),
             static_cast<int>((n + 64 * plan.nt - 1) / (64 * plan.nt)), plan.per, 0};
  log_launch("f8 tile%s%s m=%lld k=%lld n=%lld tokens=%d splits=%d", up > 0 ? " gate" : "", exact ? " exact" : "",
             (long long)m, (long long)k, (long long)n, 64 * plan.nt, plan.splits);
  auto whole = [&](int nt, int64_t first, int64_t rows) {
    a.first_row_tile = static_cast<int>(first);
    a.row_tiles = static_cast<int>(rows);
    // in pieces of the tokens: a launch of 2^23 tiles would pass 32 bits of threads
    return in_pieces((n + 64 * nt - 1) / (64 * nt), 1, 512 * rows, [&](int64_t tt, int64_t count) {
      const int64_t t0 = tt * 64 * nt, left = n - t0;
      TileArgs b = a;
      b.xq += t0 * k;
      b.xs += t0 * (k / kGroup);
      b.y = static_cast<uint8_t*>(y) + t0 * (up > 0 ? up : m * (yt == QBLK_F32 ? 4 : 2));
      if (up > 0) b.hs += t0 * (up / kGroup);
      b.n = static_cast<int>(left < count * 64 * nt ? left : count * 64 * nt);
      b.tok_tiles = static_cast<int>(count);
      return up > 0 ? tile_nt<true, false>(nt, exact, b, 1, s) : tile_nt<false, false>(nt, exact, b, 1, s);
    });
  };
  if (!split) {
    const int64_t rt = a.row_tiles;
    const Cut cut = tile_cut(plan, m, k, n, exact);
    if (cut.rows == 0) return whole(plan.nt, 0, rt);
    log_launch("  cut: %lld row tiles, tokens=%d, then tokens=%d", (long long)cut.rows, 64 * cut.nt, 64 * cut.rest_nt);
    const hipError_t e = whole(cut.nt, 0, cut.rows);
    return e == hipSuccess ? whole(cut.rest_nt, cut.rows, rt - cut.rows) : e;
  }
  const hipError_t e = tile_nt<false, true>(plan.nt, exact, a, plan.splits, s);
  if (e != hipSuccess) return e;
  if (up > 0) {  // (one launch: only a product of few tiles is split)
    const int64_t groups = n * (up / kGroup);
    k_f8_join_gate<<<dim3(static_cast<unsigned>((groups + 15) / 16)), 256, 0, s>>>(
        a.part, m * n, plan.splits, static_cast<int>(up), groups, static_cast<uint8_t*>(y), hs, at.tok, at.group);
    return hipGetLastError();
  }
  return launch_join(a.part, m, n, plan.splits, y, yt, s);
}

// Products of up to this many tokens are exact to fp32 rounding.
constexpr int64_t kExactTokens = 64;

// Whether a product runs k_f8_few: up to 16 tokens always (one operand of x per
// 16 rows); up to 64 where its estimate is below the tile kernel's.  It keeps all
// compute units busy with few rows, but reads x again for every 16 of them
// (us, few and tiles: 32 tokens, m = k = 4096: 9.1, 15.2; m = 8192, k = 8192:
// 25.9, 23.4; m = 22016, k = 4096: 38.8, 30.3; m = 4096, k = 11008: 20.7, 23.7; 64
// tokens: 13.7, 18.6; 43.1, 26.3; 72.8, 33.1; 29.3, 25.0).
bool use_few(int64_t m, int64_t k, int64_t n) {
  if (n <= 16 || n > kExactTokens) return n <= 16;
  const double rate = n > 32 ? 0.68e-6 : (m + 15) / 16 <= cu_count() ? 0.28e-6 : 0.36e-6;
  const double us = (n > 32 ? 1.0 : 3.5) + rate * m * k;
  return us <= tile_plan(m, k, n, true).us;
}

// Whether a product quantizes its x inside every workgroup: that saves a launch
// (k = 4096, us, with and without: n = 1, m = 4096 5.8, 7.5; m = 22016 21.2,
// 22.9; n = 4, m = 4096 6.5, 8.0), but each of them does it again (n = 8, m =
// 4096 8.7, 8.0; n = 4, m = 22016 24.3, 23.0; k = 11008, m = 4096, n = 2 14.9,
// 15.3; n = 4 16.8, 15.5).
bool fused_quant(int64_t n, int64_t k) { return n <= 4 && n * k <= 32768; }

// y = 0 (an empty sum), any element type
__global__ __launch_bounds__(256) void k_zero(uint8_t* __restrict__ y, int64_t bytes) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at < bytes) y[at] = 0;
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
int64_t code_bytes(int64_t n, int64_t k) { return align256(n * k) + align256(n * (k / kGroup) * 4); }

hipError_t quantize_act(const void* x, int xt, int64_t n, int64_t k, uint8_t* xq, float* scale,
                        bool by_group, hipStream_t s) {
  const int64_t groups = n * (k / kGroup);
  const int per = by_group ? static_cast<int>(k / kGroup) : 0;
  log_launch("quantize_act_f8 n=%lld k=%lld", (long long)n, (long long)k);
  return in_pieces(groups, 16, 256, [&](int64_t g0, int64_t c) {
    const dim3 grid(static_cast<unsigned>((c + 15) / 16));
    switch (xt) {
      case QBLK_F32: k_quant_act_f8<QBLK_F32><<<grid, 256, 0, s>>>(x, g0, c, xq, scale, per, static_cast<int>(n)); break;
      case QBLK_F16: k_quant_act_f8<QBLK_F16><<<grid, 256, 0, s>>>(x, g0, c, xq, scale, per, static_cast<int>(n)); break;
      default: k_quant_act_f8<QBLK_BF16><<<grid, 256, 0, s>>>(x, g0, c, xq, scale, per, static_cast<int>(n)); break;
    }
    return hipGetLastError();
  });
}

// Y = W X^T from codes, by one kernel or the other
hipError_t code_product(const uint8_t* w, const float* ws, int64_t m, int64_t k, const uint8_t* xq, const float* xs,
                        ScaleAt at, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  if (use_few(m, k, n)) return few_product(w, ws, m, k, FewX{xq, kCodes, xs, at.tok, at.group}, n, y, yt, 0, s);
  return tile_product(w, ws, m, k, xq, xs, n, y, yt, 0, nullptr, at, yt == QBLK_F32 || n <= kExactTokens, work, s);
}

}  // namespace

hipError_t launch_join(const float* part, int64_t m, int64_t n, int splits, void* y, int yt, hipStream_t s) {
  const int64_t pitch = part_pitch(m);
  return in_pieces(n * pitch / 4, 256, 256, [&](int64_t first, int64_t c) {
    k_f8_join<<<dim3(static_cast<unsigned>((c + 255) / 256)), 256, 0, s>>>(part, first, c, static_cast<int>(m), n * pitch, splits, y, yt);
    return hipGetLastError();
  });
}

hipError_t launch_quantize_act_f8(const void* x, int xt, int64_t n, int64_t k, uint8_t* xq, float* scale,
                                  hipStream_t s) {
  return quantize_act(x, xt, n, k, xq, scale, false, s);
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
  if (use_few(m, k, n)) return 0;
  const int a = tile_plan(m, k, n, false).splits, b = tile_plan(m, k, n, true).splits;
  const int most = a > b ? a : b;
  return most > 1 ? align256(most * n * part_pitch(m) * 4) : 0;
}

hipError_t launch_gemm_f8(const uint8_t* w, const float* ws, int64_t m, int64_t k, const uint8_t* xq,
                          const float* xs, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  return code_product(w, ws, m, k, xq, xs, ScaleAt{k / kGroup, 1}, n, y, yt, work, s);
}

int64_t linear_f8_workspace(int64_t m, int64_t k, int64_t n) {
  if (fused_quant(n, k)) return 0;
  return code_bytes(n, k) + gemm_f8_workspace(m, k, n);
}

hipError_t launch_linear_f8(const uint8_t* w, const float* ws, int64_t m, int64_t k, const void* x, int xt,
                            int64_t n, void* y, int yt, void* work, hipStream_t s) {
  if (fused_quant(n, k)) return few_product(w, ws, m, k, FewX{x, xt, nullptr, 0, 0}, n, y, yt, 0, s);
  uint8_t* xq = static_cast<uint8_t*>(work);
  float* xs = reinterpret_cast<float*>(xq + align256(n * k));
  const bool few = use_few(m, k, n);
  const hipError_t e = quantize_act(x, xt, n, k, xq, xs, few, s);
  if (e != hipSuccess) return e;
  return code_product(w, ws, m, k, xq, xs, few ? ScaleAt{1, n} : ScaleAt{k / kGroup, 1}, n, y, yt,
                      xq + code_bytes(n, k), s);
}

// ffn workspace.  First product by k_f8_few: h in fp32, then what the two
// products need, one after the other.  Else the codes of x, those of h, and the
// partial sums of one product or the other.
int64_t ffn_f8_workspace(int64_t h, int64_t i, int64_t n) {
  const int64_t up = gemm_f8_workspace(2 * i, h, n), down = gemm_f8_workspace(h, i, n);
  if (!use_few(2 * i, h, n)) return code_bytes(n, h) + code_bytes(n, i) + (up > down ? up : down);
  const int64_t first = fused_quant(n, h) ? 0 : code_bytes(n, h);
  const int64_t second = linear_f8_workspace(h, i, n);
  return align256(n * i * 4) + (first > second ? first : second);
}

hipError_t launch_ffn_f8(const uint8_t* w13, const float* s13, const uint8_t* w2, const float* s2, int64_t h,
                         int64_t i, const void* x, int xt, int64_t n, void* y, int yt, void* work, hipStream_t s) {
  hipError_t e;
  if (!use_few(2 * i, h, n)) {
    uint8_t* xq = static_cast<uint8_t*>(work);
    float* xs = reinterpret_cast<float*>(xq + align256(n * h));
    uint8_t* hq = xq + code_bytes(n, h);
    float* hs = reinterpret_cast<float*>(hq + align256(n * i));
    void* rest = hq + code_bytes(n, i);
    // (the codes of h turn on the last bits of the first product: see k_f8_tile)
    const bool exact = yt != QBLK_BF16 || n <= kExactTokens;
    // only a join can write the scales group by group
    const bool joined = tile_plan(2 * i, h, n, exact).splits > 1;
    const ScaleAt at = joined && use_few(h, i, n) ? ScaleAt{1, n} : ScaleAt{i / kGroup, 1};
    e = quantize_act(x, xt, n, h, xq, xs, false, s);
    if (e == hipSuccess) e = tile_product(w13, s13, 2 * i, h, xq, xs, n, hq, 0, i, hs, at, exact, rest, s);
    if (e != hipSuccess) return e;
    return code_product(w2, s2, h, i, hq, hs, at, n, y, yt, rest, s);
  }
  float* mid = static_cast<float*>(work);
  uint8_t* rest = static_cast<uint8_t*>(work) + align256(n * i * 4);
  if (fused_quant(n, h)) {
    e = few_product(w13, s13, 2 * i, h, FewX{x, xt, nullptr, 0, 0}, n, mid, QBLK_F32, i, s);
  } else {
    float* xs = reinterpret_cast<float*>(rest + align256(n * h));
    e = quantize_act(x, xt, n, h, rest, xs, true, s);
    if (e != hipSuccess) return e;
    e = few_product(w13, s13, 2 * i, h, FewX{rest, kCodes, xs, 1, n}, n, mid, QBLK_F32, i, s);
  }
  if (e != hipSuccess) return e;
  return launch_linear_f8(w2, s2, h, i, mid, QBLK_F32, n, y, yt, rest, s);
}

}  // namespace qblk
