// qblk_norm.hip -- root-mean-square norm of the residual stream with the codes
// that the next product reads, on gfx950.
//
//   t = x + residual, rounded to x's type (what the next layer adds to)
//   y = t * (1 / sqrt(mean(t^2) + eps)) * weight            in fp32
//   codes and scales of y: e4m3 with an fp32 scale per 128 columns, int8 with one
//   per row, or MXFP8 / MXFP4, each by the rule of its own quantizer
//
// The codes are made from the fp32 y: rounding it to 16 bits first would move them.  For
// the same reason the squares, eight at a time in fp32, are added up in 64 bits and the root's
// reciprocal is kept as a sum of two fp32 numbers: y is then t * weight, rounded once (16-bit
// inputs: not at all), times it.
#include <type_traits>

#include "qblk_mx_device.h"
#include "qblk_norm.h"

namespace qblk {
namespace {

// 8 values as they lie in memory: asked for first, made numbers of when they are used
struct Raw {
  u32x4 a, b;  // (b: of fp32)
};
__device__ __forceinline__ Raw fetch8(const void* x, bool wide, int64_t at) {
  Raw r;
  if (wide) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(x) + at);
    r.a = p[0];
    r.b = p[1];
  } else {
    r.a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + at);
    r.b = u32x4{0, 0, 0, 0};
  }
  return r;
}
template <int XT>
__device__ __forceinline__ void numbers(const Raw& r, float v[8]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (XT == QBLK_F32) {
      const uint32_t a = r.a[i], b = r.b[i];  // (a bit cast of a vector's element itself takes its first)
      v[i] = __builtin_bit_cast(float, a);
      v[4 + i] = __builtin_bit_cast(float, b);
    } else if constexpr (XT == QBLK_F16) {
      v[2 * i] = f16_bits_to_f32(r.a[i] & 0xffffu);
      v[2 * i + 1] = f16_bits_to_f32(r.a[i] >> 16);
    } else {
      v[2 * i] = bf16_bits_to_f32(r.a[i]);
      v[2 * i + 1] = __builtin_bit_cast(float, r.a[i] & 0xffff0000u);
    }
  }
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
    for (int i = 0; i < 2; i++) {
      const u32x2 w = pack16<XT>(float4_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]});
      h[2 * i] = w.x;
      h[2 * i + 1] = w.y;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = XT == QBLK_F16 ? f16_bits_to_f32(h[i] & 0xffffu) : bf16_bits_to_f32(h[i]);
      v[2 * i + 1] = XT == QBLK_F16 ? f16_bits_to_f32(h[i] >> 16) : __builtin_bit_cast(float, h[i] & 0xffff0000u);
    }
    if (to) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(to) + at) = u32x4{h[0], h[1], h[2], h[3]};
  }
}

// The row's sum from its threads' sums of eight squares, in every lane.  How many threads a
// row has goes by the number of rows (norm_width), what is added to what does not: rows of
// one width are taken by 2 TH threads with V / 2 units each or by TH with V (HALF), whose
// thread t stands for t and t + TH of the others.  Its two sums are joined over the lanes apart,
// as two waves would (the lower half of the lanes takes on the one, the upper the other), and
// meet as those waves' do behind the barrier.
template <int WAVES, int V, bool HALF>
__device__ __forceinline__ double row_sum(const double own[V], double* part, int wave) {
  const int lane = threadIdx.x & 63;
  double v = own[0];
  if constexpr (HALF) {
    double w = own[1];
#pragma unroll
    for (int j = 2; j < V; j += 2) {
      v += own[j];
      w += own[j + 1];
    }
    const double give = lane & 32 ? v : w;
    v = (lane & 32 ? w : v) + __shfl_xor(give, 32, kWave);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor(v, m, kWave);
    v += __shfl_xor(v, 32, kWave);
  } else {
#pragma unroll
    for (int j = 1; j < V; j++) v += own[j];
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, kWave);
  }
  if constexpr (WAVES > 1) {
    if (lane == 0) part[wave] = v;
    __syncthreads();
    auto pair = [&](int i) { return HALF ? part[i] : part[i] + part[i + WAVES / 2]; };
    v = pair(0);
#pragma unroll
    for (int i = 1; i < (HALF ? WAVES : WAVES / 2); i++) v += pair(i);
  }
  return v;
}

// The largest (NaN if one is) over `waves` waves' lanes, in every lane.
__device__ __forceinline__ float row_max(float v, float* part, int waves, int wave) {
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) v = max_nan(v, __shfl_xor(v, m, kWave));
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[wave] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int i = 1; i < waves; i++) v = max_nan(v, part[i]);
  return v;
}

// Memory bound, one pass (16384 rows of 4096 bf16 with a residual, to MXFP8: 84 to 90 us, 5.2 to
// 5.6 TB/s; 4096 rows 24 to 26 us; one row 2.7: a launch and one round trip).  1024 rows of 32768: 61
// us for 45 of bytes, since 113 registers leave room for one workgroup of 1024 threads a unit.  All loads of a row go
// out before the first use, the weights' too.
// One row by TH threads, V units of 8 values each (unit t, t + TH, ...); rows
// of one wave: four to a workgroup.  Rows wider than 8 TH V values (LOOP) are read a
// second time for the output.
template <int XT, int TH, int V, bool HALF, bool LOOP>
__global__ __launch_bounds__(TH < 256 ? 256 : TH) void k_rmsnorm(NormArgs p) {
  __shared__ double part[TH / kWave];
  __shared__ float part_max[TH / kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rows = TH < 256 ? 256 / TH : 1;
  const int64_t row = p.row0 + static_cast<int64_t>(blockIdx.x) * rows + (TH < 256 ? wave : 0);
  if (TH < 256 && row >= p.end) return;  // a wave's own row: no barrier in that form
  const int t = TH < 256 ? threadIdx.x & 63 : threadIdx.x;
  const int units = p.hidden / 8;
  const int64_t base = row * p.hidden;

  constexpr bool kWide = XT == QBLK_F32;
  const bool add = p.residual != nullptr;
  // t of unit u from what was fetched
  auto total = [&](int u, const Raw& x, const Raw& o, float v[8]) {
    numbers<XT>(x, v);
    if (add) {
      float w[8];
      numbers<XT>(o, w);
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] += w[i];
      round_store<XT>(v, p.total, base + 8 * u);
    }
  };
  auto squares = [](const float v[8]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) a = __builtin_fmaf(v[i], v[i], a);
    return a;
  };
  Raw xr[V], orr[V], wr[V];  // the weights too are asked for before the row's sum is known
  const Raw none = {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
#pragma unroll
  for (int j = 0; j < V; j++) {
    const int u = t + j * TH;
    xr[j] = u < units ? fetch8(p.x, kWide, base + 8 * u) : none;
  }
  if (add) {
#pragma unroll
    for (int j = 0; j < V; j++) {
      const int u = t + j * TH;
      orr[j] = u < units ? fetch8(p.residual, kWide, base + 8 * u) : none;
    }
  }
#pragma unroll
  for (int j = 0; j < V; j++) {
    const int u = t + j * TH;
    wr[j] = u < units ? fetch8(p.weight, p.wt == QBLK_F32, 8 * static_cast<int64_t>(u)) : none;
  }
  float v[V][8];
  double own[V];
#pragma unroll
  for (int j = 0; j < V; j++) {
    const int u = t + j * TH;
    if (u < units) {
      total(u, xr[j], orr[j], v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[j][i] = 0.0f;
    }
    own[j] = squares(v[j]);
  }
  if constexpr (LOOP) {
    for (int u = t + V * TH; u < units; u += TH) {
      float o[8];
      total(u, fetch8(p.x, kWide, base + 8 * u), add ? fetch8(p.residual, kWide, base + 8 * u) : none, o);
      own[0] += squares(o);
    }
  }
  const double sum = row_sum<TH / kWave, V, HALF>(own, part, wave);
  const double root = 1.0 / __builtin_sqrt(sum / p.hidden + p.eps);
  const float r1 = static_cast<float>(root), r2 = static_cast<float>(root - r1);  // (an infinite root: r2 NaN, as 0 * it)

  // y of N units
  auto scaled = [&](const Raw* w, float (*a)[8], auto N) {
    auto by = [&](auto T) {
#pragma unroll
      for (int j = 0; j < decltype(N)::value; j++) {
        float f[8];
        numbers<decltype(T)::value>(w[j], f);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float tw = a[j][i] * f[i];
          a[j][i] = __builtin_fmaf(tw, r1, tw * r2);
        }
      }
    };
    if (p.wt == QBLK_F32)
      by(std::integral_constant<int, QBLK_F32>());
    else if (p.wt == QBLK_F16)
      by(std::integral_constant<int, QBLK_F16>());
    else
      by(std::integral_constant<int, QBLK_BF16>());
  };
  auto largest = [](const float a[8], float top) {
#pragma unroll
    for (int i = 0; i < 8; i++) top = max_nan(top, __builtin_fabsf(a[i]));
    return top;
  };
  scaled(wr, v, std::integral_constant<int, V>());
  // LOOP: unit u again, from this thread's own stores, or x
  auto again = [&](int u, float a[1][8]) {
    numbers<XT>(fetch8(add ? p.total : p.x, kWide, base + 8 * u), a[0]);
    const Raw w = fetch8(p.weight, p.wt == QBLK_F32, 8 * static_cast<int64_t>(u));
    scaled(&w, a, std::integral_constant<int, 1>());
  };
  float top = 0.0f;
  if (p.act == QBLK_ACT_I8) {
#pragma unroll
    for (int j = 0; j < V; j++) top = t + j * TH < units ? largest(v[j], top) : top;
    if constexpr (LOOP) {
      for (int u = t + V * TH; u < units; u += TH) {
        float a[1][8];
        again(u, a);
        top = largest(a[0], top);
      }
    }
    top = row_max(top, part_max, TH / kWave, wave) / 127.0f;
    if (t == 0) static_cast<float*>(p.scale)[row] = top;
  }
  // The codes of unit u.  Whole waves take part: groups of 16 lanes and quads are on or off together.
  auto codes = [&](auto A, int u, float a[8], bool on) {
    constexpr int act = decltype(A)::value;
    uint32_t c[2];
    const int64_t at = base + 8 * u;
    if constexpr (act == QBLK_ACT_F8) {
      const float s = quant_group(a, c);
      if (on && (t & 15) == 0) static_cast<float*>(p.scale)[at / kGroup] = s;
    } else if constexpr (act == QBLK_ACT_I8) {
      int n[8];
      codes8(a, top, -127.0f, 127.0f, n);
#pragma unroll
      for (int i = 0; i < 2; i++)
        c[i] = (n[4 * i] & 255) | ((n[4 * i + 1] & 255) << 8) | ((n[4 * i + 2] & 255) << 16) | (static_cast<uint32_t>(n[4 * i + 3]) << 24);
    } else {
      const uint32_t b = mx_scale<act == QBLK_ACT_MXFP8>(quad_max(top_bits<8>(a)));
      mx_codes<act == QBLK_ACT_MXFP8, 8>(a, b, c);
      if (on && (t & 3) == 0) static_cast<uint8_t*>(p.scale)[at / kMxBlock] = static_cast<uint8_t>(b);
    }
    if (!on) return;
    if constexpr (act == QBLK_ACT_MXFP4)
      *reinterpret_cast<uint32_t*>(p.codes + at / 2) = c[0];
    else
      *reinterpret_cast<u32x2*>(p.codes + at) = u32x2{c[0], c[1]};
  };
  auto emit = [&](auto A) {
#pragma unroll
    for (int j = 0; j < V; j++) codes(A, t + j * TH, v[j], t + j * TH < units);
    if constexpr (LOOP) {
      for (int u0 = V * TH; u0 < units; u0 += TH) {
        float a[1][8] = {{0, 0, 0, 0, 0, 0, 0, 0}};
        if (u0 + t < units) again(u0 + t, a);
        codes(A, u0 + t, a[0], u0 + t < units);
      }
    }
  };
  switch (p.act) {
    case QBLK_ACT_F8: emit(std::integral_constant<int, QBLK_ACT_F8>()); break;
    case QBLK_ACT_I8: emit(std::integral_constant<int, QBLK_ACT_I8>()); break;
    case QBLK_ACT_MXFP8: emit(std::integral_constant<int, QBLK_ACT_MXFP8>()); break;
    case QBLK_ACT_MXFP4: emit(std::integral_constant<int, QBLK_ACT_MXFP4>()); break;
  }
  if (!p.y) return;
#pragma unroll
  for (int j = 0; j < V; j++)
    if (t + j * TH < units) round_store<XT>(v[j], p.y, base + 8 * (t + j * TH));
  if constexpr (LOOP) {
    for (int u = t + V * TH; u < units; u += TH) {
      float a[1][8];
      again(u, a);
      round_store<XT>(a[0], p.y, base + 8 * u);
    }
  }
}

template <int XT, int TH, int V, bool HALF, bool LOOP = false>
hipError_t norm(const NormArgs& all, int64_t n, hipStream_t s) {
  constexpr int rows = TH < 256 ? 256 / TH : 1, threads = TH < 256 ? 256 : TH;
  return in_pieces(n, rows, threads, [&](int64_t r0, int64_t c) {
    NormArgs a = all;
    a.row0 = r0;
    a.end = r0 + c;
    k_rmsnorm<XT, TH, V, HALF, LOOP><<<dim3(static_cast<unsigned>((c + rows - 1) / rows)), threads, 0, s>>>(a);
    return hipGetLastError();
  });
}

// Few rows: as many threads a row as it has work for; with more rows than compute units
// fewer, which wait for each other less (us, rows of 4096 bf16, 256 and 512 threads: 1 row with a
// residual 4.8, 3.6; 300 5.1, 5.1; 1000 8.8, 9.0, without a residual 6.0, 6.6; 1501 rows of
// 11008, 512 and 1024 threads: 35.5, 42.5).  With a residual a lane's 32 values and as many of
// it take too many registers (8192 rows of 8192, 256 and 512 threads: 91.2, 84.1; without a
// residual 43.7, 45.9).
template <int XT>
hipError_t norm_width(const NormArgs& a, int64_t n, hipStream_t s) {
  const int units = a.hidden / 8;
  const bool few = n <= cu_count();
  if (units <= 64) return norm<XT, 64, 1, false>(a, n, s);
  if (units <= 256) return norm<XT, 256, 1, false>(a, n, s);
  if (units <= 512) return few ? norm<XT, 512, 1, false>(a, n, s) : norm<XT, 256, 2, true>(a, n, s);
  if (units <= 1024) return a.residual || n <= 4 * cu_count() ? norm<XT, 512, 2, false>(a, n, s) : norm<XT, 256, 4, true>(a, n, s);
  if (units <= 2048) return few ? norm<XT, 1024, 2, false>(a, n, s) : norm<XT, 512, 4, true>(a, n, s);
  return norm<XT, 1024, 4, false, true>(a, n, s);
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
