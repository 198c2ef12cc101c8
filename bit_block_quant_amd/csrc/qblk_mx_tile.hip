// qblk_mx_tile.hip -- products of MXFP4 weights with many tokens on gfx950's
// scaled matrix instructions.
//
// A workgroup owns BM rows of W and BN tokens; 128 columns are one stage in LDS
// (64 bytes of a row of W, 64 or 128 of a token), filled by loads straight to LDS
// several stages ahead.  A K = 64 instruction of 32 x 32 results takes a block of 32
// columns from each half of the wave: half h of step t holds block 2 h + t of the
// stage, so that a lane's two scales lie together.  Results are summed by the
// matrix cores alone, scales included.
#include <type_traits>

#include "qblk_mx_device.h"
#include "qblk_mx_tile.h"

namespace qblk {
namespace {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef float float16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) uint8_t lds_byte;

constexpr int kStageBlocks = 4;  // 128 columns
constexpr int kWRow = 64;        // bytes of a row of W in a stage

// What the activations are, and how sums are formed.
constexpr int kF4 = 0, kF8 = 1;

template <int MI_, int NJ_, int WM_, int WN_, int STAGES_, int KIND_>
struct Shape {
  static constexpr int MI = MI_, NJ = NJ_, WM = WM_, WN = WN_, STAGES = STAGES_, KIND = KIND_;
  static constexpr int BM = 32 * MI * WM, BN = 32 * NJ * WN, WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int XRow = KIND == kF4 ? 64 : 128;
  static constexpr int WBytes = BM * kWRow, StageBytes = WBytes + BN * XRow;
  static constexpr int WCopies = WBytes / 1024 / WAVES, XCopies = BN * XRow / 1024 / WAVES, Copies = WCopies + XCopies;
  static constexpr int ScaleBytes = (BM + BN) * 16;  // of four stages
  static constexpr int ScaleRows = (BM + BN + THREADS - 1) / THREADS;
  static constexpr int Lds = STAGES * StageBytes + 2 * ScaleBytes;
  static_assert(WBytes % (1024 * WAVES) == 0 && BN * XRow % (1024 * WAVES) == 0 && Lds <= 163840, "");
};

// Rows of 64 bytes: 16-byte chunk c of row R lies at chunk c ^ (R >> 2 & 3).
// Rows of 128 bytes: row R lies at row R ^ (R >> 3 & 1), its chunk c at c ^ (R & 7).
// The 16 rows that one phase of an operand's read takes then start at 16 different
// columns of banks.
template <int ROW>
__device__ __forceinline__ int place(int R, int c) {
  return ROW == 64 ? R * 64 + ((c ^ ((R >> 2) & 3)) << 4) : (R ^ ((R >> 3) & 1)) * 128 + ((c ^ (R & 7)) << 4);
}
// The row and chunk that byte 16 l of KB j of a stage holds.
template <int ROW>
__device__ __forceinline__ void placed(int j, int l, int& R, int& c) {
  if (ROW == 64) {
    R = 16 * j + (l >> 2);
    c = (l & 3) ^ ((R >> 2) & 3);
  } else {
    const int s = 8 * j + (l >> 3);
    R = s ^ ((s >> 3) & 1);
    c = (l & 7) ^ (R & 7);
  }
}

// 16 bytes a lane straight to LDS.  (The host's pass has no such builtin, and would drop
// the kernels that use it.)
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t from, lds_byte* to, uint32_t lane_at, int at) {
#ifdef __HIP_DEVICE_COMPILE__
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void*)to, 16, lane_at, at, 0, 0);
#endif
}

// 16 bytes of a row's scales from block 16 g on; past the row's end zeros
__device__ __forceinline__ u32x4 scales16(const uint8_t* row, int g, int nb) {
  const uint8_t* p = row + 16 * static_cast<int64_t>(g);
  const int left = nb - 16 * g;
  if (left >= 16) return *reinterpret_cast<const u32x4_a1*>(p);
  uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 15; j++)
    if (j < left) v[j >> 2] |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
  return u32x4{v[0], v[1], v[2], v[3]};
}

// The order of a step: an operand's read and, less often, a copy behind every few
// matrix instructions.
template <int I, int ALL, int READS, int COPIES>
__device__ __forceinline__ void order() {
  if constexpr (I < ALL) {
    constexpr int reads = (I + 1) * READS / ALL - I * READS / ALL, copies = (I + 1) * COPIES / ALL - I * COPIES / ALL;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (reads > 0) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
    if constexpr (copies > 0) __builtin_amdgcn_sched_group_barrier(0x020, copies, 0);
    order<I + 1, ALL, READS, COPIES>();
  }
}

// s_waitcnt's operand: at most `vm` loads under way, no LDS operation
constexpr int vm_lgkm0(int vm) { return 0x0070 | (vm & 15) | ((vm >> 4) << 14); }

template <class S, bool SPLIT>
__global__ __launch_bounds__(S::THREADS) void k_mx_tile(MxTileArgs p) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int MI = S::MI, NJ = S::NJ;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int nb = p.k / kMxBlock, G = (nb + kStageBlocks - 1) / kStageBlocks;

  // Workgroups go to the 8 XCDs in turn; each XCD takes a run of consecutive
  // tiles (token tiles fastest, in bands of 8), so that its L2 holds the row tiles
  // and token tiles that its CUs work on together.
  const int tiles = p.row_tiles * p.tok_tiles;
  const int b = blockIdx.x, xcd = b & 7;
  const int tile = xcd * (tiles >> 3) + (xcd < (tiles & 7) ? xcd : (tiles & 7)) + (b >> 3);
  const int band = tile / (8 * p.row_tiles), in_band = tile - band * 8 * p.row_tiles;
  const int wide = p.tok_tiles - 8 * band < 8 ? p.tok_tiles - 8 * band : 8;
  const int in_rt = in_band / wide, tt = 8 * band + in_band - in_rt * wide, rt = p.first_row_tile + in_rt;
  const int row0 = rt * S::BM, t0 = tt * S::BN;
  const int g0 = SPLIT ? blockIdx.y * p.stages_per_split : 0;
  const int g1 = SPLIT ? (g0 + p.stages_per_split < G ? g0 + p.stages_per_split : G) : G;

  // What this lane copies of a stage: 16-byte chunks, as offsets from the tile's
  // first row.  Rows past the matrix repeat its last one (their results are not
  // stored); of the last stage chunks of W past the row's end repeat its first (x is
  // zero there: p.x_pitch counts whole stages).
  const int rows = p.m - row0 < S::BM ? p.m - row0 : S::BM, toks = p.n - t0 < S::BN ? p.n - t0 : S::BN;
  const int64_t wpitch = static_cast<int64_t>(nb) * 16;
  const auto wbuf = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.w + row0 * wpitch), 0,
                                                      static_cast<uint32_t>(rows * wpitch), 0x00027000);
  const auto xbuf = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.xq + t0 * p.x_pitch), 0,
                                                      static_cast<uint32_t>(toks * p.x_pitch), 0x00027000);
  uint32_t wo[S::WCopies], xo[S::XCopies];
  int wc = 0;  // this lane's chunk in every copy of W
#pragma unroll
  for (int i = 0; i < S::WCopies; i++) {
    int R;
    placed<kWRow>(wave + i * S::WAVES, lane, R, wc);
    wo[i] = static_cast<uint32_t>(R < rows ? R : rows - 1) * static_cast<uint32_t>(wpitch) + 16 * wc;
  }
#pragma unroll
  for (int i = 0; i < S::XCopies; i++) {
    int R, c;
    placed<S::XRow>(wave + i * S::WAVES, lane, R, c);
    xo[i] = static_cast<uint32_t>(R < toks ? R : toks - 1) * static_cast<uint32_t>(p.x_pitch) + 16 * c;
  }
  lds_byte* const base = (lds_byte*)lds;
  auto copy = [&](int at, int g, int i) {  // copy i of stage g into the stage at byte `at`
    if (i < S::WCopies)
      to_lds(wbuf, base + at + (wave + i * S::WAVES) * 1024, wo[i < S::WCopies ? i : 0], g * kWRow);
    else
      to_lds(xbuf, base + at + S::WBytes + (wave + (i - S::WCopies) * S::WAVES) * 1024, xo[i < S::WCopies ? 0 : i - S::WCopies], g * S::XRow);
  };
  auto clip = [&](int g) {  // before stage g's copies go out
    if (g == G - 1 && (nb & 3)) {
#pragma unroll
      for (int i = 0; i < S::WCopies; i++)
        if (wc >= (nb & 3)) wo[i] -= 16 * wc;
    }
  };

  // Scales of four stages: 16 bytes a row or token, fetched a stage before they are put to LDS.
  uint8_t* const sbase = lds + S::STAGES * S::StageBytes;
  const uint8_t* sp[S::ScaleRows];
#pragma unroll
  for (int i = 0; i < S::ScaleRows; i++) {
    const int at = threadIdx.x + i * S::THREADS;  // (past the last token: repeats it)
    const bool x = at >= S::BM;
    const int R = x ? at - S::BM : at, last = x ? toks : rows;
    sp[i] = (x ? p.xs + static_cast<int64_t>(t0 + (R < last ? R : last - 1)) * nb : p.ws + static_cast<int64_t>(row0 + (R < last ? R : last - 1)) * nb);
  }
  u32x4 sv[S::ScaleRows];
  auto fetch_scales = [&](int gg) {
#pragma unroll
    for (int i = 0; i < S::ScaleRows; i++) sv[i] = scales16(sp[i], gg, nb);
  };
  auto put_scales = [&](int which) {
#pragma unroll
    for (int i = 0; i < S::ScaleRows; i++)
      if ((i + 1) * S::THREADS <= S::BM + S::BN || threadIdx.x + i * S::THREADS < S::BM + S::BN)
        *reinterpret_cast<u32x4*>(sbase + which * S::ScaleBytes + (threadIdx.x + i * S::THREADS) * 16) = sv[i];
  };

  const int wm = wave % S::WM, wn = wave / S::WM;
  float16_t acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; i++)
#pragma unroll
    for (int j = 0; j < NJ; j++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;

  // Where this lane's operands lie in a stage: step t's is the first's with 16 t (of
  // 128-byte rows 32 t) exchanged into the address.
  const int wplace = place<kWRow>(wm * 32 * MI + r, 2 * h);
  const int xplace = S::WBytes + (S::KIND == kF4 ? place<64>(wn * 32 * NJ + r, 2 * h) : place<128>(wn * 32 * NJ + r, h));
  u32x4 wf[2][MI], xf[2][NJ][S::KIND == kF4 ? 1 : 2];
  auto read = [&](int at, int t, int to) {
#pragma unroll
    for (int i = 0; i < MI; i++) wf[to][i] = *reinterpret_cast<const u32x4*>(lds + at + (wplace ^ (16 * t)) + i * 32 * kWRow);
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      if constexpr (S::KIND == kF4) {
        xf[to][j][0] = *reinterpret_cast<const u32x4*>(lds + at + (xplace ^ (16 * t)) + j * 32 * 64);
      } else {  // the instruction's halves of e4m3: 16 columns of block t, 16 of block 2 + t
        xf[to][j][0] = *reinterpret_cast<const u32x4*>(lds + at + (xplace ^ (32 * t)) + j * 32 * 128);
        xf[to][j][1] = *reinterpret_cast<const u32x4*>(lds + at + (xplace ^ (32 * t) ^ 64) + j * 32 * 128);
      }
    }
  };
  uint32_t wsc[MI][4], xsc[NJ][4];  // per stage of four: this half's two scales
  auto read_scales = [&](int which) {
    const uint8_t* s = sbase + which * S::ScaleBytes;
#pragma unroll
    for (int i = 0; i < MI; i++) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(s + (wm * 32 * MI + 32 * i + r) * 16);
#pragma unroll
      for (int e = 0; e < 4; e++) wsc[i][e] = v[e] >> (16 * h);
    }
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(s + (S::BM + wn * 32 * NJ + 32 * j + r) * 16);
#pragma unroll
      for (int e = 0; e < 4; e++) xsc[j][e] = v[e] >> (16 * h);
    }
  };
  auto multiply = [&](int from, int t, int e) {
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
      for (int j = 0; j < NJ; j++) {
        const u32x4 a = wf[from][i], x = xf[from][j][0];
        const int8v av = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w), 0, 0, 0, 0};
        int8v bv = {static_cast<int>(x.x), static_cast<int>(x.y), static_cast<int>(x.z), static_cast<int>(x.w), 0, 0, 0, 0};
        const int sa = static_cast<int>(wsc[i][e]), sb = static_cast<int>(xsc[j][e]);
        if constexpr (S::KIND == kF4) {
          acc[i][j] = t == 0 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc[i][j], 4, 4, 0, sa, 0, sb)
                             : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc[i][j], 4, 4, 1, sa, 1, sb);
        } else {
          const u32x4 z = xf[from][j][S::KIND == kF4 ? 0 : 1];
          bv = int8v{bv[0], bv[1], bv[2], bv[3], static_cast<int>(z.x), static_cast<int>(z.y), static_cast<int>(z.z), static_cast<int>(z.w)};
          acc[i][j] = t == 0 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc[i][j], 4, 0, 0, sa, 0, sb)
                             : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc[i][j], 4, 0, 1, sa, 1, sb);
        }
      }
  };

  // One barrier a stage, between its two steps: every wave has the second step's
  // operands by then, so the stage's place is free for the copies of the stage
  // STAGES further on (half of them behind the barrier, half behind the next stage's
  // first step), and the next stage has landed.  Copies past the last stage repeat it.
  auto barrier = [&]() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_waitcnt(vm_lgkm0((S::STAGES - 2) * S::Copies));  // those of STAGES - 2 stages stay under way
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto held = [&](int g) { return g < g1 ? g : g1 - 1; };

  fetch_scales(g0 / 4);
  put_scales(0);
#pragma unroll
  for (int s = 0; s < S::STAGES; s++) {
    clip(g0 + s);
#pragma unroll
    for (int i = 0; i < (s == S::STAGES - 1 ? S::Copies / 2 : S::Copies); i++) copy(s * S::StageBytes, held(g0 + s), i);
  }
  __syncthreads();
  read_scales(0);
  read(0, 0, 0);

  const int last_scales = (G - 1) / 4;
  int at = 0;                                // the current stage's place
  int old = (S::STAGES - 1) * S::StageBytes;  // the one before
  auto stage = [&](int g, auto E) {
    constexpr int e = decltype(E)::value;
    constexpr int reads = MI + NJ * (S::KIND == kF4 ? 1 : 2);
    const int nxt = at + S::StageBytes < S::STAGES * S::StageBytes ? at + S::StageBytes : 0;
    // (splits begin at multiples of four stages)
    if (e == 0) fetch_scales(g / 4 < last_scales ? g / 4 + 1 : last_scales);
    if (e == 3) put_scales((g / 4 + 1 - g0 / 4) & 1);
    __builtin_amdgcn_sched_barrier(0);
    read(at, 1, 1);
#pragma unroll
    for (int i = S::Copies / 2; i < S::Copies; i++) copy(old, held(g + S::STAGES - 1), i);
    multiply(0, 0, e);
    order<0, MI * NJ, reads, S::Copies / 2>();
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    clip(g + S::STAGES);
    read(nxt, 0, 0);
#pragma unroll
    for (int i = 0; i < S::Copies / 2; i++) copy(at, held(g + S::STAGES), i);
    multiply(1, 1, e);
    order<0, MI * NJ, reads, S::Copies / 2>();
    __builtin_amdgcn_sched_barrier(0);
    if (e == 3) read_scales((g / 4 + 1 - g0 / 4) & 1);
    old = at;
    at = nxt;
  };
  for (int g = g0; g < g1; g += 4) {
    stage(g, std::integral_constant<int, 0>());
    if (g + 1 < g1) stage(g + 1, std::integral_constant<int, 1>());
    if (g + 2 < g1) stage(g + 2, std::integral_constant<int, 2>());
    if (g + 3 < g1) stage(g + 3, std::integral_constant<int, 3>());
  }
  // (the last copies may still be under way: a workgroup's LDS is not given away before they land)
  __builtin_amdgcn_s_waitcnt(vm_lgkm0(0));

  // lane (r, h) holds token r and rows 8 (e >> 2) + 4 h + (e & 3) of each 32 x 32
#pragma unroll
  for (int j = 0; j < NJ; j++) {
    const int tok = t0 + (wn * NJ + j) * 32 + r;
    if (tok >= p.n) continue;
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int row = row0 + (wm * MI + i) * 32 + 8 * q + 4 * h;
        if (row >= p.m) continue;
        const float4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        if constexpr (SPLIT) {
          *reinterpret_cast<float4_t*>(p.part + (static_cast<int64_t>(blockIdx.y) * p.n + tok) * part_pitch(p.m) + row) = v;
          continue;
        }
        const int64_t to = static_cast<int64_t>(tok) * p.m + row;
        if (row + 4 <= p.m) {
          if (p.yt == QBLK_F32)
            *reinterpret_cast<float4_a4*>(static_cast<float*>(p.y) + to) = v;
          else
            *reinterpret_cast<u32x2_a2*>(static_cast<uint16_t*>(p.y) + to) = bits16(v, p.yt);
        } else {
#pragma unroll
          for (int e = 0; e < 4; e++)
            if (row + e < p.m) store_y(p.y, to + e, v[e], p.yt);
        }
      }
  }
}

template <class S, bool SPLIT>
hipError_t go(const MxTileArgs& a, int splits, hipStream_t s) {
  static const hipError_t allowed = hipFuncSetAttribute(reinterpret_cast<const void*>(k_mx_tile<S, SPLIT>),
                                                        hipFuncAttributeMaxDynamicSharedMemorySize, S::Lds);
  if (allowed != hipSuccess) return allowed;
  k_mx_tile<S, SPLIT><<<dim3(static_cast<unsigned>(a.row_tiles * a.tok_tiles), static_cast<unsigned>(splits)), S::THREADS, S::Lds, s>>>(a);
  return hipGetLastError();
}

// Tokens of a tile: 256, 128 or 64.
template <int KIND, bool SPLIT>
hipError_t by_tokens(int tokens, const MxTileArgs& a, int splits, hipStream_t s) {
  switch (tokens) {
    case 64: return go<Shape<4, 1, 2, 2, KIND == kF4 ? 6 : 5, KIND>, SPLIT>(a, splits, s);
    case 128: return go<Shape<2, 2, 4, 2, KIND == kF4 ? 5 : 4, KIND>, SPLIT>(a, splits, s);
    default: return go<Shape<4, 2, 2, 4, KIND == kF4 ? 4 : 3, KIND>, SPLIT>(a, splits, s);
  }
}

}  // namespace

hipError_t mx_tile(int tokens, bool f8, const MxTileArgs& a, int splits, hipStream_t s) {
  if (splits > 1) return f8 ? by_tokens<kF8, true>(tokens, a, splits, s) : by_tokens<kF4, true>(tokens, a, splits, s);
  return f8 ? by_tokens<kF8, false>(tokens, a, 1, s) : by_tokens<kF4, false>(tokens, a, 1, s);
}

}  // namespace qblk
