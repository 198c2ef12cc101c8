// qblk_mx_tile.hip -- products of MXFP4 weights with many tokens on gfx950's
// scaled matrix instructions.
//
// A workgroup owns BM rows of W and BN tokens; 128 bytes of a token, 256 columns or
// (e4m3) 128, are one stage in LDS, filled by loads straight to LDS ahead of their use.
// A K = 64 instruction of 32 x 32 results takes a block of 32 columns from each half of
// the wave: half h of step t holds block Steps h + t of the stage, so that the scales
// of a lane's blocks lie together.  Results are summed by the
// matrix cores alone, scales included.
//
// Large products (8192^3: e2m1 261 us, 4.2 PFLOP/s, e4m3 399, 2.75; the instructions alone
// sustain 6.9 and 4.2) have matrix instructions in half (e2m1) to two thirds (e4m3) of the
// cycles: a unit's one workgroup of 256 x 256 waits at a barrier a stage, and its tile's first
// copies and last stores stand alone.  Power takes the clock down besides (zeros as operands: 219
// and 338 us).  Some hundred tokens are bound by the copies into LDS (5003 x 11008, 333 tokens, e2m1: 22
// us, 11 TB/s out of L2).  What bounds the shapes: at BM x BN results a stage a unit copies
// 128 (BM + BN) bytes of e2m1 for BM BN / 1024 matrix instructions of each of its four
// SIMDs, so wide tiles where there are enough of them.
#include <type_traits>

#include "qblk_lds.h"
#include "qblk_mx_device.h"
#include "qblk_mx_tile.h"

namespace qblk {
namespace {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef float float16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) uint8_t lds_byte;

// What the activations are.  kExact: e4m3 with fp32 results, both operands widened to bf16
// with their scales (k_mx_few says why) and multiplied there, at a quarter of the rate.
constexpr int kF4 = 0, kF8 = 1, kExact = 2;

// MI x NJ results of 32 x 32 a wave, WM x WN waves, STAGES stages in LDS.
template <int MI_, int NJ_, int WM_, int WN_, int STAGES_, int KIND_>
struct Shape {
  static constexpr int MI = MI_, NJ = NJ_, WM = WM_, WN = WN_, STAGES = STAGES_, KIND = KIND_;
  static constexpr int BM = 32 * MI * WM, BN = 32 * NJ * WN, WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int Blocks = KIND == kF4 ? 8 : 4;  // of 32 columns, a stage
  static constexpr int Steps = Blocks / 2;            // of 64 columns
  static constexpr int WRow = 16 * Blocks, XRow = 128;  // bytes of a row in a stage
  static constexpr int WBytes = BM * WRow, StageBytes = WBytes + BN * XRow;
  static constexpr int WCopies = WBytes / 1024 / WAVES, XCopies = BN * XRow / 1024 / WAVES, Copies = WCopies + XCopies;
  static constexpr int Early = (Copies + 1) / 2;  // copies behind the barrier; the others in the next stage's first step
  // Scales: of four stages at a time
  static constexpr int ScaleRow = 4 * Blocks, ScaleBytes = (BM + BN) * ScaleRow;
  static constexpr int ScaleUnits = (BM + BN) * (ScaleRow / 16), ScaleLoads = (ScaleUnits + THREADS - 1) / THREADS;
  static constexpr int Lds = STAGES * StageBytes + 2 * ScaleBytes;
  static constexpr int OutRow = 32 * MI * 4 + 16;  // bytes of a token's rows of one wave on their way out (fp32)
  static_assert(WBytes % (1024 * WAVES) == 0 && BN * XRow % (1024 * WAVES) == 0 && Lds <= 163840 && WAVES * 32 * OutRow <= Lds, "");
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

// 16 bytes of a row's scales, block `past` of which is the first wanted: moved to the
// front, zeros behind them.
__device__ __forceinline__ u32x4 moved(const u32x4& v, int past) {
  uint64_t lo = (static_cast<uint64_t>(v.y) << 32) | v.x, hi = (static_cast<uint64_t>(v.w) << 32) | v.z;
  if (past >= 16) lo = hi = 0;
  if (past >= 8) {
    lo = hi;
    hi = 0;
    past -= 8;
  }
  if (past > 0 && past < 8) {
    lo = (lo >> (8 * past)) | (hi << (64 - 8 * past));
    hi >>= 8 * past;
  }
  return u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
}

// The scales of a row of nb < 16 blocks from block b on.
__device__ __forceinline__ u32x4 few_scales(const uint8_t* row, int b, int nb) {
  uint64_t lo = 0, hi = 0;
#pragma nounroll
  for (int j = 0; j < nb; j++) {
    const uint64_t byte = row[j];
    if (j < 8)
      lo |= byte << (8 * j);
    else
      hi |= byte << (8 * j - 64);
  }
  return moved(u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)}, b);
}

// The order of a step: the next step's operands behind the first matrix
// instructions, the copies spread over all of them.
template <int I, int ALL, int READS, int COPIES>
__device__ __forceinline__ void order() {
  if constexpr (I < ALL) {
    constexpr int left = READS - 3 * I, reads = left > 3 ? 3 : left > 0 ? left : 0, copies = (I + 1) * COPIES / ALL - I * COPIES / ALL;
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
  const int nb = p.k / kMxBlock, G = (nb + S::Blocks - 1) / S::Blocks;

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
#pragma unroll
  for (int i = 0; i < S::WCopies; i++) {
    int R, c;
    placed<S::WRow>(wave + i * S::WAVES, lane, R, c);
    wo[i] = static_cast<uint32_t>(R < rows ? R : rows - 1) * static_cast<uint32_t>(wpitch) + 16 * c;
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
      to_lds(wbuf, base + at + (wave + i * S::WAVES) * 1024, wo[i < S::WCopies ? i : 0], g * S::WRow);
    else
      to_lds(xbuf, base + at + S::WBytes + (wave + (i - S::WCopies) * S::WAVES) * 1024, xo[i < S::WCopies ? 0 : i - S::WCopies], g * S::XRow);
  };
  auto clip = [&](int g) {  // before stage g's copies go out
    if (g == G - 1 && nb % S::Blocks) {
#pragma unroll
      for (int i = 0; i < S::WCopies; i++) {
        int R, c;
        placed<S::WRow>(wave + i * S::WAVES, lane, R, c);
        if (c >= nb % S::Blocks) wo[i] -= 16 * c;
      }
    }
  };

  // Scales of four stages, 16 bytes a thread, fetched some stages before they are put
  // to LDS.  Rows of 32 bytes: eight-byte part s of row R lies at part s ^ (R >> 3 & 3).
  uint8_t* const sbase = lds + S::STAGES * S::StageBytes;
  constexpr int kPerRow = S::ScaleRow / 16;
  const uint8_t* sp[S::ScaleLoads];  // a wave's units are all of W or all of x
  uint32_t so[S::ScaleLoads];
#pragma unroll
  for (int i = 0; i < S::ScaleLoads; i++) {
    const bool x = (wave * 64 + i * S::THREADS) / kPerRow >= S::BM;
    const int R = (threadIdx.x + i * S::THREADS) / kPerRow - (x ? S::BM : 0), last = x ? toks : rows;  // (past the last: repeats it)
    sp[i] = x ? p.xs + static_cast<int64_t>(t0) * nb : p.ws + static_cast<int64_t>(row0) * nb;
    so[i] = static_cast<uint32_t>(R < last ? R : last - 1) * static_cast<uint32_t>(nb);
  }
  // A group whose end lies past the row's is read so much before its start.
  u32x4 sv[S::ScaleLoads];
  const int in_row = 16 * (threadIdx.x % kPerRow);
  auto first_block = [&](int g) { return g * S::Blocks + in_row; };  // of this thread's, of the four stages from g on
  auto fetch_scales = [&](int g) {
    const int b = first_block(g), from = b < nb - 16 ? b : nb - 16;
#pragma unroll
    for (int i = 0; i < S::ScaleLoads; i++) sv[i] = *reinterpret_cast<const u32x4_a1*>(sp[i] + (so[i] + from));
  };
  auto put_scales = [&](int which, int g) {
    if ((g + 4) * S::Blocks > nb && nb >= 16) {
      const int b = first_block(g);
#pragma unroll
      for (int i = 0; i < S::ScaleLoads; i++) sv[i] = moved(sv[i], b > nb - 16 ? b - (nb - 16) : 0);
    }
#pragma unroll
    for (int i = 0; i < S::ScaleLoads; i++) {
      const int u = threadIdx.x + i * S::THREADS;
      if ((i + 1) * S::THREADS > S::ScaleUnits && u >= S::ScaleUnits) continue;
      uint8_t* to = sbase + which * S::ScaleBytes;
      if constexpr (kPerRow == 1) {
        *reinterpret_cast<u32x4*>(to + u * 16) = sv[i];
      } else {
        const int key = (u >> 4) & 3;
        const u32x4 v = key & 1 ? u32x4{sv[i].z, sv[i].w, sv[i].x, sv[i].y} : sv[i];
        *reinterpret_cast<u32x4*>(to + (u ^ (key >> 1)) * 16) = v;
      }
    }
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
  // e4m3 32 t) exchanged into the address.
  const int wplace = place<S::WRow>(wm * 32 * MI + r, S::Steps * h);
  const int xplace = S::WBytes + place<S::XRow>(wn * 32 * NJ + r, S::KIND == kF4 ? S::Steps * h : S::KIND == kF8 ? h : 4 * h);
  u32x4 wf[2][MI], xf[2][NJ][S::KIND == kF4 ? 1 : 2];
  auto read = [&](int at, int t, int to) {
#pragma unroll
    for (int i = 0; i < MI; i++) wf[to][i] = *reinterpret_cast<const u32x4*>(lds + at + (wplace ^ (16 * t)) + i * 32 * S::WRow);
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      if constexpr (S::KIND == kF4) {
        xf[to][j][0] = *reinterpret_cast<const u32x4*>(lds + at + (xplace ^ (16 * t)) + j * 32 * S::XRow);
      } else {  // the instruction's halves of e4m3, 16 columns of block t and 16 of block 2 + t; or a whole block
        xf[to][j][0] = *reinterpret_cast<const u32x4*>(lds + at + (xplace ^ (32 * t)) + j * 32 * S::XRow);
        xf[to][j][1] = *reinterpret_cast<const u32x4*>(lds + at + (xplace ^ (32 * t) ^ (S::KIND == kF8 ? 64 : 16)) + j * 32 * S::XRow);
      }
    }
  };
  // This half's scales of a stage: four bytes, or two.
  const int splace = S::KIND == kF4 ? r * 32 + ((r & 24)) + 4 * h : r * 16;
  uint32_t wsc[2][MI], xsc[2][NJ];
  auto read_scales = [&](int which, int s, int to) {
    const uint8_t* from = sbase + which * S::ScaleBytes + (S::KIND == kF4 ? splace ^ (8 * s) : splace + 4 * s);
    constexpr int row = S::ScaleRow;
#pragma unroll
    for (int i = 0; i < MI; i++) wsc[to][i] = *reinterpret_cast<const uint32_t*>(from + (wm * MI + i) * 32 * row);
#pragma unroll
    for (int j = 0; j < NJ; j++) xsc[to][j] = *reinterpret_cast<const uint32_t*>(from + (S::BM + (wn * NJ + j) * 32) * row);
  };
  auto shift_scales = [&](int to) {
    if constexpr (S::KIND != kF4) {
#pragma unroll
      for (int i = 0; i < MI; i++) wsc[to][i] >>= 16 * h;
#pragma unroll
      for (int j = 0; j < NJ; j++) xsc[to][j] >>= 16 * h;
    }
  };
  auto multiply = [&](int from, auto T, int sc) {
    constexpr int t = decltype(T)::value;
    if constexpr (S::KIND == kExact) {
      auto scale = [](uint32_t v) { return __builtin_bit_cast(float, ((v >> (8 * t)) & 255u) << 23); };
#pragma unroll
      for (int g = 0; g < 4; g++) {  // 8 of the block's columns
        bf16x8_n b[NJ];
#pragma unroll
        for (int j = 0; j < NJ; j++) {
          const u32x4 x = xf[from][j][(g >> 1) * (S::KIND == kF4 ? 0 : 1)];
          b[j] = wide8(x[2 * (g & 1)], x[2 * (g & 1) + 1], scale(xsc[sc][j]));
        }
#pragma unroll
        for (int i = 0; i < MI; i++) {
          const bf16x8_n a = wide4(wf[from][i][g], scale(wsc[sc][i]));
#pragma unroll
          for (int j = 0; j < NJ; j++) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b[j], acc[i][j], 0, 0, 0);
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
    for (int j = 0; j < NJ; j++) {
      const u32x4 a = wf[from][i], x = xf[from][j][0];
      const int8v av = {static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z), static_cast<int>(a.w), 0, 0, 0, 0};
      int8v bv = {static_cast<int>(x.x), static_cast<int>(x.y), static_cast<int>(x.z), static_cast<int>(x.w), 0, 0, 0, 0};
      const int sa = static_cast<int>(wsc[sc][i]), sb = static_cast<int>(xsc[sc][j]);
      if constexpr (S::KIND == kF4) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc[i][j], 4, 4, t, sa, t, sb);
      } else {
        const u32x4 z = xf[from][j][S::KIND == kF4 ? 0 : 1];
        bv = int8v{bv[0], bv[1], bv[2], bv[3], static_cast<int>(z.x), static_cast<int>(z.y), static_cast<int>(z.z), static_cast<int>(z.w)};
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc[i][j], 4, 0, t, sa, t, sb);
      }
    }
  };

  // The end of a step: its matrix instructions stay before it.
  auto pin = [&]() {
#pragma unroll
    for (int i = 0; i < MI; i++)
#pragma unroll
      for (int j = 0; j < NJ; j++) asm volatile("" : "+v"(acc[i][j]));
    __builtin_amdgcn_sched_barrier(0);
  };

  // One barrier a stage, before its last step: every wave has that step's operands
  // by then, so the stage's place is free for the copies of the stage STAGES further on
  // (half of them behind the barrier, half in the next stage's first step), and the
  // next stage has landed.  Copies past the last stage repeat it.
  auto barrier = [&](auto Newer) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    // those of STAGES - 2 stages stay under way, and the scales' loads behind them (rows
    // of fewer than 16 blocks have none)
    constexpr int stay = (S::STAGES - 2) * S::Copies, newer = decltype(Newer)::value;
    if (newer > 0 && nb < 16)
      __builtin_amdgcn_s_waitcnt(vm_lgkm0(stay));
    else
      __builtin_amdgcn_s_waitcnt(vm_lgkm0(stay + newer));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto held = [&](int g) { return g < g1 ? g : g1 - 1; };
  constexpr int reads = MI + NJ * (S::KIND == kF4 ? 1 : 2);

#pragma unroll
  for (int s = 0; s < S::STAGES; s++) {
    clip(g0 + s);
#pragma unroll
    for (int i = 0; i < (s == S::STAGES - 1 ? S::Early : S::Copies); i++) copy(s * S::StageBytes, held(g0 + s), i);
  }
  if (nb >= 16) {
    fetch_scales(g0);
  } else {
#pragma unroll
    for (int i = 0; i < S::ScaleLoads; i++) sv[i] = few_scales(sp[i] + so[i], in_row, nb);
  }
  put_scales(0, g0);
  __builtin_amdgcn_s_waitcnt(vm_lgkm0(0));  // (a barrier alone does not promise that copies to LDS have landed)
  __syncthreads();
  read_scales(0, 0, 0);
  shift_scales(0);
  read(0, 0, 0);

  int at = 0;                                // the current stage's place
  int old = (S::STAGES - 1) * S::StageBytes;  // the one before
  int group = 0;  // scales in turn: this group of four stages is in buffer `group`
  // Stage g, the Q-th of its group (splits begin with one).  The next group's scales are
  // fetched in its first stage and put in its last one; past the last group the last one's
  // (their rows have more than 16 blocks where there are two groups).
  auto stage = [&](int g, auto Q) {
    constexpr int q = decltype(Q)::value, set = q & 1;
    const int nxt = at + S::StageBytes < S::STAGES * S::StageBytes ? at + S::StageBytes : 0;
    const int next = g - q + 4 < G ? g - q + 4 : g - q;
    if (q == 3) put_scales(group ^ 1, next);
    __builtin_amdgcn_sched_barrier(0);
    auto step = [&](auto T) {
      constexpr int t = decltype(T)::value;
      read(at, t + 1, (t + 1) & 1);
      if constexpr (t == 0) {
#pragma unroll
        for (int i = S::Early; i < S::Copies; i++) copy(old, held(g + S::STAGES - 1), i);
      }
      multiply(t & 1, T, set);
      if constexpr (S::KIND != kExact) order<0, MI * NJ, reads, (t == 0 ? S::Copies - S::Early : 0)>();
      pin();
    };
    step(std::integral_constant<int, 0>());
    if (q == 0) {
      if (nb >= 16) fetch_scales(next);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (S::Steps == 4) {
      step(std::integral_constant<int, 1>());
      step(std::integral_constant<int, 2>());
    }
    barrier(std::integral_constant<int, q == 0 ? S::ScaleLoads : 0>());
    clip(g + S::STAGES);
    read(nxt, 0, 0);
    read_scales(q == 3 ? group ^ 1 : group, (q + 1) & 3, set ^ 1);
#pragma unroll
    for (int i = 0; i < S::Early; i++) copy(at, held(g + S::STAGES), i);
    multiply(1, std::integral_constant<int, S::Steps - 1>(), set);
    if constexpr (S::KIND != kExact) order<0, MI * NJ, reads + MI + NJ, S::Early>();
    pin();
    shift_scales(set ^ 1);
    old = at;
    at = nxt;
  };
  for (int g = g0; g < g1; g += 4) {
    stage(g, std::integral_constant<int, 0>());
    if (g + 1 < g1) stage(g + 1, std::integral_constant<int, 1>());
    if (g + 2 < g1) stage(g + 2, std::integral_constant<int, 2>());
    if (g + 3 < g1) stage(g + 3, std::integral_constant<int, 3>());
    group ^= 1;
  }
  __builtin_amdgcn_s_waitcnt(vm_lgkm0(0));
  __syncthreads();  // the last copies have landed: LDS may be used again, and left

  // Lane (r, h) holds token r and rows 8 (e >> 2) + 4 h + (e & 3) of each 32 x 32.  32
  // tokens at a time go through the wave's own part of LDS, so that 32 MI rows of a
  // token leave together.
  uint8_t* const out = lds + wave * 32 * S::OutRow;
  const int rowb = row0 + wm * 32 * MI;
  auto wave_fence = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };
  auto part = [&](int i, int j, int q) {
    return float4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
  };
  auto leave16 = [&](auto T) {
    constexpr int lanes = 4 * MI;  // a token's rows, eight each
#pragma unroll
    for (int j = 0; j < NJ; j++) {
#pragma unroll
      for (int i = 0; i < MI; i++)
#pragma unroll
        for (int q = 0; q < 4; q++)
          *reinterpret_cast<u32x2*>(out + r * (S::OutRow / 2) + (32 * i + 8 * q + 4 * h) * 2) = pack16<decltype(T)::value>(part(i, j, q));
      wave_fence();
      const int tok0 = t0 + (wn * NJ + j) * 32 + lane / lanes, row = rowb + 8 * (lane % lanes);
#pragma unroll
      for (int u = 0; u < 32 * lanes / 64; u++) {
        const int tok = tok0 + u * (64 / lanes);
        const u32x4 v = *reinterpret_cast<const u32x4*>(out + (u * (64 / lanes) + lane / lanes) * (S::OutRow / 2) + (row - rowb) * 2);
        if (tok >= p.n || row >= p.m) continue;
        uint16_t* y = static_cast<uint16_t*>(p.y) + static_cast<int64_t>(tok) * p.m + row;
        if (row + 8 <= p.m) {
          *reinterpret_cast<u32x4_a2*>(y) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 7; e++)
            if (row + e < p.m) y[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
        }
      }
      wave_fence();
    }
  };
  auto leave32 = [&] {
    constexpr int lanes = 8 * MI;  // four each
#pragma unroll
    for (int j = 0; j < NJ; j++) {
#pragma unroll
      for (int i = 0; i < MI; i++)
#pragma unroll
        for (int q = 0; q < 4; q++) *reinterpret_cast<float4_t*>(out + r * S::OutRow + (32 * i + 8 * q + 4 * h) * 4) = part(i, j, q);
      wave_fence();
      const int tok0 = t0 + (wn * NJ + j) * 32 + lane / lanes, row = rowb + 4 * (lane % lanes);
#pragma unroll
      for (int u = 0; u < 32 * lanes / 64; u++) {
        const int tok = tok0 + u * (64 / lanes);
        const float4_t v = *reinterpret_cast<const float4_t*>(out + (u * (64 / lanes) + lane / lanes) * S::OutRow + (row - rowb) * 4);
        if (tok >= p.n || row >= p.m) continue;
        if constexpr (SPLIT) {  // rows of partial sums lie 16-byte aligned, with room behind the last
          *reinterpret_cast<float4_t*>(p.part + (static_cast<int64_t>(blockIdx.y) * p.n + tok) * part_pitch(p.m) + row) = v;
        } else {
          float* y = static_cast<float*>(p.y) + static_cast<int64_t>(tok) * p.m + row;
          if (row + 4 <= p.m) {
            *reinterpret_cast<float4_a4*>(y) = v;
          } else {
#pragma unroll
            for (int e = 0; e < 3; e++)
              if (row + e < p.m) y[e] = v[e];
          }
        }
      }
      wave_fence();
    }
  };
  if (SPLIT || p.yt == QBLK_F32)
    leave32();
  else if (p.yt == QBLK_F16)
    leave16(std::integral_constant<int, QBLK_F16>());
  else
    leave16(std::integral_constant<int, QBLK_BF16>());
}

template <class S, bool SPLIT>
hipError_t go(const MxTileArgs& a, int splits, hipStream_t s) {
  static std::atomic<uint64_t> done{0};
  const hipError_t allowed = allow_lds(done, reinterpret_cast<const void*>(k_mx_tile<S, SPLIT>), S::Lds);
  if (allowed != hipSuccess) return allowed;
  log_launch("mx tile %s %dx%d stages=%d%s m=%d k=%d n=%d tiles=%dx%d from=%d splits=%d", S::KIND == kF4 ? "f4" : S::KIND == kF8 ? "f8" : "exact",
             S::BM, S::BN, S::STAGES, SPLIT ? " split" : "", a.m, a.k, a.n, a.row_tiles, a.tok_tiles, a.first_row_tile, splits);
  k_mx_tile<S, SPLIT><<<dim3(static_cast<unsigned>(a.row_tiles * a.tok_tiles), static_cast<unsigned>(splits)), S::THREADS, S::Lds, s>>>(a);
  return hipGetLastError();
}

// kMxTiles.  The tiles of 128 rows leave room for two workgroups a compute unit, which
// hide each other's ends and barriers.  Of e2m1 activations that takes two stages each;
// where there is one workgroup a unit anyway it has three (us, two and three stages: 4096 x
// 4096, 64 tokens, 128 x 64: 12.4, 9.6; 11008 x 4096, 333 tokens, 128 x 128: 21.2, 25.7).
// Tiles of 64 rows are for products that else leave compute units idle or have to be
// split (14336 x 4096, 64 tokens, 128 rows and 64: e2m1 14.2, 11.9, e4m3 16.4, 15.7; 22016
// rows 15.8, 16.9); with three to eight stages they take the same time within 5%.
template <int KIND, bool SPLIT>
hipError_t by_shape(int shape, const MxTileArgs& a, int splits, hipStream_t s) {
  constexpr bool f4 = KIND == kF4;
  const bool many = !f4 || static_cast<int64_t>(a.row_tiles) * a.tok_tiles * splits > cu_count();
  switch (shape) {
    case 0: return go<Shape<4, 2, 2, 4, f4 ? 2 : 3, KIND>, SPLIT>(a, splits, s);
    case 1:  // (e4m3 only)
      if constexpr (f4)
        return hipErrorInvalidValue;
      else
        return go<Shape<2, 2, 4, 2, 4, KIND>, SPLIT>(a, splits, s);
    case 2: return go<Shape<4, 1, 2, 2, f4 ? 3 : 5, KIND>, SPLIT>(a, splits, s);
    case 3: return many ? go<Shape<2, 2, 2, 2, f4 ? 2 : 3, KIND>, SPLIT>(a, splits, s) : go<Shape<2, 2, 2, 2, 3, KIND>, SPLIT>(a, splits, s);
    case 4: return many ? go<Shape<2, 1, 2, 2, f4 ? 2 : 4, KIND>, SPLIT>(a, splits, s) : go<Shape<2, 1, 2, 2, f4 ? 3 : 4, KIND>, SPLIT>(a, splits, s);
    default: return go<Shape<1, 1, 2, 2, f4 ? 3 : 5, KIND>, SPLIT>(a, splits, s);
  }
}

}  // namespace

hipError_t mx_tile_exact(int shape, const MxTileArgs& a, int splits, hipStream_t s) {
  using Wide = Shape<2, 2, 4, 2, 4, kExact>;
  using Small = Shape<2, 1, 2, 2, 4, kExact>;
  if (shape == 1) return splits > 1 ? go<Wide, true>(a, splits, s) : go<Wide, false>(a, 1, s);
  return splits > 1 ? go<Small, true>(a, splits, s) : go<Small, false>(a, 1, s);
}

hipError_t mx_tile(int shape, bool f8, const MxTileArgs& a, int splits, hipStream_t s) {
  if (splits > 1) return f8 ? by_shape<kF8, true>(shape, a, splits, s) : by_shape<kF4, true>(shape, a, splits, s);
  return f8 ? by_shape<kF8, false>(shape, a, 1, s) : by_shape<kF4, false>(shape, a, 1, s);
}

}  // namespace qblk
