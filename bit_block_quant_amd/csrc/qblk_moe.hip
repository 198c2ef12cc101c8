// qblk_moe.hip -- a mixture-of-experts layer for a few tokens, straight out of
// the packed 4-bit experts, in two kernels on gfx950.
//
//   route     the top_k experts of a token by logit (ties: the lowest index;
//             -inf and NaN never taken), softmax weights in fp32
//   k_moe_up  h[p] = silu(G_e x) * (U_e x) for every pair p of a token and one
//             of its experts e
//   k_moe_down  y[t] = sum_j w[t,j] D_e h[(t,j)]
//
// Both are bound by the packed bytes of the experts that are reached.  The
// tokens of one expert are gathered into a matrix-core tile of up to 16, so an
// expert's weights are read once for all of them; the codes are decoded into
// registers in the operand layout of the 16x16x32 matrix instructions.
//
// Layout.  Weights are loaded by halves of a super-block (128 columns) of 16
// rows: four neighbouring lanes load the four units of 32 of one row, 64
// consecutive bytes, and the scale of their unit.  (In operand order, with
// neighbouring lanes in different rows, every lane is an access of its own to
// the vector cache, which then bounds the kernel: 581 accesses instead of
// about 150 per half of a gate and an up tile.)  Through 1.5 KB of LDS per
// wave they become matrix operands: quarter q of the lanes holds weights
// 4q..4q+3 (low nibbles) and 16+4q..16+4q+3 (high) of a unit.  The other
// operand is brought into that order too.  A code byte 0..15 is the e4m3
// number code * 2^-9 as it stands (subnormals below 8, the first binade from 8
// on), so one conversion with scale 2^9 gives two exact codes as f16 or bf16.
//
// Sums.  Codes and activations are exact in the operands, products and sums
// fp32.  The offset of the format (-8, or the affine formats' own) multiplies
// sum(x) of the unit, which a matrix product with a constant operand gives in
// the layout of the result.  h is carried as two bf16 parts (hi + lo, 2^-17
// relative), which is half the size of what a third part would make it and
// ahead of every 16-bit result.
#include "qblk_device.h"
#include "qblk_launch.h"
#include "qblk_moe.h"

namespace qblk {
namespace {

typedef __bf16 bf16x2_n __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_n __attribute__((ext_vector_type(8)));
typedef half_t half8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kSplit = 4;       // waves that share the columns of one tile of gate or up rows
constexpr int kUpWaves = 2 * kSplit;
constexpr int kDownWaves = 16;  // waves that share the experts of one tile
constexpr uint32_t kLo4 = 0x0F0F0F0Fu;

// The routing of one piece, in LDS or in the workspace: experts with at least
// one pair are slots 0 .. active-1; slot s owns places off[s] .. off[s+1] - 1
// of the lists of pairs (token * top_k + choice) and of their tokens.
struct Table {
  int active;
  int expert[kMoeMaxExperts];
  int off[kMoeMaxExperts + 1];
  uint16_t pair[kMoeMaxPairs];
  uint16_t token[kMoeMaxPairs];
};

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + __builtin_expf(-g)) * u; }

// ------------------------------------------------------------ the operands
// 16-bit operand types of the matrix cores
template <bool F16>
struct Op;
template <>
struct Op<true> {
  typedef half8_t v8;
  static __device__ __forceinline__ uint32_t two(uint32_t codes, bool hi) {
    const half2_t p = hi ? __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 512.0f, true))
                         : __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, 512.0f, false));
    return __builtin_bit_cast(uint32_t, p);
  }
  static __device__ __forceinline__ float4_t mma(u32x4 a, u32x4 b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static constexpr uint32_t one2 = 0x3C003C00u, minus8 = 0xC800C800u;
};
template <>
struct Op<false> {
  typedef bf16x8_n v8;
  static __device__ __forceinline__ uint32_t two(uint32_t codes, bool hi) {
    const bf16x2_n p = hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 512.0f, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 512.0f, false);
    return __builtin_bit_cast(uint32_t, p);
  }
  static __device__ __forceinline__ float4_t mma(u32x4 a, u32x4 b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  static constexpr uint32_t one2 = 0x3F803F80u, minus8 = 0xC100C100u;
};

template <bool F16>
__device__ __forceinline__ u32x4 codes8_op(uint32_t t) {
  const uint32_t lo = t & kLo4, hi = (t >> 4) & kLo4;
  return u32x4{Op<F16>::two(lo, false), Op<F16>::two(lo, true), Op<F16>::two(hi, false), Op<F16>::two(hi, true)};
}

// ------------------------------------------------------------- the formats
// One unit of 32 weights per lane: unit u = lane & 3 of half super-block hf
// of row lane >> 2.  `load` fetches it, scale() and offset() decode its scale
// (weight = scale * code + offset, for the formats with affine = false offset
// is -8 * scale and not formed).  `units` is the number of units of a row:
// only Q4_0 rows may end inside a half; units past the end repeat the last
// one's codes and scale by zero.
template <int FMT>
struct Unit;

// (global loads take any address: blocks of 18 and 138 bytes start at every other byte)
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));

template <>
struct Unit<QBLK_SB4> {
  static constexpr bool affine = false;
  u32x4_a2 raw;
  uint32_t h;
  __device__ __forceinline__ void pin() { asm volatile("" : "+v"(raw), "+v"(h)); }
  __device__ __forceinline__ u32x4 codes() const { return raw; }
  template <int I>
  __device__ __forceinline__ uint32_t head() const {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(h), I * 0x55, 0xF, 0xF, true));
  }
  __device__ __forceinline__ void load(const uint8_t* row, int hf, int u, int) {
    const uint8_t* p = row + static_cast<int64_t>(hf >> 1) * 138;
    raw = *reinterpret_cast<const u32x4_a2*>(p + 10 + 64 * (hf & 1) + 16 * u);
    // the first lane the super-scale, the others the half's four sub-scales
    h = *reinterpret_cast<const u32_a2*>(p + (u == 0 ? 0 : 2 + 4 * (hf & 1)));
  }
  __device__ __forceinline__ float scale(int, int u, int) const {
    return f16_bits_to_f32(head<0>() & 0xffffu) * static_cast<float>(static_cast<int8_t>(head<1>() >> (8 * u)));
  }
  __device__ __forceinline__ float offset(int, int) const { return 0.0f; }
};

template <>
struct Unit<QBLK_SB4_AFFINE> {
  static constexpr bool affine = true;
  u32x4_a4 raw;
  uint32_t h;
  __device__ __forceinline__ void pin() { asm volatile("" : "+v"(raw), "+v"(h)); }
  __device__ __forceinline__ u32x4 codes() const { return raw; }
  template <int I>
  __device__ __forceinline__ uint32_t head() const {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(h), I * 0x55, 0xF, 0xF, true));
  }
  __device__ __forceinline__ void load(const uint8_t* row, int hf, int u, int) {
    const uint8_t* p = row + static_cast<int64_t>(hf >> 1) * 148;  // a multiple of 4: codes are dword aligned
    const int j = 4 * (hf & 1) + u;
    raw = *reinterpret_cast<const u32x4_a4*>(p + 20 + 16 * j);
    // dword 0 (both super-scales), the half's four sub-scales and its four offsets, one to a lane
    h = reinterpret_cast<const uint32_t*>(p)[u == 0 ? 0 : u == 1 ? 1 + (hf & 1) : 3 + (hf & 1)];
  }
  __device__ __forceinline__ float scale(int, int u, int) const {
    return f16_bits_to_f32(head<0>() & 0xffffu) * static_cast<float>(static_cast<int8_t>(head<1>() >> (8 * u)));
  }
  __device__ __forceinline__ float offset(int, int u) const {
    return f16_bits_to_f32(head<0>() >> 16) * static_cast<float>(static_cast<int8_t>(head<2>() >> (8 * u)));
  }
};

template <>
struct Unit<QBLK_Q4_K> {
  static constexpr bool affine = true;
  u32x4 raw;
  uint32_t h;
  __device__ __forceinline__ void pin() { asm volatile("" : "+v"(raw), "+v"(h)); }
  __device__ __forceinline__ u32x4 codes() const { return raw; }
  __device__ __forceinline__ void load(const uint8_t* row, int hf, int u, int) {
    const u32x4* p = reinterpret_cast<const u32x4*>(row + static_cast<int64_t>(hf >> 1) * 144);  // 16-byte aligned
    raw = p[1 + 4 * (hf & 1) + u];
    h = reinterpret_cast<const uint32_t*>(p)[u];  // a dword of the header each
  }
  template <int I>
  __device__ __forceinline__ uint32_t head() const {  // dword I of it, from lane I of the four
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(h), I * 0x55, 0xF, 0xF, true));
  }
  __device__ __forceinline__ float scale(int hf, int u, int) const {
    return f16_bits_to_f32(head<0>() & 0xffffu) * static_cast<float>(q4k_scale6(head<1>(), head<2>(), 4 * (hf & 1) + u));
  }
  __device__ __forceinline__ float offset(int hf, int u) const {
    return -(f16_bits_to_f32(head<0>() >> 16) * static_cast<float>(q4k_min6(head<2>(), head<3>(), 4 * (hf & 1) + u)));
  }
};

template <>
struct Unit<QBLK_Q4_0> {
  static constexpr bool affine = false;
  u32x4_a2 raw;
  uint32_t d;
  __device__ __forceinline__ void pin() { asm volatile("" : "+v"(raw), "+v"(d)); }
  __device__ __forceinline__ u32x4 codes() const { return raw; }
  __device__ __forceinline__ void load(const uint8_t* row, int hf, int u, int units) {
    const int at = 4 * hf + u;
    const uint8_t* p = row + static_cast<int64_t>(at < units ? at : units - 1) * 18;
    raw = *reinterpret_cast<const u32x4_a2*>(p + 2);
    d = load_u16(p);
  }
  __device__ __forceinline__ float scale(int hf, int u, int units) const {
    return 4 * hf + u < units ? f16_bits_to_f32(d) : 0.0f;
  }
  __device__ __forceinline__ float offset(int, int) const { return 0.0f; }
};

// The exchange of one half of 16 rows from units per lane to operands, in a
// wave's own LDS (its accesses there are executed in order).
struct Stage {
  u32x4 codes[64];  // row, unit ^ (row >> 2 & 3): the 16 rows' dwords of one unit lie in different banks
  float scale[64], offset[64];
};
// One row of 128 weights per lane row: unit u's dword of this quarter, scales, offsets.
struct Operand {
  uint32_t t[4];
  float4_t s, o;
};
template <int FMT>
__device__ __forceinline__ Operand to_operand(Unit<FMT>& w, int hf, int units, Stage& st) {
  // What was loaded is looked at from here on: without this the compiler
  // decodes it where it was loaded, a loop turn earlier, and waits there.
  w.pin();
  const int lane = threadIdx.x & 63, row = lane >> 2, u = lane & 3, r = lane & 15, q = lane >> 4;
  st.codes[4 * row + (u ^ ((row >> 2) & 3))] = w.codes();
  st.scale[lane] = w.scale(hf, u, units);
  if constexpr (Unit<FMT>::affine) st.offset[lane] = w.offset(hf, u);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  Operand p;
  const uint32_t* c = reinterpret_cast<const uint32_t*>(st.codes);
#pragma unroll
  for (int i = 0; i < 4; i++) p.t[i] = c[16 * r + 4 * (i ^ ((r >> 2) & 3)) + q];
  p.s = *reinterpret_cast<const float4_t*>(st.scale + 4 * r);
  if constexpr (Unit<FMT>::affine) p.o = *reinterpret_cast<const float4_t*>(st.offset + 4 * r);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return p;
}

// acc += (unit u of 16 rows) x (16 gathered token rows), the operand in PARTS summands
template <int FMT, bool F16, int PARTS>
__device__ __forceinline__ void mul_unit(const Operand& w, int u, const u32x4 (&a)[PARTS], const float4_t& xs,
                                         float4_t& acc) {
  const u32x4 b = codes8_op<F16>(w.t[u]);
  float4_t p = Unit<FMT>::affine ? float4_t{0, 0, 0, 0} : xs;
#pragma unroll
  for (int i = 0; i < PARTS; i++) p = Op<F16>::mma(a[i], b, p);
#pragma unroll
  for (int i = 0; i < 4; i++) acc[i] = __builtin_fmaf(w.s[u], p[i], acc[i]);
  if constexpr (Unit<FMT>::affine) {
#pragma unroll
    for (int i = 0; i < 4; i++) acc[i] = __builtin_fmaf(w.o[u], xs[i], acc[i]);
  }
}

// sum(x) of the unit per token (times -8 for the formats whose offset that is)
template <int FMT, bool F16, int PARTS>
__device__ __forceinline__ float4_t unit_sum(const u32x4 (&a)[PARTS]) {
  const uint32_t c = Unit<FMT>::affine ? Op<F16>::one2 : Op<F16>::minus8;
  float4_t p = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < PARTS; i++) p = Op<F16>::mma(a[i], u32x4{c, c, c, c}, p);
  return p;
}

// ---------------------------------------------------------------- routing
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
// Over the 16 lanes of a DPP row, in every lane: exchanges with lanes ^1, ^2,
// then mirrored in 8 and in 16.
template <class Op>
__device__ __forceinline__ float row16(float v, Op op) {
  v = op(v, __builtin_bit_cast(float, dpp<0xB1>(__builtin_bit_cast(int, v))));
  v = op(v, __builtin_bit_cast(float, dpp<0x4E>(__builtin_bit_cast(int, v))));
  v = op(v, __builtin_bit_cast(float, dpp<0x141>(__builtin_bit_cast(int, v))));
  return op(v, __builtin_bit_cast(float, dpp<0x140>(__builtin_bit_cast(int, v))));
}
__device__ __forceinline__ int row16_min(int v) {
  int o = dpp<0xB1>(v);
  v = v < o ? v : o;
  o = dpp<0x4E>(v);
  v = v < o ? v : o;
  o = dpp<0x141>(v);
  v = v < o ? v : o;
  o = dpp<0x140>(v);
  return v < o ? v : o;
}

// Four tokens by one wave, 16 lanes to each: lane l of a row looks at experts
// l, l + 16, ...  A round takes the largest logit that is left and, of equal
// ones, the lowest expert.  `token` may be past the end (its row idles).
template <int PER>
__device__ void route_tokens(const MoeArgs& a, int token, int* ids, bool write) {
  const float none = -__builtin_huge_valf();
  const int l = threadIdx.x & 15;
  const bool on = token < a.n;
  const float* logits = a.logits + static_cast<int64_t>(on ? token : 0) * a.experts;
  float v[PER];
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int e = 16 * i + l;
    const float x = on && e < a.experts ? logits[e] : none;
    v[i] = x > none ? __builtin_fminf(x, 3.402823466e38f) : none;  // NaN is never taken
  }
  const auto max2 = [](float x, float y) { return __builtin_fmaxf(x, y); };
  const auto sum2 = [](float x, float y) { return x + y; };
  float top = none, sum = 0.0f, mine[2] = {0.0f, 0.0f};
  int id[2] = {-1, -1};  // choices l and l + 16
  for (int j = 0; j < a.top_k; j++) {
    float m = v[0];
    int at = l;
#pragma unroll
    for (int i = 1; i < PER; i++) {
      at = v[i] > m ? 16 * i + l : at;
      m = __builtin_fmaxf(m, v[i]);
    }
    const float best = row16(m, max2);
    const int e = row16_min(m == best ? at : 1 << 30);
    if (j == 0) {
      top = best;
      if (!a.renorm) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; i++) s += v[i] > none ? __builtin_expf(v[i] - top) : 0.0f;
        sum = row16(s, sum2);
      }
    }
    if (best > none) {
      const float p = __builtin_expf(best - top);
      if (a.renorm) sum += p;
      if ((j & 15) == l) {
        id[j >> 4] = e;
        mine[j >> 4] = p;
      }
#pragma unroll
      for (int i = 0; i < PER; i++) v[i] = 16 * i + l == e ? none : v[i];
    }
  }
#pragma unroll
  for (int h = 0; h < 2; h++)
    if (on && 16 * h + l < a.top_k) {
      const int p = token * a.top_k + 16 * h + l;
      ids[p] = id[h];
      if (write) {
        a.ids[p] = id[h];
        a.weights[p] = id[h] >= 0 ? mine[h] / sum * a.wscale : 0.0f;
      }
    }
}

// The table of up to 64 pairs, by one wave: the pairs of the first expert that
// is left, found by comparing with it, until none is.
__device__ void few_pairs_table(const int* ids, int pairs, int top_k, Table& t) {
  const int lane = threadIdx.x & 63;
  const int id = lane < pairs ? ids[lane] : -1;
  uint64_t left = __builtin_amdgcn_ballot_w64(id >= 0);
  int slot = 0, off = 0;
  while (left != 0) {
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t same = __builtin_amdgcn_ballot_w64(id == e);
    if (lane == 0) {
      t.expert[slot] = e;
      t.off[slot] = off;
    }
    if (id == e) {
      const int at = off + __popcll(same & ((uint64_t(1) << lane) - 1));
      t.pair[at] = static_cast<uint16_t>(lane);
      t.token[at] = static_cast<uint16_t>(lane / top_k);
    }
    off += __popcll(same);
    slot++;
    left &= ~same;
  }
  if (lane == 0) {
    t.active = slot;
    t.off[slot] = off;
  }
}

// The table of any number of pairs, by all threads of the workgroup.  A pair's
// place must not depend on timing (every workgroup makes the table for itself
// and h is stored by place), so it is counted: the pairs of its expert in the
// blocks of 64 before its own, then those before it in the block.
struct TableScratch {
  int ids[kMoeMaxPairs];
  int base[kMoeMaxExperts];
  uint16_t count[kMoeMaxPairs / 64][kMoeMaxExperts];
};

__device__ void build_table(int pairs, int experts, int top_k, Table& t, TableScratch& z) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, blocks = (pairs + 63) / 64;
  constexpr int kRounds = (kMoeMaxPairs / 64 + kUpWaves - 1) / kUpWaves;
  for (int i = threadIdx.x; i < blocks * kMoeMaxExperts; i += blockDim.x) (&z.count[0][0])[i] = 0;
  __syncthreads();
  int id[kRounds], rank[kRounds];
#pragma unroll
  for (int k = 0; k < kRounds; k++) {
    const int b = wave + k * kUpWaves, p = 64 * b + lane;
    id[k] = b < blocks && p < pairs ? z.ids[p] : -1;
    uint64_t same = __builtin_amdgcn_ballot_w64(id[k] >= 0);  // the lanes with this lane's expert, a bit at a time
#pragma unroll
    for (int bit = 1; bit < kMoeMaxExperts; bit <<= 1) {
      const uint64_t set = __builtin_amdgcn_ballot_w64((id[k] & bit) != 0);
      same &= (id[k] & bit) ? set : ~set;
    }
    rank[k] = __popcll(same & ((uint64_t(1) << lane) - 1));
    if (id[k] >= 0 && rank[k] == 0) z.count[b][id[k]] = static_cast<uint16_t>(__popcll(same));
  }
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += blockDim.x) {
    int before = 0;
    for (int b = 0; b < blocks; b++) {
      const int c = z.count[b][e];
      z.count[b][e] = static_cast<uint16_t>(before);
      before += c;
    }
    z.base[e] = before;
  }
  __syncthreads();
  if (wave == 0) {
    int slots = 0, total = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
      const int e = e0 + lane;
      const int c = e < experts ? z.base[e] : 0;
      int run = c;  // inclusive sum over the lanes
#pragma unroll
      for (int x = 1; x < kWave; x <<= 1) {
        const int o = __shfl_up(run, x, kWave);
        if (lane >= x) run += o;
      }
      const uint64_t some = __builtin_amdgcn_ballot_w64(c > 0);
      if (c > 0) {
        const int s = slots + __popcll(some & ((uint64_t(1) << lane) - 1));
        t.expert[s] = e;
        t.off[s] = total + run - c;
        z.base[e] = total + run - c;
      }
      slots += __popcll(some);
      total += __shfl(run, 63, kWave);
    }
    if (lane == 0) {
      t.active = slots;
      t.off[slots] = total;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kRounds; k++)
    if (id[k] >= 0) {
      const int b = wave + k * kUpWaves;
      const int at = z.base[id[k]] + z.count[b][id[k]] + rank[k], p = 64 * b + lane;
      t.pair[at] = static_cast<uint16_t>(p);
      t.token[at] = static_cast<uint16_t>(p / top_k);
    }
  __syncthreads();
}

// --------------------------------------------------------------- gate, up
// A workgroup takes tiles of 16 gate rows and the 16 up rows that go with
// them, for all tokens of one expert.  Four waves work on the gate rows, four
// on the up rows; the four split the columns (wave k takes halves k, k + 4,
// ...) and their sums meet in LDS.  One tile per wave leaves the registers for
// weights two halves ahead of the multiply: what bounds the kernel is how many
// bytes are on their way.  Workgroups are persistent, so the routing is worked
// out once in each rather than by a launch of its own.
//
// Measured: one token, 8 of 64 experts of 2048/1024, Type 0: 11.9 us, 2.5 of them
// the routing, 1 the table; the 18 MB of weights come in 3.6.  64 tokens, 4 of 32
// experts of 4096/2048, Type 1: 106 us, 2.9 TB/s: about 75 VALU operations for 1.1
// KB of weights take as long to issue as those take to come (without the weights'
// loads 78 us, with nothing but them 75).
template <int FMT, bool F16>
__global__ __launch_bounds__(kUpWaves* kWave, 4) void k_moe_up(MoeArgs a) {
  // two workgroups to a CU: at most 80 KB each
  __shared__ Table table;
  struct Tiles {
    float4_t red[2][kUpWaves][64];
    u32x4 x[kUpWaves][256];
    Stage stage[kUpWaves];
  };
  __shared__ union {
    Tiles tiles;
    TableScratch scratch;  // before the first tile
  } lds;
  static_assert(sizeof lds + sizeof table <= 80 * 1024);
  TableScratch& scratch = lds.scratch;
  int* const ids = scratch.ids;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4, wrow = lane >> 2, wu = lane & 3;
  const int pairs = a.n * a.top_k;

  if (a.logits != nullptr) {
    for (int t = 4 * wave; t < a.n; t += 4 * kUpWaves) {
      const bool write = blockIdx.x == 0;
      if (a.experts <= 64)
        route_tokens<4>(a, t + q, ids, write);
      else if (a.experts <= 128)
        route_tokens<8>(a, t + q, ids, write);
      else
        route_tokens<kMoeMaxExperts / 16>(a, t + q, ids, write);
    }
  } else {
    for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
      const int e = a.ids[p];
      ids[p] = e >= 0 && e < a.experts ? e : -1;
    }
  }
  __syncthreads();
  if (pairs <= 64) {
    if (wave == 0) few_pairs_table(ids, pairs, a.top_k, table);
    __syncthreads();
  } else {
    build_table(pairs, a.experts, a.top_k, table, scratch);
  }
  if (blockIdx.x == 0) {
    Table* t = static_cast<Table*>(a.table);
    for (int s = threadIdx.x; s <= table.active; s += blockDim.x) {
      if (s < table.active) t->expert[s] = table.expert[s];
      t->off[s] = table.off[s];
    }
    for (int p = threadIdx.x; p < table.off[table.active]; p += blockDim.x) t->pair[p] = table.pair[p];
    if (threadIdx.x == 0) t->active = table.active;
  }

  const int tiles = a.inter / 16, units = a.hidden / 32, halves = (units + 3) / 4;
  // tiles of all experts in a row; at most 2^24 (512 experts, 2^19 rows)
  const uint32_t tasks = static_cast<uint32_t>(table.active) * static_cast<uint32_t>(tiles);
  if (blockIdx.x >= tasks) return;
  const int slot_step = gridDim.x / tiles, tile_step = gridDim.x % tiles;
  const int side = wave / kSplit, part = wave % kSplit;  // gate or up; share of the columns
  const bool busy = part < halves;
  u32x4* const xw = lds.tiles.x[wave];
  Stage& stage = lds.tiles.stage[wave];

  // A place in the sequence of halves that this wave multiplies: for its
  // workgroup's tiles, each expert's pairs 16 at a time, halves part, part +
  // kSplit, ...  At the end it stays at the last tile (loaded, not used).
  struct Place {
    uint32_t task;
    int slot, tile, first, count, c0, hf;
  };
  auto pairs_of = [&](Place& p) {
    p.first = __builtin_amdgcn_readfirstlane(table.off[p.slot]);
    p.count = __builtin_amdgcn_readfirstlane(table.off[p.slot + 1]) - p.first;
    p.c0 = 0;
  };
  auto next_task = [&](Place& p) {  // false at the last
    p.c0 = 0;
    if (p.task + gridDim.x >= tasks) return false;
    p.task += gridDim.x;
    p.slot += slot_step;
    p.tile += tile_step;
    if (p.tile >= tiles) {
      p.tile -= tiles;
      p.slot++;
    }
    pairs_of(p);
    return true;
  };
  auto advance = [&](Place& p) {  // whether the tile or the 16 pairs changed
    p.hf += kSplit;
    if (p.hf < halves) return false;
    p.hf = part;
    p.c0 += 16;
    if (p.c0 >= p.count) next_task(p);
    return true;
  };
  auto row_of = [&](const Place& p) {
    const int64_t e = __builtin_amdgcn_readfirstlane(table.expert[p.slot]);
    return a.gate_up + (e * 2 * a.inter + static_cast<int64_t>(side) * a.inter + 16 * p.tile + wrow) * a.up_row_bytes;
  };

  // x by halves (128 columns), whole rows at a time: 16 lanes load 256 bytes of
  // a token's row, four rows an instruction and only as many as the expert
  // has; through LDS they become operands.  (Loaded as operands from memory,
  // 16 rows lie 2 * hidden bytes apart and every load asks for 16 lines.)
  // Row i of the four: token row 4i + q, its 16-byte chunk r ^ row going to LDS
  // chunk r: 16 rows of one chunk column then lie in 16 different columns of
  // banks.
  const uint8_t* xp4[4];
  int xrows = 0;
  u32x4 xr[4];
  auto x_rows = [&](const Place& p) {  // its 16 pairs; past the last one that again
    xrows = p.count - p.c0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int at = 4 * i + q < xrows ? 4 * i + q : xrows - 1;
      xp4[i] = static_cast<const uint8_t*>(a.x) + static_cast<int64_t>(table.token[p.first + p.c0 + at]) * (a.hidden * 2ll) +
               16 * (r ^ (4 * i + q));
    }
  };
  auto x_load = [&](int hf) {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (4 * i < xrows) {
        int at = 256 * hf;
        if constexpr (FMT == QBLK_Q4_0) {
          // past the row's end the last chunk again: those weights scale by zero
          const int chunk = 16 * hf + (r ^ (4 * i + q));
          if (chunk >= 4 * units) at = 64 * units - 16 - 16 * (r ^ (4 * i + q));
        }
        xr[i] = *reinterpret_cast<const u32x4*>(xp4[i] + at);
      }
  };

  // The tile's sums, put together by four of the waves, another four (and in
  // them another first one: few tokens keep only it busy) each time.  One
  // barrier: the other buffer is read by nobody any more once it is passed.
  int turn = 0;
  auto finish = [&](const Place& p, const float4_t& acc) {
    auto& red = lds.tiles.red[turn & 1];
    red[wave][lane] = acc;
    __syncthreads();
    const int duty = (wave + 3 * turn) & (kUpWaves - 1);
    turn++;
    if (duty < 4) {
      // lane (row r, quarter q) of the sums holds tokens 4q .. 4q+3
      const int tok = 4 * duty + (lane >> 4), rr = lane & 15;
      if (p.c0 + tok < p.count) {
        float gs = 0.0f, us = 0.0f;
#pragma unroll
        for (int w = 0; w < kSplit; w++) {
          gs += red[w][(tok >> 2) * 16 + rr][tok & 3];
          us += red[kSplit + w][(tok >> 2) * 16 + rr][tok & 3];
        }
        const float h = silu_mul(gs, us);
        const uint16_t hi = f32_to_bf16_bits(h);
        const float rest = h - bf16_bits_to_f32(hi);
        const int tile = p.tile;
        // operand order, see h_rows in k_moe_down: unit tile/2 of this expert's pairs
        uint16_t* out = static_cast<uint16_t*>(a.h) + static_cast<int64_t>(p.first) * a.inter * 2 +
                        (static_cast<int64_t>((tile & ~1) * 4 + (rr >> 2)) * p.count + p.c0 + tok) * 8 + 4 * (tile & 1) + (rr & 3);
        out[0] = hi;
        out[static_cast<int64_t>(p.count) * 32] = __builtin_isfinite(rest) ? f32_to_bf16_bits(rest) : 0;
      }
    }
  };

  Place p;  // what is multiplied now
  p.task = blockIdx.x;
  p.slot = blockIdx.x / tiles;
  p.tile = blockIdx.x % tiles;
  p.hf = part;
  pairs_of(p);
  float4_t acc = {0, 0, 0, 0};
  // after the last half of 16 pairs: their sums; false after the last tile
  auto next_pairs = [&]() {
    finish(p, acc);
    acc = float4_t{0, 0, 0, 0};
    p.c0 += 16;
    return p.c0 < p.count || next_task(p);
  };
  if (!busy) {
    while (next_pairs()) {
    }
    return;
  }

  Place wp = p, xp = p;  // of the weights two halves on, of x one half on
  const uint8_t* row = row_of(wp);
  Unit<FMT> w0, w1;
  // (in the loop's order: the waits in it count what was issued since)
  w0.load(row, wp.hf, wu, units);
  __builtin_amdgcn_sched_barrier(0);
  x_rows(xp);
  x_load(xp.hf);
  if (advance(wp)) row = row_of(wp);
  __builtin_amdgcn_sched_barrier(0);
  w1.load(row, wp.hf, wu, units);
  __builtin_amdgcn_sched_barrier(0);
  bool done = false;
  // One half.  `w` is emptied into LDS and loaded anew, two halves on, in
  // place: copying one register set to another would wait for its loads.
  auto half = [&](Unit<FMT>& w) {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (4 * i < p.count - p.c0) xw[64 * i + lane] = xr[i];
    const Operand o = to_operand(w, p.hf, units, stage);
    u32x4 xa[4];
    const uint8_t* from = reinterpret_cast<const uint8_t*>(xw) + 256 * r + 8 * (q & 1);
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const u32x2 l0 = *reinterpret_cast<const u32x2*>(from + 16 * ((4 * u + (q >> 1)) ^ r));
      const u32x2 l1 = *reinterpret_cast<const u32x2*>(from + 16 * ((4 * u + 2 + (q >> 1)) ^ r));
      xa[u] = u32x4{l0.x, l0.y, l1.x, l1.y};
    }
    if (advance(xp)) x_rows(xp);
    x_load(xp.hf);
    if (advance(wp)) row = row_of(wp);
    w.load(row, wp.hf, wu, units);
    __builtin_amdgcn_sched_barrier(0);  // the loads are under way before the multiply
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const u32x4 op[1] = {xa[u]};
      const float4_t xs = unit_sum<FMT, F16, 1>(op);
      mul_unit<FMT, F16, 1>(o, u, op, xs, acc);
    }
    p.hf += kSplit;
    if (p.hf >= halves) {
      p.hf = part;
      if (!done) done = !next_pairs();
    }
  };
  // Always both: with a way out between them every wait for w0 would also
  // have to hold where w1 has not been loaded after it.  A half past the last
  // tile multiplies what is there and is not used.
  do {
    half(w0);
    half(w1);
  } while (!done);
}

// The same value, unknown to the compiler: what is derived from it is formed where
// it is used, by an instruction or two, and not kept in registers across the loop.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// -------------------------------------------------------------------- down
// A workgroup owns rows of y for every token.  Its waves take the pairs of
// (expert, slice of the columns); each writes its fp32 sums per pair to a
// slot of its own in LDS, and at the end y is put together from the slots in
// the order of the token's experts: no atomics, no second pass over memory.
//
// SPAN = 1: 16 rows, one expert at a time, up to 16 of its pairs.  SPAN = 2: 8
// rows of two experts side by side, up to 8 pairs of each: the matrix tile
// then holds both products on its diagonal (and products of one expert's rows
// with the other's pairs off it, which nobody reads).  Twice the workgroups
// for the same weights, where 16 rows each would leave compute units idle.
//
// Measured, same layers: one token 9.2 us; 64 tokens 75 us, 2.1 TB/s (45 without
// the loads of h, of which a half takes 8 and of weights 2).
template <int FMT, int SPAN>
__global__ __launch_bounds__(kDownWaves* kWave) void k_moe_down(MoeArgs a, int max_slices) {
  constexpr int ROWS = 16 / SPAN;
  extern __shared__ __align__(16) float slots[];  // [slice][pair][ROWS]
  __shared__ Table table;
  __shared__ Stage stages[kDownWaves];
  __shared__ float share[kMoeMaxPairs];  // a pair's weight
  __shared__ bool valid[kMoeMaxPairs];   // and whether it has an expert
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4, wu = lane & 3;
  Stage& stage = stages[wave];
  const int pairs = a.n * a.top_k;
  {
    // all of the table at once: it is read by one round trip, not by three
    const Table* t = static_cast<const Table*>(a.table);
    const int most = pairs < a.experts ? pairs : a.experts;
    if (threadIdx.x == 0) table.active = t->active;
    for (int i = threadIdx.x; i <= most; i += kDownWaves * kWave) {
      if (i < most) table.expert[i] = t->expert[i];
      table.off[i] = t->off[i];
    }
    for (int i = threadIdx.x; i < pairs; i += kDownWaves * kWave) {
      table.pair[i] = t->pair[i];
      const int e = a.ids[i];
      const float w = a.weights[i];
      valid[i] = e >= 0 && e < a.experts;
      share[i] = w;
    }
    __syncthreads();
  }
  const int active = table.active, groups = (active + SPAN - 1) / SPAN;
  const int units = a.inter / 32, halves = (units + 3) / 4;
  // Slice i of a row is its halves i, i + slices, ...: neighbouring waves load
  // the two halves of a super-block, which share its lines, at the same time.
  // As many slices as give every wave work, evenly, and two at least.
  int slices = groups > 0 ? (2 * kDownWaves + groups - 1) / groups : 1;
  slices = slices < 2 ? 2 : slices;
  slices = slices < max_slices ? slices : max_slices;
  slices = slices < halves ? slices : halves;
  const int row0 = blockIdx.x * ROWS, tasks = groups * slices;

  // This lane's expert of a group: of its weight row, and of its pair and
  // its column of the result (the last expert again where there is no second).
  auto slot_of = [&](int group, int half16) {
    if constexpr (SPAN == 1) return group;
    const int s = 2 * group + half16;
    return s < active ? s : active - 1;
  };
  auto row = [&](int group) {
    const int wrow = fresh(lane) >> 2, e = table.expert[slot_of(group, wrow >> 3)];
    return a.down + (static_cast<int64_t>(e) * a.hidden + row0 + (wrow & (ROWS - 1))) * a.down_row_bytes;
  };
  // h of an expert's pairs is stored as operands: per unit of 32 columns the hi
  // parts, then the lo parts, each per lane quarter 16 bytes of every pair.
  // Buffer loads: a lane past the last pair has an offset past the buffer's end,
  // gets zeros and costs the vector cache no access (16 for a load by all lanes,
  // 4 for up to 4 pairs), and the waits stay countable as they would not behind
  // a branch.  h is at most 2 GB (kMoeMaxDim).
  const auto hbuf = __builtin_amdgcn_make_buffer_rsrc(a.h, 0, static_cast<uint32_t>(pairs) * static_cast<uint32_t>(a.inter) * 4u,
                                                      0x00027000);
  uint32_t h = 0, hstep = 0;  // offset; between the parts of a unit
  auto h_rows = [&](int group, int c0) {
    const int slot = slot_of(group, r >> 3);
    uint32_t first = table.off[slot], count = table.off[slot + 1] - first;
    if constexpr (SPAN == 1) {
      first = __builtin_amdgcn_readfirstlane(first);
      count = __builtin_amdgcn_readfirstlane(count);
    }
    const uint32_t at = c0 + (r & (ROWS - 1));
    h = at < count ? first * static_cast<uint32_t>(a.inter) * 4u + (q * count + at) * 16u : 0x80000000u;
    hstep = count * 64;
  };
  auto h_load = [&](int hf, u32x4(&to)[4][2]) {
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const uint32_t at = 2 * hstep * (FMT != QBLK_Q4_0 || 4 * hf + u < units ? 4 * hf + u : units - 1);
      const uint32_t v = SPAN == 1 ? h : h + at, s = SPAN == 1 ? at : 0;
#pragma unroll
      for (int part = 0; part < 2; part++)
        to[u][part] = SPAN == 1 ? __builtin_amdgcn_raw_buffer_load_b128(hbuf, v, s + part * hstep, 0)
                                : __builtin_amdgcn_raw_buffer_load_b128(hbuf, v + part * hstep, s, 0);
    }
  };
  // A place in the sequence of halves that this wave multiplies: its tasks,
  // each group's pairs ROWS at a time, the slice's halves.  At the end it
  // stays at the last task (loaded, not used).
  struct Place {
    int task, group, slice, count, c0, hf;
  };
  auto at_task = [&](Place& p, int task) {
    p.task = task;
    p.group = task / slices;
    p.slice = task - p.group * slices;
    p.count = 0;  // the larger, of two experts
#pragma unroll
    for (int i = 0; i < SPAN; i++) {
      const int slot = slot_of(p.group, i);
      const int c = __builtin_amdgcn_readfirstlane(table.off[slot + 1] - table.off[slot]);
      p.count = c > p.count ? c : p.count;
    }
    p.c0 = 0;
    p.hf = p.slice;
  };
  auto advance = [&](Place& p) {  // whether the task or the pairs changed
    p.hf += slices;
    if (p.hf < halves) return false;
    p.hf = p.slice;
    p.c0 += ROWS;
    if (p.c0 >= p.count) at_task(p, p.task + kDownWaves < tasks ? p.task + kDownWaves : p.task);
    return true;
  };
  if (wave < tasks) {
    Place p, wp, hp;  // what is multiplied now; of the weights, two halves on; of h, one half on
    at_task(p, wave);
    wp = hp = p;
    const uint8_t* w = row(wp.group);
    Unit<FMT> w0, w1;
    u32x4 h0[4][2], h1[4][2];
    // (in the loop's order: the waits in it count what was issued since)
    w0.load(w, wp.hf, wu, units);
    __builtin_amdgcn_sched_barrier(0);
    h_rows(hp.group, hp.c0);
    h_load(hp.hf, h0);
    if (advance(wp)) w = row(wp.group);
    __builtin_amdgcn_sched_barrier(0);
    w1.load(w, wp.hf, wu, units);
    __builtin_amdgcn_sched_barrier(0);
    float4_t acc = {0, 0, 0, 0};
    bool done = false;
    // one half; the weights are emptied into LDS and loaded anew in place, h
    // changes places (a copy between register sets would wait for its loads)
    auto half = [&](Unit<FMT>& wn, u32x4(&ha)[4][2], u32x4(&hn)[4][2]) {
      const Operand so = to_operand(wn, p.hf, units, stage);
      if (advance(hp)) h_rows(hp.group, hp.c0);
      h_load(hp.hf, hn);
      if (advance(wp)) w = row(wp.group);
      wn.load(w, wp.hf, wu, units);
      __builtin_amdgcn_sched_barrier(0);  // the loads are under way before the multiply
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const float4_t xs = unit_sum<FMT, false, 2>(ha[u]);
        mul_unit<FMT, false, 2>(so, u, ha[u], xs, acc);
      }
      p.hf += slices;
      if (p.hf < halves) return;
      // lane (column r, quarter q): pairs 4q .. 4q+3 of the tile; of two experts
      // the first has the tile's first 8 pairs and columns
      const int l = fresh(lane), col = l & 15, quarter = l >> 4;
      if (!done && (SPAN == 1 || ((quarter >> 1) == (col >> 3) && 2 * p.group + (col >> 3) < active))) {
        const int slot = slot_of(p.group, col >> 3);
        const int first = table.off[slot], count = table.off[slot + 1] - first;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int at = p.c0 + ((4 * quarter + i) & (ROWS - 1));
          if (at < count) slots[(p.slice * pairs + table.pair[first + at]) * ROWS + (col & (ROWS - 1))] = acc[i];
        }
      }
      acc = float4_t{0, 0, 0, 0};
      p.hf = p.slice;
      p.c0 += ROWS;
      if (p.c0 < p.count) return;
      if (p.task + kDownWaves < tasks)
        at_task(p, p.task + kDownWaves);
      else
        done = true;
    };
    // always both, as in k_moe_up; a half past the last task is not used
    do {
      half(w0, h0, h1);
      half(w1, h1, h0);
    } while (!done);
  }
  __syncthreads();
  // the slices of a pair, then the pairs of a token, each in order
  for (int o = threadIdx.x; o < pairs * ROWS; o += kDownWaves * kWave) {
    const int p = o / ROWS;
    float sum = 0.0f;
#pragma unroll 4
    for (int s = 0; s < slices; s++) sum += slots[s * pairs * ROWS + o];
    slots[o] = valid[p] ? share[p] * sum : 0.0f;
  }
  __syncthreads();
  for (int o = threadIdx.x; o < a.n * ROWS; o += kDownWaves * kWave) {
    const int t = o / ROWS, rr = o & (ROWS - 1);
    float y = 0.0f;
#pragma unroll 4
    for (int j = 0; j < a.top_k; j++) y += slots[(t * a.top_k + j) * ROWS + rr];
    const int64_t at = static_cast<int64_t>(t) * a.hidden + row0 + rr;
    if (a.yt == QBLK_F32)
      static_cast<float*>(a.y)[at] = y;
    else
      static_cast<uint16_t*>(a.y)[at] = a.yt == QBLK_F16 ? f32_to_f16_bits(y) : f32_to_bf16_bits(y);
  }
}

template <int FMT, int SPAN>
hipError_t down(const MoeArgs& a, hipStream_t s) {
  const int pairs = a.n * a.top_k;
  const int max_slices = kMoeMaxPairs / pairs < 2 * kDownWaves ? kMoeMaxPairs / pairs : 2 * kDownWaves;
  const size_t lds = static_cast<size_t>(max_slices) * pairs * (64 / SPAN);
  const unsigned grid = static_cast<unsigned>(a.hidden / (16 / SPAN));
  log_launch("moe down fmt=%d n=%d top_k=%d experts=%d hidden=%d inter=%d grid=%u rows=%d slices<=%d", FMT, a.n, a.top_k,
             a.experts, a.hidden, a.inter, grid, 16 / SPAN, max_slices);
  k_moe_down<FMT, SPAN><<<grid, kDownWaves * kWave, lds, s>>>(a, max_slices);
  return hipGetLastError();
}

template <int FMT>
hipError_t run(const MoeArgs& a, hipStream_t s) {
  const int64_t reach = static_cast<int64_t>(a.n) * a.top_k < a.experts ? static_cast<int64_t>(a.n) * a.top_k : a.experts;
  const int64_t tasks = reach * (a.inter / 16);
  const int64_t most = static_cast<int64_t>(cu_count()) * 2;  // what fits at once, by registers
  const unsigned grid = static_cast<unsigned>(tasks < most ? tasks : most);
  if (a.xt == QBLK_F16)
    k_moe_up<FMT, true><<<grid, kUpWaves * kWave, 0, s>>>(a);
  else
    k_moe_up<FMT, false><<<grid, kUpWaves * kWave, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // 8 rows of two experts a workgroup where 16 rows leave compute units idle
  // (hidden 2048, inter 1024, us, whole call in a graph, 8 rows and 16; 64 experts,
  // 8 of them a token: one token Type 0 20.8 and 23.2, Type 1 21.2 and 23.0, Q4_K
  // 20.9 and 22.6, Q4_0 22.8 and 25.3; 16 tokens 78 and 103, 78 and 101, 77 and 98,
  // 87 and 115; 64 tokens 128 and 135, 129 and 136, 124 and 131, 135 and 142; 16
  // experts, 2 of them, one token, Type 0: 13.5 and 15.6).  Where they do not, half of
  // the tile's products are for nothing (hidden 4096, inter 2048, 4 of 32 experts:
  // one token Type 0 31.7 and 26.6, Type 1 31.2 and 25.9; 16 tokens 144 and 136, 145
  // and 135; 64 tokens 238 and 180, 242 and 183).
  return a.hidden / 16 < cu_count() ? down<FMT, 2>(a, s) : down<FMT, 1>(a, s);
}

}  // namespace

int64_t moe_table_bytes() { return static_cast<int64_t>((sizeof(Table) + 255) / 256 * 256); }

hipError_t launch_moe(int fmt, const MoeArgs& all, int64_t n, hipStream_t s) {
  const int64_t per = kMoeMaxPairs / all.top_k;
  const int64_t ybytes = all.yt == QBLK_F32 ? 4 : 2;
  for (int64_t t0 = 0; t0 < n; t0 += per) {
    MoeArgs a = all;
    a.n = static_cast<int>(n - t0 < per ? n - t0 : per);
    a.x = static_cast<const uint8_t*>(all.x) + t0 * all.hidden * 2;
    a.y = static_cast<uint8_t*>(all.y) + t0 * all.hidden * ybytes;
    if (all.logits != nullptr) a.logits = all.logits + t0 * all.experts;
    a.ids = all.ids + t0 * all.top_k;
    a.weights = all.weights + t0 * all.top_k;
    hipError_t e;
    switch (fmt) {
      case QBLK_Q4_0: e = run<QBLK_Q4_0>(a, s); break;
      case QBLK_SB4: e = run<QBLK_SB4>(a, s); break;
      case QBLK_SB4_AFFINE: e = run<QBLK_SB4_AFFINE>(a, s); break;
      default: e = run<QBLK_Q4_K>(a, s); break;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qblk
