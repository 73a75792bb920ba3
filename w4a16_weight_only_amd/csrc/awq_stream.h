// Streaming of packed weights for few rows: the part that the kernels of routed experts, of a whole
// routed layer and of one dense weight have in common.
//
// A wave takes up to 16 or 32 rows of x, 256 columns and a run of 32-row k-steps.  On
// v_mfma_f32_16x16x32 lane l = 16 q + c loads words 2 c, 2 c + 1 of rows 8 q .. 8 q + 7 (16
// lanes: 128 contiguous bytes of a row) and unpacks them into operands of exact integers, 16
// columns x 8 rows; its rows of x are rows l % 16 (and 16 + l % 16: an operand unpacked once
// serves both blocks of 16 rows) of the entry.
// q - z; in bfloat16, which has no packed addition on this chip, by way of fp32.
// The running sums are in units of the current group's scale u: a group boundary multiplies
// them by u / u', exactly 1 where the scale stays the same (u times its reciprocal may be a step
// off, always to one side, which equal groups would add up).  (A second set of 64 accumulator
// registers, scaled group by group, spills.)
// A scale of zero cannot be a unit: the unit stays, and the column's operands become zeros, by
// its codes replaced with its zero code.  That is rare, and outside the MFMAs' code: a second copy
// of those makes the compiler move accumulators about.
// A ring of two k-steps is in flight, and with each a group's zeros and scales where one begins.
// bfloat16 sums of 32 rows leave no registers for two sets of those: there the next group's are
// asked for when a group begins (both ways: 64 tokens through 8 x 4096 -> 14336 209 -> 187 us in
// bfloat16, which had spilled; one token through 64 x 2048 -> 1408 25.0 -> 27.0 in fp16).
// Of the waves of a SIMD the oldest goes first, and ends far ahead of the others, which then are too few to keep
// the memory busy.  So a wave's priority falls where a half, a quarter and an eighth of its run are left: who is
// behind goes first, and all end together (without / with, us in a graph: one token through 8 x 4096 -> 14336, whose
// gated product's waves ended 10 us apart and now 1.3, 63.4 / 58.7; 16 tokens 169 / 160; 7 tokens through 64 x
// 2048 -> 1408 68.3 / 64.7; 19 x 4096 -> 2 x 11008 29.6 / 28.1; 1 x 8192 -> 28672 32.0 / 30.9).
// A decoding step's h may be two terms, h rounded and what that left out (REST): a second MFMA
// on the same operand, whose result's error is y's rounding alone (with one term 1.3 to 1.5 times
// that).
#pragma once

#include "awq_device.h"
#include "awq_kernels.h"

namespace awq {
namespace stream {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kPF = 2;           // k-steps in flight per wave
constexpr int kYld = kExpertStreamCols + 4;  // floats of a staged output row

// Entry v of a lane's 16 columns: word v / 8, byte (v / 2) % 4, nibble v % 2.
__device__ constexpr int col_of(int v) { return (v & 1) ? hi_col((v >> 1) & 3) : lo_col((v >> 1) & 3); }

template <int RB, bool REST>
struct Step {
  u32x2 w[8];        // rows 8 q .. 8 q + 7
  half8v x[RB];      // x[row][8 q ..], a row of each block
  half8v rest[REST ? RB : 1];
};

// Codes to (code - zero) in bfloat16, exact, by way of fp32: the nibbles in bits 0-3 (or 4-7) of a
// word's halves are the subnormal halves q 2^-24 (or q 2^-20), so that one mixed-precision fma
// makes q - z of each; two rows' are then narrowed together.  2.1 vector instructions a weight,
// where fp16's 1024 + q takes 1.25 with packed additions.  (A bfloat16 128 + q takes 1.0, but leaves
// x . (128 + q) - (128 + z) x . 1 to be formed: partial sums with four to five bits fewer, and NaN
// where an infinite x gives an infinity.  That / this, us: gate_up of 45 tokens 64 x 2048 -> 1408
// 61 / 64, mlp of 16 tokens 8 x 4096 -> 14336 157 / 163, of 256 tokens 64 x 2048 -> 1408 170 / 165.)
__device__ __forceinline__ uint32_t minus_zero_bf16(uint32_t a, uint32_t b, int half, float scale, float z) {
  return pack_bf16x2(fmaf((float)as_h2(a)[half], scale, -z), fmaf((float)as_h2(b)[half], scale, -z));
}

// The 16 RB MFMAs of a k-step.  zs: per column, fp16: -(1024 + z) or -(64 + z) twice (low or high
// nibble); bfloat16: z as a float.
template <bool BF16, int RB, bool REST>
__device__ __forceinline__ void multiply(const Step<RB, REST>& st, const uint32_t (&zs)[16], const UnpackConsts& uk,
                                         floatx4 (&part)[RB][16]) {
  auto mfma = [](const half8v& x, const u32x4& w, const floatx4& c) {
    if constexpr (BF16)
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, w), c, 0,
                                                     0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, __builtin_bit_cast(half8v, w), c, 0, 0, 0);
  };
  auto column = [&](int v, const u32x4& op) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      part[rb][v] = mfma(st.x[rb], op, part[rb][v]);
      if constexpr (REST) part[rb][v] = mfma(st.rest[rb], op, part[rb][v]);
    }
  };
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if constexpr (BF16) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {  // nibbles 2 s, 2 s + 1 and, in the upper half, 2 s + 4, 2 s + 5
        u32x4 op[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t a = st.w[2 * p][w] >> (8 * s), b = st.w[2 * p + 1][w] >> (8 * s);
          const uint32_t al = a & 0x000F000Fu, bl = b & 0x000F000Fu, ah = a & 0x00F000F0u, bh = b & 0x00F000F0u;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int v = 8 * w + 2 * s + 4 * half;
            op[2 * half][p] = minus_zero_bf16(al, bl, half, 0x1p24f, __builtin_bit_cast(float, zs[v]));
            op[2 * half + 1][p] = minus_zero_bf16(ah, bh, half, 0x1p20f, __builtin_bit_cast(float, zs[v + 1]));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) column(8 * w + 2 * s + 4 * (i >> 1) + (i & 1), op[i]);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        u32x4 lo, hi;
        const int il = 8 * w + 2 * t, ih = il + 1;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t wa = st.w[2 * p][w], wb = st.w[2 * p + 1][w];
          uint32_t pb;
          if (t == 0) pb = pair_byte<0>(wa, wb);
          else if (t == 1) pb = pair_byte<1>(wa, wb);
          else if (t == 2) pb = pair_byte<2>(wa, wb);
          else pb = pair_byte<3>(wa, wb);
          lo[p] = as_u32(lo_minus_zero(pb, as_h2(zs[il]), uk));
          hi[p] = as_u32(hi_minus_zero(pb, as_h2(zs[ih]), uk));
        }
        column(il, lo);
        column(ih, hi);
      }
    }
  }
}

// Zeros and scales of a group, for a lane's two words.
struct GroupData {
  u32x2 z;
  half8v s[2];
};

// Rows of a workgroup's entry: its expert, how many, and their slots (LDS).
struct Entry {
  int expert, rows;
};

// Set bits of mask below this lane.
__device__ __forceinline__ int bits_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// Entries of at most 64 slots, ranked by each wave (lane l: slot l): the slots of an expert,
// in order, in blocks of ROWS; entries in the order of their first slot.
// A lane's mask of slots with its expert comes from one ballot per bit of the id (a loop over
// the slots took 5 us of 64 slots' 20).
struct Ranks {
  int rank;        // among the lower slots of the same expert
  uint64_t leads;  // slots that begin an entry
  int entries;
  bool routed;
};
template <int ROWS>
__device__ __forceinline__ Ranks rank_slots(int id, int E) {
  const bool routed = id >= 0 && id < E;
  uint64_t same = __ballot(routed);
#pragma unroll
  for (int b = 0; b < 10; ++b) {  // E <= 1024
    const uint64_t set = __ballot((id >> b) & 1);
    same &= ((id >> b) & 1) ? set : ~set;
  }
  const int rank = bits_below(same);
  const uint64_t leads = __ballot(routed && rank % ROWS == 0);
  return Ranks{rank, leads, (int)__builtin_popcountll(leads), routed};
}
// The entry's expert and rows, its slots to LDS (every wave writes the same); rows 0: no such entry.
template <int ROWS>
__device__ __forceinline__ Entry entry_of(const Ranks& k, int id, int entry, int lane, int32_t* slots) {
  const uint64_t found = __ballot(((k.leads >> lane) & 1) != 0 && bits_below(k.leads) == entry);
  if (found == 0) return Entry{0, 0};
  const int at = __builtin_ctzll(found);
  const int expert = __builtin_amdgcn_readlane(id, at);
  const int first = __builtin_amdgcn_readlane(k.rank, at);
  const bool mine = k.routed && id == expert && k.rank >= first && k.rank < first + ROWS;
  if (mine) slots[k.rank - first] = lane;
  return Entry{expert, (int)__builtin_popcountll(__ballot(mine))};
}

// A wave's part of a product: the weight of one expert (NW packed words a row, K rows), the lane's
// first word column wc, byte offsets of its rows of x (at k = 8 (lane / 16)), k-steps kb .. ke.
template <int RB>
struct Share {
  const uint32_t *qweight, *qzeros;
  const uint16_t* scales;
  int NW, K, g, wc;
  const uint16_t *x, *x_rest;
  uint32_t x_off[RB];
  int kb, ke;
};

struct Now {
  __device__ void operator()() const {}
};

// 16 bytes as every XCD sees them alike.
__device__ __forceinline__ half8v device_load(const uint16_t* base, uint64_t at) {
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), (short)0, -1, 0x00020000);
  return __builtin_bit_cast(half8v, __builtin_amdgcn_raw_buffer_load_b128(rs, (uint32_t)at, 0, kCpolDevice));
}

struct NoSource {};

// part[rb][v] * unit: sums of entry v's column and four rows (4 (lane / 16) ..) of block rb.
// ready(): called by every wave before anything of x is read, behind the first loads of the weights.
// source(k, rest), if given, is x[k ..] (or the second term's) of every row in place of memory.
template <bool BF16, int RB, bool REST, typename Ready, typename Source = NoSource>
__device__ __forceinline__ void stream_sums(const Share<RB>& s, Ready ready, floatx4 (&part)[RB][16],
                                            half8v (&unit)[2], Source source = Source{}) {
  constexpr bool kSource = !__is_same(Source, NoSource);
  constexpr bool kWaits = !__is_same(Ready, Now);
  const int q = (threadIdx.x & 63) >> 4;
  const int K = s.K, NW = s.NW, wc = s.wc, gsteps = s.g / 32, kb = s.kb, ke = s.ke;
  const uint32_t *qzeros = s.qzeros;
  const uint16_t* scales = s.scales;
  const uint32_t row_bytes = (uint32_t)NW * 4u;
  const uint32_t w_off = (uint32_t)(8 * q) * row_bytes + (uint32_t)wc * 4u;
  const __amdgpu_buffer_rsrc_t wrs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint32_t*>(s.qweight), (short)0, (int)(row_bytes * (uint32_t)K), 0x00020000);

  // Group data: one set for each k-step in flight, or one in all.
  constexpr bool kOneSet = BF16 && RB == 2;
  // Loads of steps past a run's end are made as well, which lets a step's loads stay in flight
  // during the one before (without / with: mlp of 256 tokens 64 x 2048 -> 1408, g 64, bfloat16 181 /
  // 171 us, of 128 tokens 8 x 4096 -> 14336 304 / 283; one block of rows 86 / 88 us for 16 tokens of
  // the first and fp16's two blocks 152 / 159 for 256: there the loads of short runs cost more).
  constexpr bool kAlways = BF16 && RB == 2;
  GroupData data[kOneSet ? 1 : kPF];
  // The group loaded next and entered next, and the k-steps they begin with.
  int load_group = kb / gsteps, load_at = kb, enter_at = kb;
  const int first_end = (load_group + 1) * gsteps;
  auto fetch = [&](GroupData& d) {
    const int64_t at = (int64_t)load_group * NW + wc;
    d.z = *reinterpret_cast<const u32x2*>(qzeros + at);
    d.s[0] = *reinterpret_cast<const half8v*>(scales + 8 * at);
    d.s[1] = *reinterpret_cast<const half8v*>(scales + 8 * at + 8);
    load_at = ++load_group * gsteps;
  };
  // Loads of a k-step.  Group data goes first: a wait for the weights counts back from the newest
  // load, and must not have to allow for loads that may not have been made.  kAlways: for the same
  // reason the loads of steps past the run are made too; the weights' offset is the buffer's end
  // there, past which nothing is read, and x is read at k = 0 again.
  auto issue_weights = [&](Step<RB, REST>& st, int slot, int ks) {
    const bool live = !kAlways || ks < ke;
    if (!kOneSet && live && ks == load_at) fetch(data[kOneSet ? 0 : slot]);
    const uint32_t r0 = live ? (uint32_t)ks * 32u : 0u;
    const uint32_t at_w = live ? w_off : row_bytes * (uint32_t)K, row_step = live ? row_bytes : 0u;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      st.w[r] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(wrs, at_w, (r0 + r) * row_step, 2));
  };
  auto issue_x = [&](Step<RB, REST>& st, int ks) {
    const uint32_t r0 = !kAlways || ks < ke ? (uint32_t)ks * 32u : 0u;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      [[maybe_unused]] const uint64_t at = (uint64_t)s.x_off[rb] + r0 * 2u;
      if constexpr (kSource) {
        st.x[rb] = source((int)r0 + 8 * q, false);
        if constexpr (REST) st.rest[rb] = source((int)r0 + 8 * q, true);
        continue;
      }
      if constexpr (kWaits) {  // written by this kernel's other workgroups
        st.x[rb] = device_load(s.x, at);
        if constexpr (REST) st.rest[rb] = device_load(s.x_rest, at);
        continue;
      }
      st.x[rb] = *reinterpret_cast<const half8v*>(reinterpret_cast<const char*>(s.x) + at);
      if constexpr (REST) st.rest[rb] = *reinterpret_cast<const half8v*>(reinterpret_cast<const char*>(s.x_rest) + at);
    }
  };
  auto issue = [&](Step<RB, REST>& st, int slot, int ks) {
    issue_weights(st, slot, ks);
    issue_x(st, ks);
  };

  const UnpackConsts uk = unpack_consts();
  uint32_t zs[16];
  // unit: the columns' current units
  u32x2 zw = {0u, 0u};     // the current group's zero codes
  u32x2 nil = {0u, 0u};    // nibbles of columns whose scale is zero in the current group
  bool any_nil = false;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) part[rb][v] = floatx4{0.f, 0.f, 0.f, 0.f};
    zs[v] = 0;
    unit[v >> 3][v & 7] = (_Float16)1.f;  // (columns in order)
  }
  // A group begins: the sums so far change units (there are none when the run begins).  A scale of
  // zero is looked for in pairs of halves, and dealt with column by column where there is one (every
  // column asking for itself: gate_up of 45 tokens 64 x 2048 -> 1408, g 64, bfloat16 68 / 63.7 us).
  auto enter = [&](const GroupData& d, bool begin) {
    half8v now[2] = {d.s[0], d.s[1]};
    nil = u32x2{0u, 0u};
    uint32_t zero = 0;  // a half of zero, either sign: the halves' borrow trick
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t s = __builtin_bit_cast(u32x4, now[w])[i] & 0x7FFF7FFFu;
        zero |= (s - 0x00010001u) & ~s & 0x80008000u;
      }
    any_nil = __builtin_amdgcn_ballot_w64(zero != 0) != 0;
    if (any_nil) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const bool none = now[v >> 3][col_of(v)] == (_Float16)0.f;
        now[v >> 3][col_of(v)] = none ? unit[v >> 3][col_of(v)] : now[v >> 3][col_of(v)];
        nil[v >> 3] |= none ? 0xFu << (4 * (v & 7)) : 0u;  // entry v is nibble v % 8 of its word
      }
    }
    if (!begin) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const float o = (float)unit[v >> 3][col_of(v)], n = (float)now[v >> 3][col_of(v)];
        const float ratio = n == o ? 1.f : o * __builtin_amdgcn_rcpf(n);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) part[rb][v] *= ratio;
      }
    }
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      if constexpr (BF16) {
        const uint32_t z = (v & 1 ? d.z[v >> 3] >> 4 : d.z[v >> 3]) & 0x0F0F0F0Fu;
        zs[v] = __builtin_bit_cast(uint32_t, (float)((z >> (8 * ((v & 7) >> 1))) & 0xFFu));
      } else {
        const uint32_t z = zero_code(d.z[v >> 3], col_of(v));
        const uint32_t h = (v & 1) ? (0xD400u | (z << 4)) : (0xE400u | z);  // -(64 + z), -(1024 + z)
        zs[v] = h | (h << 16);
      }
    }
    unit[0] = now[0];
    unit[1] = now[1];
    zw = d.z;
    enter_at = begin ? first_end : enter_at + gsteps;
  };
  Step<RB, REST> ring[kPF];
  if (kOneSet && kb < ke) fetch(data[0]);
  if constexpr (kWaits) {
#pragma unroll
    for (int j = 0; j < kPF; ++j)
      if (kAlways || kb + j < ke) issue_weights(ring[j], j, kb + j);
    ready();
#pragma unroll
    for (int j = 0; j < kPF; ++j)
      if (kAlways || kb + j < ke) issue_x(ring[j], kb + j);
  } else {
#pragma unroll
    for (int j = 0; j < kPF; ++j) {
      if (kAlways || kb + j < ke) issue(ring[j], j, kb + j);
      if constexpr (kAlways) __builtin_amdgcn_sched_barrier(0);
    }
  }
  int level = 3, fall = ke - (ke - kb) / 2;
  __builtin_amdgcn_s_setprio(3);
  for (int base = kb; base < ke; base += kPF) {
    if (base >= fall) {
      fall = ke - (ke - fall) / 2;
      --level;
      if (level == 2) __builtin_amdgcn_s_setprio(2);
      else if (level == 1) __builtin_amdgcn_s_setprio(1);
      else __builtin_amdgcn_s_setprio(0);
    }
#pragma unroll
    for (int j = 0; j < kPF; ++j) {
      const int ks = base + j;
      if ((kAlways && j == 0) || ks < ke) {
        const bool begins = ks == enter_at;
        if (begins) enter(data[kOneSet ? 0 : j], ks == kb);
        if (any_nil) {
#pragma unroll
          for (int r = 0; r < 8; ++r) ring[j].w[r] = (ring[j].w[r] & ~nil) | (zw & nil);
        }
        multiply<BF16>(ring[j], zs, uk, part);
        if (kOneSet && begins && load_at < ke) fetch(data[0]);
        if (!kAlways && ks + kPF < ke) issue(ring[j], j, ks + kPF);
      }
      if (kAlways) issue(ring[j], j, ks + kPF);
    }
  }
  __builtin_amdgcn_s_setprio(0);
}

// Waves along K of a workgroup of WAVES: all, or gated every other one (even ones the gate's columns,
// odd ones the up projection's).
template <bool GATED, int WAVES = kWaves>
constexpr int kParts = GATED ? WAVES / 2 : WAVES;

// The sums of a column in R adjacent rows (4, or 1 where there is one row in all).
template <int R>
struct RowsOf {
  using type = floatx4;
};
template <>
struct RowsOf<1> {
  using type = float;
};
template <int R>
using Rows = typename RowsOf<R>::type;
template <int R>
__device__ __forceinline__ float row_of(const Rows<R>& v, int r) {
  if constexpr (R == 1) return v;
  else return v[r];
}
// Slots per thread (see wave_sums).
template <int RL, int WAVES>
constexpr int kSlots = (16 * RL + 64 * WAVES - 1) / (64 * WAVES);

// The waves' sums of one block of 16 rows, over LDS: sum k of thread i, slot s = i + 64 WAVES k (of
// 16 RL), is column entry (s / 16) % 16 of word pair s % 16, rows 4 (s / 256) ...  Only RL lanes' rows are
// kept.  The caller sees to it that nothing else uses red before and after (barriers).
template <bool GATED, int RL, int WAVES = kWaves, int R = 4>
__device__ __forceinline__ void wave_sums(Rows<R> (&red)[WAVES][16][RL], const floatx4 (&part)[16],
                                          const half8v (&unit)[2],
                                          Rows<R> (&sum)[kSlots<RL, WAVES>][GATED ? 2 : 1]) {
  static_assert(R == 4 || RL == 16, "one row is in the first 16 lanes");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (lane < RL) {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const float u = (float)unit[v >> 3][col_of(v)];
      if constexpr (R == 1) red[wave][v][lane] = part[v][0] * u;
      else red[wave][v][lane] = part[v] * u;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSlots<RL, WAVES>; ++k) {
    const int i = 64 * WAVES > 16 * RL ? min(tid, 16 * RL - 1) : tid + k * 64 * WAVES;
    const int v = (i >> 4) & 15, ln = (i >> 8) * 16 + (i & 15);
#pragma unroll
    for (int hf = 0; hf < (GATED ? 2 : 1); ++hf) {
      Rows<R> a = red[hf][v][ln];
#pragma unroll
      for (int w = 1; w < kParts<GATED, WAVES>; ++w) a += red[GATED ? 2 * w + hf : w][v][ln];
      sum[k][hf] = a;
    }
  }
}
// R floats to and from where every XCD sees the same.
template <int R>
__device__ __forceinline__ void device_store(const __amdgpu_buffer_rsrc_t& rs, uint32_t at, const Rows<R>& v) {
  if constexpr (R == 1) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), rs, at, 0, kCpolDevice);
  else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, at, 0, kCpolDevice);
}
template <int R>
__device__ __forceinline__ Rows<R> device_read(const __amdgpu_buffer_rsrc_t& rs, uint32_t at) {
  if constexpr (R == 1) return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, kCpolDevice));
  else return __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, kCpolDevice));
}
// sum[i] = sum in order of the n Rows at at(split, i), for COUNT of them side by side: the loads of a
// few splits of all of them go out together (a join is a matter of latency: 19 rows of 4096 -> 2 x 11008, four
// splits, one sum after another / together: 7 / 2.5 us of the call).
template <int R, int COUNT, typename At>
__device__ __forceinline__ void device_sums(const __amdgpu_buffer_rsrc_t& rs, int n, At at, Rows<R> (&sum)[COUNT]) {
  constexpr int B = COUNT * R >= 32 ? 2 : COUNT * R >= 8 ? 4 : 8;
#pragma unroll
  for (int i = 0; i < COUNT; ++i) sum[i] = Rows<R>{};
  int s0 = 0;
  for (; s0 + B <= n; s0 += B) {
    Rows<R> v[COUNT][B];
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
#pragma unroll
      for (int j = 0; j < B; ++j) v[i][j] = device_read<R>(rs, at(s0 + j, i));
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
#pragma unroll
      for (int j = 0; j < B; ++j) sum[i] += v[i][j];
  }
  if (s0 < n) {  // the last few: those past the last read it again and are dropped
    Rows<R> v[COUNT][B - 1];
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
#pragma unroll
      for (int j = 0; j < B - 1; ++j) v[i][j] = device_read<R>(rs, at(min(s0 + j, n - 1), i));
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
#pragma unroll
      for (int j = 0; j < B - 1; ++j)
        if (s0 + j < n) sum[i] += v[i][j];
  }
}

// Column within the tile of slot s (see wave_sums), its first row within the block.
__device__ __forceinline__ int slot_col(int s) {
  const int v = (s >> 4) & 15;
  return 8 * (2 * (s & 15) + (v >> 3)) + col_of(v);
}
__device__ __forceinline__ int slot_row(int s) { return 4 * (s >> 8); }

}  // namespace stream
}  // namespace awq
