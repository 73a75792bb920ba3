// Few rows per routed expert: bandwidth-bound streaming of the experts' packed weights.
//
// A workgroup takes up to 16 or 32 routed rows of one expert (an entry), 256 columns (gated:
// the same 256 of both halves) and one K split.  Its four waves each take a run of 32-row
// k-steps; gated, even waves take the gate's columns and odd ones the up projection's.  On
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
// A decoding step's h may be two terms, h rounded and what that left out (REST): a second MFMA
// on the same operand, whose result's error is y's rounding alone (with one term 1.3 to 1.5 times
// that).
// The waves meet in LDS.  With one split a gated workgroup writes h; otherwise fp32 sums
// [split][slot][column] leave for the next kernel, which adds the splits in order.
//
// Which rows a workgroup has: up to 64 slots, every wave ranks them itself (one slot per
// lane); above, the table of launch_moe_align in blocks of 16 or 32 rows.
//
// Bound by HBM from a few rows on (medians of 27 calls): one token's two experts of 4096 -> 2 x
// 14336, 117 MB, 29.7 us (4.0 TB/s; a copy of 2 GiB 4.96, of which half are writes); 19 rows of
// 14336 -> 4096 over 8 experts, 235 MB, 48.2 us (4.9).  By latency below that (8 slots of 2048 -> 2 x
// 1408, 23 MB, 12.3 us), and by unpacking beside HBM at 32 rows and in bfloat16 (16 tokens' 8 x
// 4096 -> 2 x 14336, 470 MB, 115 us, 4.1 TB/s; 107 at best).
#include "awq_device.h"
#include "awq_kernels.h"

namespace awq {

namespace {

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
// in order, in blocks of ROWS; entries in the order of their first slot.  rows 0: no such entry.
// A lane's mask of slots with its expert comes from one ballot per bit of the id (a loop over
// the slots took 5 us of 64 slots' 20).
template <int ROWS>
__device__ __forceinline__ Entry rank_entry(const int32_t* ids, int S, int E, int entry, int lane, int32_t* slots) {
  const int id = lane < S ? ids[lane] : -1;
  const bool routed = id >= 0 && id < E;
  const uint64_t live = __ballot(routed);
  uint64_t same = live;
#pragma unroll
  for (int b = 0; b < 10; ++b) {  // E <= 1024
    const uint64_t set = __ballot((id >> b) & 1);
    same &= ((id >> b) & 1) ? set : ~set;
  }
  const int rank = bits_below(same);  // among the lower slots of the same expert
  const bool lead = routed && rank % ROWS == 0;
  const uint64_t leads = __ballot(lead);
  const uint64_t found = __ballot(lead && bits_below(leads) == entry);
  if (found == 0) return Entry{0, 0};
  const int at = __builtin_ctzll(found);
  const int expert = __builtin_amdgcn_readlane(id, at);
  const int first = __builtin_amdgcn_readlane(rank, at);
  const bool mine = routed && id == expert && rank >= first && rank < first + ROWS;
  if (mine) slots[rank - first] = lane;  // every wave writes the same
  return Entry{expert, (int)__builtin_popcountll(__ballot(mine))};
}

}  // namespace

// RB: blocks of 16 rows.  RL: lanes whose sums are kept, 16 per four rows (an entry of one block
// never has more than RL / 4 rows).  REST: rows of two terms, x and x_rest.
template <bool GATED, bool BF16, int RB, int RL, bool REST>
__global__ __launch_bounds__(kThreads, 2) void expert_stream_kernel(const ExpertProduct p, int by_xcd, int tiles,
                                                                    int splits, int steps,
                                                                    const int32_t* __restrict__ sorted,
                                                                    const int32_t* __restrict__ table) {
  constexpr int PARTS = GATED ? kWaves / 2 : kWaves;  // waves along K
  __shared__ union {
    floatx4 red[kWaves][16][RL];  // [wave][column entry][lane]
    float ys[RL / 4][GATED ? 2 : 1][kYld];
  } sh;
  __shared__ int32_t slots[16 * RB];

  // Block order: splits fastest, then column tiles, then entries; by_xcd: eight entries
  // abreast, so that an entry's blocks share an XCD.
  const int of_entry = tiles * splits;
  const int group = by_xcd ? blockIdx.x / (8 * of_entry) : 0;
  const int in_group = blockIdx.x - group * 8 * of_entry;
  const int at_entry = by_xcd ? in_group >> 3 : in_group % of_entry;
  const int entry = by_xcd ? 8 * group + (in_group & 7) : in_group / of_entry;
  const int split = at_entry % splits;
  const int tile = at_entry / splits;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, c = lane & 15;
  Entry en;
  if (table == nullptr) {
    en = rank_entry<16 * RB>(p.ids, p.S, p.E, entry, lane, slots);
  } else {
    en.expert = table[4 * entry];
    en.rows = en.expert < 0 ? 0 : table[4 * entry + 2];
    if (lane < en.rows) slots[lane] = sorted[table[4 * entry + 1] + lane];
  }
  if (en.rows == 0) return;  // the same in every wave
  __syncthreads();

  const int K = p.K, N = p.N;
  const int half = GATED ? (wave & 1) : 0;
  const int part_of = GATED ? wave >> 1 : wave;
  const int NW = (GATED ? 2 * N : N) >> 3;
  const int G = K / p.g, gsteps = p.g / 32;
  const uint32_t* qweight = p.qweight + (int64_t)en.expert * K * NW;
  const uint32_t* qzeros = p.qzeros + (int64_t)en.expert * G * NW;
  const uint16_t* scales = p.scales + (int64_t)en.expert * G * NW * 8;

  // Columns past N read the tile's first ones and are not stored.
  const int wc_in = tile * (kExpertStreamCols / 8) + 2 * c;
  const int wc = (wc_in < (N >> 3) ? wc_in : tile * (kExpertStreamCols / 8)) + half * (N >> 3);
  uint32_t x_off[RB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int r = 16 * rb + c;
    const int xrow = slots[r < en.rows ? r : 0] / p.row_div;
    x_off[rb] = ((uint32_t)xrow * (uint32_t)K + 8u * q) * 2u;
  }
  const uint32_t row_bytes = (uint32_t)NW * 4u;
  const uint32_t w_off = (uint32_t)(8 * q) * row_bytes + (uint32_t)wc * 4u;
  const __amdgpu_buffer_rsrc_t wrs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint32_t*>(qweight), (short)0, (int)(row_bytes * (uint32_t)K), 0x00020000);

  const int T = K / 32;
  const int s0 = split * PARTS * steps;
  const int kb = min(T, s0 + part_of * steps), ke = min(T, kb + steps);

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
  auto issue = [&](Step<RB, REST>& st, int slot, int ks) {
    const bool live = !kAlways || ks < ke;
    if (!kOneSet && live && ks == load_at) fetch(data[kOneSet ? 0 : slot]);
    const uint32_t r0 = live ? (uint32_t)ks * 32u : 0u;
    const uint32_t at_w = live ? w_off : row_bytes * (uint32_t)K, row_step = live ? row_bytes : 0u;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      st.w[r] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(wrs, at_w, (r0 + r) * row_step, 2));
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const uint64_t at = (uint64_t)x_off[rb] + r0 * 2u;
      st.x[rb] = *reinterpret_cast<const half8v*>(reinterpret_cast<const char*>(p.x) + at);
      if constexpr (REST) st.rest[rb] = *reinterpret_cast<const half8v*>(reinterpret_cast<const char*>(p.x_rest) + at);
    }
  };

  const UnpackConsts uk = unpack_consts();
  floatx4 part[RB][16];
  uint32_t zs[16];
  half8v unit[2];          // the columns' current units
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
#pragma unroll
  for (int j = 0; j < kPF; ++j) {
    if (kAlways || kb + j < ke) issue(ring[j], j, kb + j);
    if constexpr (kAlways) __builtin_amdgcn_sched_barrier(0);
  }
  for (int base = kb; base < ke; base += kPF) {
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

  // Per block of 16 rows: waves -> LDS, then one thread per (column entry, lane of rows) sums
  // four rows of one column, and the rows leave in order.
  constexpr int SLOTS = 16 * RL / kThreads;  // sums per thread: 1, 2 or 4
  constexpr int HALVES = GATED ? 2 : 1;
  const bool finish = GATED && splits == 1;
  const int n0 = tile * kExpertStreamCols;
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int rows = min(en.rows - 16 * rb, 16);
    if (rows <= 0) break;  // the same in every wave
    if (rb > 0) __syncthreads();  // the last block's rows have left
    if (lane < RL) {
#pragma unroll
      for (int v = 0; v < 16; ++v) sh.red[wave][v][lane] = part[rb][v] * (float)unit[v >> 3][col_of(v)];
    }
    __syncthreads();
    floatx4 sum[SLOTS][HALVES];
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
      const int i = tid + k * kThreads;
      const int v = (i >> 4) & 15, ln = (i >> 8) * 16 + (i & 15);
#pragma unroll
      for (int hf = 0; hf < HALVES; ++hf) {
        floatx4 a = sh.red[hf][v][ln];
#pragma unroll
        for (int w = 1; w < PARTS; ++w) a += sh.red[GATED ? 2 * w + hf : w][v][ln];
        sum[k][hf] = a;
      }
    }
    __syncthreads();  // the sums are in registers: their LDS takes the output rows
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
      const int i = tid + k * kThreads;
      const int v = (i >> 4) & 15, cc = i & 15;
      const int col = 8 * (2 * cc + (v >> 3)) + col_of(v);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 4 * (i >> 8) + r;
        if constexpr (GATED) {
          sh.ys[row][0][col] = finish ? gated(sum[k][0][r], sum[k][1][r]) : sum[k][0][r];
          sh.ys[row][1][col] = sum[k][1][r];
        } else {
          sh.ys[row][0][col] = sum[k][0][r];
        }
      }
    }
    __syncthreads();
    if (finish) {
      for (int i = tid; i < rows * (kExpertStreamCols / 8); i += kThreads) {
        const int row = i / (kExpertStreamCols / 8), cp = 8 * (i % (kExpertStreamCols / 8));
        if (n0 + cp < N) {
          const float* y = &sh.ys[row][0][cp];
          const int64_t at = (int64_t)slots[16 * rb + row] * N + n0 + cp;
          *reinterpret_cast<u32x4*>(p.h + at) = u32x4{pack_act2<BF16>(y[0], y[1]), pack_act2<BF16>(y[2], y[3]),
                                                      pack_act2<BF16>(y[4], y[5]), pack_act2<BF16>(y[6], y[7])};
          if (p.h_rest != nullptr) {
            u32x4 rest;
#pragma unroll
            for (int j = 0; j < 4; ++j) rest[j] = pack_act2<BF16>(rest_of<BF16>(y[2 * j]), rest_of<BF16>(y[2 * j + 1]));
            *reinterpret_cast<u32x4*>(p.h_rest + at) = rest;
          }
        }
      }
    } else {
      float* out = p.sums + (int64_t)split * p.S * (HALVES * N);
      for (int i = tid; i < rows * HALVES * (kExpertStreamCols / 4); i += kThreads) {
        const int row = i / (HALVES * kExpertStreamCols / 4);
        const int r = i - row * (HALVES * kExpertStreamCols / 4);
        const int hf = r / (kExpertStreamCols / 4), cp = 4 * (r % (kExpertStreamCols / 4));
        if (n0 + cp < N)
          *reinterpret_cast<floatx4*>(out + ((int64_t)slots[16 * rb + row] * HALVES + hf) * N + n0 + cp) =
              *reinterpret_cast<const floatx4*>(&sh.ys[row][hf][cp]);
      }
    }
  }
}

hipError_t launch_expert_stream(const ExpertProduct& p, const ExpertPlan& ep, const int32_t* sorted,
                                const int32_t* table, hipStream_t stream) {
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)ep.grid), dim3(kThreads), 0, stream, p, (int)ep.by_xcd, ep.col_tiles,
                       ep.splits, ep.steps, sorted, table);
  };
#define AWQ_STREAM(GATED, BF16, REST)                                            \
  do {                                                                           \
    if (ep.rows == 4) go(expert_stream_kernel<GATED, BF16, 1, 16, REST>);        \
    else if (ep.rows == 8) go(expert_stream_kernel<GATED, BF16, 1, 32, REST>);   \
    else if (ep.rows == 16) go(expert_stream_kernel<GATED, BF16, 1, 64, REST>);  \
    else go(expert_stream_kernel<GATED, BF16, 2, 64, false>);                    \
  } while (0)
  if (p.gated) {
    if (p.bf16) AWQ_STREAM(true, true, false);
    else AWQ_STREAM(true, false, false);
  } else if (p.x_rest != nullptr) {
    if (p.bf16) AWQ_STREAM(false, true, true);
    else AWQ_STREAM(false, false, true);
  } else {
    if (p.bf16) AWQ_STREAM(false, true, false);
    else AWQ_STREAM(false, false, false);
  }
#undef AWQ_STREAM
  return hipGetLastError();
}

// h = silu(gate) up from the splits' sums [splits][S][2 N], four columns per thread.
template <bool BF16>
__global__ __launch_bounds__(256) void expert_gate_kernel(const float* __restrict__ sums,
                                                          const int32_t* __restrict__ ids, int64_t quads, int S, int E,
                                                          int N, int splits, uint16_t* __restrict__ h,
                                                          uint16_t* __restrict__ h_rest) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  const int64_t s = i / (N / 4);
  const int n = 4 * (int)(i - s * (N / 4));
  const int e = ids[s];
  const float* at = sums + s * 2 * N + n;
  const int64_t stride = (int64_t)S * 2 * N;
  const floatx4 g = sum_splits<8>(at, stride, splits), u = sum_splits<8>(at + N, stride, splits);
  if (e < 0 || e >= E) return;  // behind the loads, which need not wait for it
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = gated(g[j], u[j]);
  *reinterpret_cast<u32x2*>(h + s * N + n) = u32x2{pack_act2<BF16>(v[0], v[1]), pack_act2<BF16>(v[2], v[3])};
  if (h_rest != nullptr)
    *reinterpret_cast<u32x2*>(h_rest + s * N + n) =
        u32x2{pack_act2<BF16>(rest_of<BF16>(v[0]), rest_of<BF16>(v[1])),
              pack_act2<BF16>(rest_of<BF16>(v[2]), rest_of<BF16>(v[3]))};
}

hipError_t launch_expert_gate(const float* sums, const int32_t* ids, int S, int E, int N, int splits, bool bf16,
                              uint16_t* h, uint16_t* h_rest, hipStream_t stream) {
  const int64_t quads = (int64_t)S * (N / 4);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, sums, ids, quads, S, E, N,
                       splits, h, h_rest);
  };
  if (bf16) go(expert_gate_kernel<true>);
  else go(expert_gate_kernel<false>);
  return hipGetLastError();
}

}  // namespace awq
