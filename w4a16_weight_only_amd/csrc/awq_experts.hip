// Row tiles of routed experts: x . dequant(W[e]) over slots sorted by expert, with the gated
// activation or the fp32 sums as its epilogue.
//
// A group's scale is a factor of whole columns, so the matrix cores multiply x with the
// integers (q - z) (exact in fp16 and bfloat16) and the scales stay outside, in fp32:
//   sum_k x_k (q - z) s_g(k)  =  u * acc,   acc in units of the current group's scale u;
// at a group boundary acc *= u / u', u = u' (one multiplication per sum and group, no second
// set of accumulators and no rounding of weights; exactly 1 where the scale stays the same).  A scale of zero cannot be a unit: the
// unit stays and that group's (q - z) of the column are staged as zeros.
//
// Workgroup: 8 waves as 2 (rows) x 4 (columns), 256 weight columns (gated: 128 of each half,
// so that a wave holds both of a pair) by 256, 192, 128 or 64 rows, whichever holds the entry; a
// wave's part is 32 FM x 64 of v_mfma_f32_32x32x16.  Per k-tile of 64 the x rows go straight
// to LDS; each thread unpacks 4 rows of one packed word column (8 columns) and writes the
// integers to LDS with k innermost, so a weight is unpacked once per workgroup.
//
// The two waves of a SIMD take turns: while one multiplies (the 4 FM MFMAs of half a k-tile,
// operands in registers; beside the first half's, in their shadow, it unpacks and stages its
// share of k-tile t + 1), the other reads its next operands from LDS.  At a group boundary it
// also rescales the sums of its first 32 columns; those of the other 32 follow in the shadow of
// the first MFMAs (wherever a group may begin, by 1 where none does: a second copy of the MFMAs
// without it makes the compiler move accumulators about).  A barrier ends each turn, and the
// second four waves are one turn behind.
// x is loaded two k-tiles ahead (three LDS buffers), words three (registers).
// Entries of up to 128 rows have the registers for the operands of a whole k-tile, and take one
// pair of turns for it instead of two: what such a turn costs is its reads and its barrier.  The
// integers are then staged two k-tiles ahead (three LDS buffers) and x loaded three (four).  Half
// k-tiles / whole ones, us: gate_up of 128 tokens, one expert 4096 -> 32768, fp16 101 / 95; mlp
// 64 x 2048 -> 1408, 700 and 1000 tokens top 8, 291 / 281 and 338 / 321; 8 x 4096 -> 14336, 512 and
// 1500 tokens top 2, 666 / 650 and 1520 / 1465.
//
// Bound by the matrix cores and what does not hide behind them.  2048 rows of 4096 -> 2 x 4096,
// g 128, take 127 us: 1.08 PFLOP/s (a large dense product 1.19; the MFMAs alone 79 us), 13 us of
// it the launch, the first k-tiles and the epilogue.  Groups of 32 take 175: the rescaling, 128
// vector multiplications per 16 MFMAs of a wave, no longer hides.  A tile of 64, 128, 192 rows
// takes 0.60, 0.70, 0.83 of a tile of 256: unpacking and staging the weights is the same for all,
// so experts' last, short entries add 24 to 36% to a prompt's products.
#include <type_traits>

#include "awq_device.h"
#include "awq_kernels.h"

namespace awq {

namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kBK = 64;
constexpr int kRows = kExpertTileRows;
constexpr int kCols = kExpertTileCols;
constexpr int kThreads = 512;
constexpr int kFN = 2;  // 32 x 32 column blocks of a wave
constexpr int kWM = 2, kWN = 4;
static_assert(kWN * kFN * 32 == kCols && kWM * 4 * 32 == kRows, "8 waves cover the tile");

// LDS: three (or four) k-tiles of x, then two (or three) of the staged integers.
//   x         row r: 128 bytes (64 k), 16-byte chunk c at position c ^ ((r / 2) % 8)
//   integers  column c: 128 bytes at row c ^ ((c / 8 + c / 16) % 2), chunk o at position
//             o ^ swz(c), swz(c) = (c ^ (c / 16)) % 8
// A 16-byte read serves 16 lanes at a time from the 64 banks, of each 32 first those with an even
// number of ones in lane / 4, 0-3, 12-15, 20-27, then the others (measured, lane by lane): either
// half's rows (or columns) of one chunk fall on all sixteen 16-byte slots, and so do the writes of
// one chunk of columns 8 w + j for 16 consecutive w.  (Columns spread for 16 consecutive lanes
// met in pairs.)  Chunks and columns differ in address bits that rows do not reach, so a
// thread keeps one address each and flips bits of it: chunk c + 2 s is address ^ (32 s), column
// 8 w + j of a writer's word is address ^ (144 j).
constexpr int kBTile = kCols * kBK * 2;
constexpr int kLdsBytes = 3 * kRows * kBK * 2 + 2 * kBTile;
static_assert(kLdsBytes <= 160 * 1024, "the compute unit's LDS");
__device__ __forceinline__ int b_addr(int c, int chunk) {
  return (c ^ (((c >> 3) ^ (c >> 4)) & 1)) * (2 * kBK) + 16 * (chunk ^ ((c ^ (c >> 4)) & 7));
}

// 16 bytes per lane from a buffer (bounds-checked: past its end nothing is read) straight into
// LDS: lane l's data lands at lds + 16 l.  Not tracked by the compiler: the kernel waits itself.
// The whole offset is the lane's: a scalar one is not sure to count in the bounds check.
__device__ __forceinline__ void load_lds16_buffer(u32x4 rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc),
               "s"(lds)
               : "memory", "m0");
}
// Raw buffer descriptor of `bytes` bytes at a uniform address.
__device__ __forceinline__ u32x4 buffer_of(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) & 0xFFFFu,
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}

}  // namespace

// FM: 32-row blocks of a wave; the entry has at most 64 FM rows.  BEGINS: groups
// begin at even k-tiles only (2: g is a multiple of 128, or there is one group), at any k-tile
// (1: a multiple of 64), or also in the middle of one (0).  WHOLE: turns of whole k-tiles (K is
// a multiple of 64 and BEGINS is not 0).
template <int FM, bool GATED, bool BF16, int BEGINS, bool WHOLE>
__device__ __forceinline__ void expert_tile(const ExpertProduct& p, char* lds, int e, int first, int rows, int tile,
                                            const int32_t* __restrict__ sorted) {
  static_assert(!WHOLE || BEGINS > 0, "a whole k-tile's turn has one place to change units");
  constexpr int kWaveRows = 32 * FM;
  constexpr int kXBufs = WHOLE ? 4 : 3, kBBufs = WHOLE ? 3 : 2;
  constexpr int kATile = (WHOLE ? 64 * FM : kRows) * kBK * 2;
  constexpr int kBBase = kXBufs * kATile;
  static_assert(kBBase + kBBufs * kBTile <= kLdsBytes, "LDS");
  constexpr int kSteps = WHOLE ? 4 : 2;  // k16 steps of a turn
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / kWN, wn = wave % kWN;
  const int lc = lane & 31;
  const int K = p.K, N = p.N;
  const int NW = (GATED ? 2 * N : N) >> 3;  // packed words of a weight row
  const int G = K / p.g;
  const uint32_t* qweight = p.qweight + (int64_t)e * K * NW;
  const uint32_t* qzeros = p.qzeros + (int64_t)e * G * NW;
  const uint16_t* scales = p.scales + (int64_t)e * G * NW * 8;
  const int n0 = tile * (GATED ? kCols / 2 : kCols);
  const int KT = (K + kBK - 1) / kBK;

  // x rows: wave w stages rows 8 FM w .. 8 FM w + 8 FM - 1, 8 rows a load; lane l fetches chunk
  // (l % 8) ^ ((row / 2) % 8) of row l / 8 of the eight (rows past the entry repeat its last).
  // The upper chunks of a last k-tile of 32 are the next row's, or past the end of x, and are
  // not multiplied.  Loads past the last k-tile re-read it (clamped) and are not multiplied.
  const u32x4 xrs = buffer_of(p.x, (uint32_t)p.S / (uint32_t)p.row_div * (uint32_t)K * 2u);
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds);
  uint32_t a_off[FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int r = 8 * (FM * wave + j) + (lane >> 3);
    const int row = sorted[first + min(r, rows - 1)] / p.row_div;
    a_off[j] = ((uint32_t)row * (uint32_t)K + 8u * (uint32_t)((lane & 7) ^ ((r >> 1) & 7))) * 2u;
  }
  auto load_a = [&](int buf, int kt) {
    const uint32_t at = lds0 + (uint32_t)(buf * kATile + FM * wave * 1024);
#pragma unroll
    for (int j = 0; j < FM; ++j)
      load_lds16_buffer(xrs, a_off[j] + (uint32_t)min(kt, KT - 1) * (kBK * 2u), at + 1024u * j);
  };

  // This thread's share of the weights: rows 4 o .. 4 o + 3 of a k-tile, packed column pw.  A
  // wave has 8 rows, one chunk; its lanes' halves of the chunk alternate with the column so
  // that 32 lanes' 8-byte writes fill all banks.  Rows past K (of a last k-tile of 32, and of
  // k-tiles past the last) are read from rows in range instead and not multiplied.
  const int w = lane & 31;
  const int o_half = (lane >> 5) ^ ((w >> 4) & 1);
  const int half_words = N >> 3;
  int pw;
  if constexpr (GATED) pw = min(n0 / 8 + (w & 15), half_words - 1) + (w >> 4) * half_words;
  else pw = min(n0 / 8 + w, half_words - 1);
  const uint32_t row_bytes = (uint32_t)NW * 4u;
  const __amdgpu_buffer_rsrc_t wrs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint32_t*>(qweight), (short)0, (int)(row_bytes * (uint32_t)K), 0x00020000);
  const uint32_t w_off = (uint32_t)min(8 * wave + 4 * o_half, K - 4) * row_bytes + (uint32_t)pw * 4u;
  const int w_last = wave < 4 ? K - 32 : max(K - kBK, 0);  // where this wave's last rows' k-tile begins
  auto load_words = [&](uint32_t (&words)[4], int kt) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      words[r] = __builtin_amdgcn_raw_buffer_load_b32(wrs, w_off, (uint32_t)(min(kt * kBK, w_last) + r) * row_bytes, 0);
  };
  uint32_t zword;
  u32x4 sraw;
  auto load_group = [&](int gi) {
    zword = qzeros[(int64_t)gi * NW + pw];
    sraw = *reinterpret_cast<const u32x4*>(scales + ((int64_t)gi * NW + pw) * 8);
  };
  const UnpackConsts uk = unpack_consts();
  uint32_t zs[8];     // the operands' zero terms, by nibble
  uint32_t nil = 0;   // columns whose scale is zero (either sign): staged as zeros
  bool any_nil = false;
  auto enter_group = [&] {
    nil = 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t zl = 0xE400u | zero_code(zword, lo_col(t)), zh = 0xD400u | (zero_code(zword, hi_col(t)) << 4);
      zs[2 * t] = zl | (zl << 16);
      zs[2 * t + 1] = zh | (zh << 16);
    }
    uint32_t zero = 0;  // a half of zero, either sign: the halves' borrow trick
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = sraw[i] & 0x7FFF7FFFu;
      zero |= (v - 0x00010001u) & ~v & 0x80008000u;
    }
    any_nil = __builtin_amdgcn_ballot_w64(zero != 0) != 0;
    if (any_nil) {
#pragma unroll
      for (int c = 0; c < 8; ++c) nil |= ((sraw[c >> 1] >> (16 * (c & 1))) & 0x7FFFu) == 0 ? 1u << c : 0u;
    }
  };
  // Where this thread's four values of its column c go.
  const int b_write = kBBase + b_addr(8 * w, wave) + 8 * o_half;
  auto b_at = [&](int buf, int c) { return reinterpret_cast<u32x2_t*>(lds + ((b_write + buf * kBTile) ^ (144 * c))); };
  // Byte t of the words: two columns of the staged tile.
  auto stage = [&](const uint32_t (&words)[4], int buf, int t) {
    half2v lo[2], hi[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t pb;
      if (t == 0) pb = pair_byte<0>(words[2 * i], words[2 * i + 1]);
      else if (t == 1) pb = pair_byte<1>(words[2 * i], words[2 * i + 1]);
      else if (t == 2) pb = pair_byte<2>(words[2 * i], words[2 * i + 1]);
      else pb = pair_byte<3>(words[2 * i], words[2 * i + 1]);
      lo[i] = lo_minus_zero(pb, as_h2(zs[2 * t]), uk);
      hi[i] = hi_minus_zero(pb, as_h2(zs[2 * t + 1]), uk);
    }
    auto put = [&](int c, const half2v (&v)[2]) {
      u32x2_t d;
#pragma unroll
      for (int i = 0; i < 2; ++i) d[i] = BF16 ? pack_bf16x2((float)v[i][0], (float)v[i][1]) : as_u32(v[i]);
      *b_at(buf, c) = d;
    };
    put(lo_col(t), lo);
    put(hi_col(t), hi);
  };
  // Columns without a scale (rare) are staged once more, as zeros.
  auto stage_nil = [&](int buf) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if ((nil >> c) & 1) *b_at(buf, c) = u32x2_t{0u, 0u};
  };

  // This wave's columns: block j, columns tcol(j) + lc of the tile.
  auto tcol = [&](int j) { return GATED ? 32 * wn + j * (kCols / 2) : 32 * (wn * kFN + j); };
  int scol[kFN];  // column of the scales
#pragma unroll
  for (int j = 0; j < kFN; ++j)
    scol[j] = GATED ? min(n0 + 32 * wn + lc, N - 1) + j * N : min(n0 + tcol(j) + lc, N - 1);
  uint16_t s_next[kFN];
  auto load_scales = [&](int gi) {
#pragma unroll
    for (int j = 0; j < kFN; ++j) s_next[j] = scales[(int64_t)min(gi, G - 1) * NW * 8 + scol[j]];
  };

  floatx16 acc[FM][kFN];
  float unit[kFN];
#pragma unroll
  for (int j = 0; j < kFN; ++j) {
    unit[j] = 1.f;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  }

  // Operands of a turn: half a k-tile or a whole one.
  half8v fa[kSteps][FM], fb[kSteps][kFN];
  const int r0 = wm * kWaveRows + lc;
  const int a_read = r0 * (2 * kBK) + 16 * ((lane >> 5) ^ ((r0 >> 1) & 7));
  int b_read[kFN];
#pragma unroll
  for (int j = 0; j < kFN; ++j) b_read[j] = kBBase + b_addr(tcol(j) + lc, lane >> 5);
  auto read = [&](int abuf, int bbuf, int hf) {
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      const int flip = 32 * (2 * hf + st);
#pragma unroll
      for (int j = 0; j < kFN; ++j)
        fb[st][j] = *reinterpret_cast<const half8v*>(lds + ((b_read[j] ^ flip) + bbuf * kBTile));
#pragma unroll
      for (int i = 0; i < FM; ++i)
        fa[st][i] = *reinterpret_cast<const half8v*>(lds + ((a_read ^ flip) + abuf * kATile + 32 * i * (2 * kBK)));
    }
  };
  // A group boundary: new units; the factors of the old sums.
  int group = 0, boundary = 0;
  float ratio[kFN];
  auto change_units = [&] {
    boundary += p.g;
#pragma unroll
    for (int j = 0; j < kFN; ++j) {
      const float s = act_to_float<false>(s_next[j]);
      const float u = s == 0.f ? unit[j] : s;
      ratio[j] = u == unit[j] ? 1.f : unit[j] * __builtin_amdgcn_rcpf(u);
      unit[j] = u;
    }
    load_scales(++group);
  };
  auto rescale = [&](int j) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] *= ratio[j];
  };
  // The 2 FM MFMAs of each step.  SCALE: the second column block's sums still await their
  // factor; the first block's MFMAs go first.  STAGE: with the unpacking of the next k-tile, 8 LDS
  // writes and about 40 vector instructions (88 with the conversions to bfloat16).  The matrix
  // core works on one MFMA while the next share of vector instructions issues.
  auto multiply = [&](auto scale, auto stages, const uint32_t (&next)[4], int to) {
    constexpr bool SCALE = decltype(scale)::value, STAGE = decltype(stages)::value;
    if constexpr (SCALE) rescale(1);
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int j = 0; j < kFN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[i][j] = mfma32<BF16>(fa[st][i], fb[st][j], acc[i][j]);
    if constexpr (STAGE) {
#pragma unroll
      for (int t = 0; t < 4; ++t) stage(next, to, t);
    }
    constexpr int kHalf = FM * kFN;  // MFMAs of one k16 step
    constexpr int kStageValu = STAGE ? (BF16 ? 96 : 48) : 0;
    if constexpr (SCALE) {
#pragma unroll
      for (int i = 0; i < kHalf; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // MFMA
        __builtin_amdgcn_sched_group_barrier(0x002, 10, 0);  // VALU
      }
    }
    if constexpr (STAGE) {
      constexpr int kLeft = (SCALE ? kSteps - 1 : kSteps) * kHalf;
#pragma unroll
      for (int i = 0; i < kLeft; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, (kStageValu + kLeft - 1) / kLeft, 0);
        __builtin_amdgcn_sched_group_barrier(0x200, (8 + kLeft - 1) / kLeft, 0);  // LDS writes
      }
    }
  };
  // Turns end at a barrier; a wave's LDS writes of the turn are done.
  auto turn = [] {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // Group whose zeros this wave unpacks with (its 8 rows of a k-tile lie in one), where it
  // ends, and how many groups on the wave's next one is.
  const int row_half = 32 * (wave >> 2);
  const int stride = p.g == 32 ? 2 : 1;
  int pg = p.g == 32 ? wave >> 2 : 0;
  int pend = (pg + 1) * p.g;

  uint32_t words[2][4];  // of k-tiles t + 1 and t + 2, by parity
  load_group(min(pg, G - 1));
  load_words(words[0], 0);
  load_words(words[1], 1);
  load_scales(0);
  load_a(0, 0);
  enter_group();
  load_group(min(pg + stride, G - 1));
#pragma unroll
  for (int t = 0; t < 4; ++t) stage(words[0], 0, t);
  if (any_nil) stage_nil(0);
  if (kBK + row_half >= pend) {  // the zeros of k-tile 1
    enter_group();
    pg += stride;
    pend += stride * p.g;
    load_group(min(pg + stride, G - 1));
  }
  load_words(words[0], 2);
  load_a(1, 1);
  if constexpr (WHOLE) {
#pragma unroll
    for (int t = 0; t < 4; ++t) stage(words[1], 1, t);
    if (any_nil) stage_nil(1);
    load_words(words[1], 3);
    load_a(2, 2);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (wave >= 4) turn();  // one turn behind

  using yes = std::true_type;
  using no = std::false_type;
  using even = std::integral_constant<int, 0>;
  using odd = std::integral_constant<int, 1>;
  int ab = 0;  // LDS buffer of this k-tile's x
  // The zeros of k-tile kt + 2, which is staged next.
  auto next_zeros = [&](int k0) {
    if (k0 + 2 * kBK + row_half >= pend) {
      enter_group();  // loaded when the last group began
      pg += stride;
      pend += stride * p.g;
      load_group(min(pg + stride, G - 1));
    }
  };
  if constexpr (WHOLE) {
    int bb = 0;  // and of its integers
    auto body = [&](int kt, auto parity, uint32_t (&next)[4]) {
      const int k0 = kt * kBK;
      constexpr bool kBegin = BEGINS < 2 || decltype(parity)::value == 0;
      read(ab, bb, 0);
      if constexpr (kBegin) {
        ratio[1] = 1.f;
        if (k0 == boundary) {
          change_units();
          rescale(0);
        }
      }
      next_zeros(k0);
      load_a((ab + 3) & 3, kt + 3);
      // x of k-tile kt + 1 has landed: 2 FM loads of kt + 2 and kt + 3 and the words of kt + 3
      // are younger.  (Its buffer's last readers, of k-tile kt - 1, ended a turn ago at least, and
      // so did those of the integers that kt + 2's replace below.)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * FM + 4) : "memory");
      turn();
      const int to = bb == 0 ? 2 : bb - 1;
      multiply(std::integral_constant<bool, kBegin>{}, yes{}, next, to);
      if (any_nil) stage_nil(to);
      load_words(next, kt + 4);
      turn();
      ab = (ab + 1) & 3;
      bb = bb == 2 ? 0 : bb + 1;
    };
    int kt = 0;
    for (; kt + 1 < KT; kt += 2) {
      body(kt, even{}, words[0]);
      body(kt + 1, odd{}, words[1]);
    }
    if (kt < KT) body(kt, even{}, words[0]);
  } else {
    auto body = [&](int kt, auto parity, uint32_t (&next)[4]) {
      constexpr int buf = decltype(parity)::value;  // kt % 2
      const int k0 = kt * kBK;
      const bool full = k0 + 32 < K;  // the last k-tile may hold 32 rows
      read(ab, buf, 0);
      constexpr bool kBegin = BEGINS < 2 || buf == 0;
      if constexpr (kBegin) {
        ratio[1] = 1.f;
        if (k0 == boundary) {
          change_units();
          rescale(0);
        }
      }
      turn();
      multiply(std::integral_constant<bool, kBegin>{}, yes{}, next, buf ^ 1);
      if (any_nil) stage_nil(buf ^ 1);
      turn();
      if (full) read(ab, buf, 1);
      if constexpr (BEGINS == 0) {
        ratio[1] = 1.f;
        if (full && k0 + 32 == boundary) {
          change_units();
          rescale(0);
        }
      }
      next_zeros(k0);
      // Behind this turn's waits for scales and zeros: they count back from the newest load the
      // compiler knows, would take these in, and wait for memory (12288 slots of 1408 -> 2048,
      // g32: 266 -> 219 us).
      load_a(ab == 0 ? 2 : ab - 1, kt + 2);
      // x of k-tile kt + 1 has landed: the words of kt + 2 and FM loads of kt + 2 are younger.
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(FM + 4) : "memory");
      turn();
      if (full) multiply(std::integral_constant<bool, BEGINS == 0>{}, no{}, next, 0);
      load_words(next, kt + 3);
      turn();
      ab = ab == 2 ? 0 : ab + 1;
    };
    int kt = 0;
    for (; kt + 1 < KT; kt += 2) {
      body(kt, even{}, words[1]);
      body(kt + 1, odd{}, words[0]);
    }
    if (kt < KT) body(kt, even{}, words[1]);
  }
  if (wave < 4) turn();
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the loads past the last k-tile have landed
  __syncthreads();

  // The LDS tiles are dead: the entry's slots go there, and gated the rounded outputs, so that
  // h is written in 16-byte pieces of rows.
  int32_t* slots = reinterpret_cast<int32_t*>(lds);
  for (int r = tid; r < rows; r += kThreads) slots[r] = sorted[first + r];
  // 32 x 32 block: register r of lane l holds row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.
  auto row_of = [&](int i, int r) { return wm * kWaveRows + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3); };
  if constexpr (GATED) {
    constexpr int kOut = kCols / 2;  // output columns of the tile
    constexpr int kLd = kOut + 8;    // halves of a staged row
    uint16_t* ys = reinterpret_cast<uint16_t*>(lds + kRows * 4);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        ys[row_of(i, r) * kLd + tcol(0) + lc] =
            float_to_act<BF16>(gated(acc[i][0][r] * unit[0], acc[i][1][r] * unit[1]));
    __syncthreads();
    for (int q = tid; q < rows * (kOut / 8); q += kThreads) {
      const int row = q / (kOut / 8), c = 8 * (q % (kOut / 8));
      if (n0 + c < N)
        *reinterpret_cast<u32x4*>(p.h + (int64_t)slots[row] * N + n0 + c) =
            *reinterpret_cast<const u32x4*>(&ys[row * kLd + c]);
    }
  } else {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = row_of(i, r);
        if (row >= rows) continue;
        float* out = p.sums + (int64_t)slots[row] * N;
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
          const int n = n0 + tcol(j) + lc;
          if (n < N) out[n] = acc[i][j][r] * unit[j];
        }
      }
  }
}

template <bool GATED, bool BF16, int BEGINS>
__global__ __launch_bounds__(kThreads, 2) void expert_tile_kernel(const ExpertProduct p, int n_tiles, int tiles,
                                                                  const int32_t* __restrict__ sorted,
                                                                  const int32_t* __restrict__ table) {
  __shared__ __attribute__((aligned(1024))) char lds[kLdsBytes];
  // Every (entry, column tile) twice: the entries of more than 128 rows in the first half of
  // the grid, the others in the second, so that the short ones fill the last round.
  const int small = blockIdx.x >= (uint32_t)(tiles * n_tiles);
  int block = blockIdx.x - small * tiles * n_tiles;
  if constexpr (GATED) {
    // A tile's 64 bytes of a half's row share a 128-byte line with its neighbour's: the two go to
    // one XCD, whose L2 then fetches it once.  Without / with, the same routing, us: gate_up 8 x 4096
    // -> 14336, 700, 1024, 2048 tokens 447 / 441, 606 / 596, 1068 / 1051; 64 x 2048 -> 1408, 700, 1200,
    // 2048 tokens 192 / 190, 237 / 220, 313 / 303.
    if (block < ((tiles * n_tiles) & ~15)) block = (block & ~15) | ((block & 7) << 1) | ((block >> 3) & 1);
  }
  const int entry = block / n_tiles;
  const int tile = block - entry * n_tiles;
  const int e = table[4 * entry];
  const int first = table[4 * entry + 1];
  const int rows = table[4 * entry + 2];
  if (e < 0 || (rows > 128) == small) return;  // the whole workgroup, before any barrier
  if (rows > 192) return expert_tile<4, GATED, BF16, BEGINS, false>(p, lds, e, first, rows, tile, sorted);
  if (rows > 128) return expert_tile<3, GATED, BF16, BEGINS, false>(p, lds, e, first, rows, tile, sorted);
  if constexpr (BEGINS > 0) {
    if (p.K % kBK == 0) {
      if (rows > 64) return expert_tile<2, GATED, BF16, BEGINS, true>(p, lds, e, first, rows, tile, sorted);
      return expert_tile<1, GATED, BF16, BEGINS, true>(p, lds, e, first, rows, tile, sorted);
    }
  }
  if (rows > 64) return expert_tile<2, GATED, BF16, BEGINS, false>(p, lds, e, first, rows, tile, sorted);
  expert_tile<1, GATED, BF16, BEGINS, false>(p, lds, e, first, rows, tile, sorted);
}

hipError_t launch_expert_tiles(const ExpertProduct& p, const ExpertPlan& tp, const int32_t* sorted,
                               const int32_t* table, hipStream_t stream) {
  const int cols = p.gated ? kCols / 2 : kCols;
  const int n_tiles = (p.N + cols - 1) / cols;
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)tp.grid), dim3(kThreads), 0, stream, p, n_tiles, (int)tp.tiles, sorted,
                       table);
  };
  auto pick = [&](auto gated, auto bf16) {
    constexpr bool G = decltype(gated)::value, B = decltype(bf16)::value;
    if (p.g % (2 * kBK) == 0 || p.g == p.K) go(expert_tile_kernel<G, B, 2>);
    else if (p.g % kBK == 0) go(expert_tile_kernel<G, B, 1>);
    else go(expert_tile_kernel<G, B, 0>);
  };
  using yes = std::true_type;
  using no = std::false_type;
  if (p.gated) p.bf16 ? pick(yes{}, yes{}) : pick(yes{}, no{});
  else p.bf16 ? pick(no{}, yes{}) : pick(no{}, no{});
  return hipGetLastError();
}

// y[t] = sum over j of weights[t, j] * (sum over splits of sums[split][t topk + j]).  A
// workgroup takes 256 / PARTS groups of four columns; PARTS threads share one, each adding
// every PARTS-th (slot, split) term in order, and meet in LDS in order: the bits do not
// depend on the schedule.  PARTS > 1 where there are few columns in all.  Four terms' loads go
// out together, whether routed or not (the sums of a slot that is not are memory no one wrote,
// and are dropped), so a term's latency is not the next one's.
template <bool BF16, int PARTS>
__global__ __launch_bounds__(256) void expert_combine_kernel(const float* __restrict__ sums,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ weights, int64_t quads, int S,
                                                             int topk, int E, int N, int splits, int nan_weights,
                                                             uint16_t* __restrict__ y) {
  __shared__ floatx4 meet[PARTS > 1 ? 256 : 1];
  const int part = threadIdx.x % PARTS;
  const int64_t q_raw = (int64_t)blockIdx.x * (256 / PARTS) + threadIdx.x / PARTS;
  const int64_t q = q_raw < quads ? q_raw : quads - 1;
  const int64_t t = q / (N / 4);
  const int n = 4 * (int)(q - t * (N / 4));
  const int terms = topk * splits;
  floatx4 a = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = part; i0 < terms; i0 += 4 * PARTS) {
    floatx4 v[4];
    float w[4];
    int e[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = min(i0 + u * PARTS, terms - 1);
      const int j = splits == 1 ? i : i / splits;
      const int64_t s = t * topk + j;
      e[u] = ids[s];
      w[u] = weights[s];
      v[u] = *reinterpret_cast<const floatx4*>(sums + ((int64_t)(i - j * splits) * S + s) * N + n);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i0 + u * PARTS < terms && e[u] >= 0 && e[u] < E) a += w[u] * v[u];
      else if (nan_weights && w[u] != w[u]) a += w[u];  // (a term read twice is the token's own)
    }
  }
  if constexpr (PARTS > 1) {
    meet[threadIdx.x] = a;
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int i = 1; i < PARTS; ++i) a += meet[threadIdx.x + i];
  }
  if (q_raw < quads)
    *reinterpret_cast<u32x2_t*>(y + t * N + n) = u32x2_t{pack_act2<BF16>(a[0], a[1]), pack_act2<BF16>(a[2], a[3])};
}

// Up to here eight threads per four columns.  One / eight, us per call: down of one token's 8
// slots, 1408 -> 2048, 14.2 / 10.8; mlp 64 x 2048 -> 1408 top 8, 16 tokens 78.2 / 77.7, 128 tokens
// (65536 quads) 114.8 / 115.9.
constexpr int64_t kFewQuads = 32768;

hipError_t launch_expert_combine(const float* sums, const int32_t* ids, const float* weights, int T, int topk, int E,
                                 int N, int splits, bool bf16, bool nan_weights, uint16_t* y, hipStream_t stream) {
  const int64_t quads = (int64_t)T * (N / 4);
  auto go = [&](auto kern, int parts) {
    const int64_t per = 256 / parts;
    hipLaunchKernelGGL(kern, dim3((unsigned)((quads + per - 1) / per)), dim3(256), 0, stream, sums, ids, weights,
                       quads, T * topk, topk, E, N, splits, (int)nan_weights, y);
  };
  const bool few = quads <= kFewQuads && topk * splits > 2;
  if (bf16) {
    if (few) go(expert_combine_kernel<true, 8>, 8);
    else go(expert_combine_kernel<true, 1>, 1);
  } else {
    if (few) go(expert_combine_kernel<false, 8>, 8);
    else go(expert_combine_kernel<false, 1>, 1);
  }
  return hipGetLastError();
}

}  // namespace awq
