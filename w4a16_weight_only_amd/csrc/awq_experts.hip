// Row tiles of routed experts: x . dequant(W[e]) over slots sorted by expert, with the gated
// activation or the fp32 sums as its epilogue.
//
// A group's scale is a factor of whole columns, so the matrix cores multiply x with the
// integers (q - z) (exact in fp16 and bfloat16) and the scales stay outside, in fp32:
//   sum_k x_k (q - z) s_g(k)  =  u * acc,   acc in units of the current group's scale u;
// at a group boundary acc *= u / u', u = u' (one multiplication per sum and group, no second
// set of accumulators and no rounding of weights).  A scale of zero cannot be a unit: the
// unit stays and that group's (q - z) of the column are staged as zeros.
//
// Workgroup: 128 rows x 256 weight columns (gated: 128 columns of each half, so that a wave
// holds both of a pair), 4 waves of 64 x 128, v_mfma_f32_32x32x16.  Per k-tile of 64 the x
// rows go straight to LDS; each thread unpacks 8 rows of one packed word column (8 columns)
// and writes the integers to LDS with k innermost, so each weight is unpacked once per
// workgroup.  Two workgroups share a compute unit: one multiplies while the other unpacks.
#include "awq_device.h"
#include "awq_kernels.h"

namespace awq {

namespace {

constexpr int kBK = 64;
constexpr int kRows = kExpertTileRows;
constexpr int kCols = kExpertTileCols;
constexpr int kThreads = 256;
constexpr int kFM = 2, kFN = 4;  // 32 x 32 blocks of a wave: 64 rows x 128 columns
constexpr int kWaveRows = 32 * kFM;

// LDS rows of the staged integers: column c's 64 k values take 128 bytes, 16-byte chunk o at
// position o ^ b_swz(c) of row b_row(c).  Writers hold one chunk of columns 8 w + j for 16
// consecutive w at a time and readers one chunk of 16 consecutive columns: both reach all
// sixteen 16-byte slots of the 64 banks.
__device__ __forceinline__ int b_row(int c) { return c ^ ((c >> 3) & 1); }
__device__ __forceinline__ int b_swz(int c) { return (c ^ (c >> 4)) & 7; }

}  // namespace

template <bool GATED, bool BF16>
__global__ __launch_bounds__(kThreads, 2) void expert_tile_kernel(const ExpertProduct p, int n_tiles, int tiles,
                                                                  const int32_t* __restrict__ sorted,
                                                                  const int32_t* __restrict__ table) {
  __shared__ __attribute__((aligned(16))) uint16_t As[2][kRows * kBK];
  __shared__ __attribute__((aligned(16))) uint16_t Bs[kCols * kBK];
  __shared__ int32_t slots[kRows];

  const int entry = blockIdx.x / n_tiles;
  const int tile = blockIdx.x - entry * n_tiles;
  if (entry >= tiles) return;
  const int e = table[4 * entry];
  if (e < 0) return;  // an unused entry: the whole workgroup leaves before any barrier
  const int first = table[4 * entry + 1];
  const int rows = table[4 * entry + 2];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int lc = lane & 31;
  const int K = p.K, N = p.N;
  const int NW = (GATED ? 2 * N : N) >> 3;  // packed words of a weight row
  const int G = K / p.g;
  const uint32_t* qweight = p.qweight + (int64_t)e * K * NW;
  const uint32_t* qzeros = p.qzeros + (int64_t)e * G * NW;
  const uint16_t* scales = p.scales + (int64_t)e * G * NW * 8;
  const int n0 = tile * (GATED ? kCols / 2 : kCols);

  for (int r = tid; r < kRows; r += kThreads) slots[r] = sorted[first + min(r, rows - 1)];

  // x rows: wave w stages rows 32 w .. 32 w + 31, 8 rows a load; lane l fetches chunk
  // (l % 8) ^ ((row / 2) % 8) of row l / 8 of the eight (rows past the entry repeat its last).
  uint32_t a_off[4];
  int a_ch[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 32 * wave + 8 * j + (lane >> 3);
    const int row = sorted[first + min(r, rows - 1)] / p.row_div;
    a_ch[j] = (lane & 7) ^ ((r >> 1) & 7);
    a_off[j] = ((uint32_t)row * (uint32_t)K + 8u * (uint32_t)a_ch[j]) * 2u;
  }
  auto load_a = [&](int buf, int k0) {
    const bool part = K - k0 < kBK;  // the last 32 of K: the upper chunks re-read the lower
#pragma unroll
    for (int j = 0; j < 4; ++j)
      load_lds16_s(p.x + k0, a_off[j] - (part && a_ch[j] >= 4 ? 64u : 0u), &As[buf][(32 * wave + 8 * j) * kBK]);
  };

  // This thread's share of the weights: rows 8 o .. 8 o + 7 of packed column pw.
  const int o = tid >> 5, w = tid & 31;
  const int half_words = N >> 3;
  int pw;
  if constexpr (GATED) pw = min(n0 / 8 + (w & 15), half_words - 1) + (w >> 4) * half_words;
  else pw = min(n0 / 8 + w, half_words - 1);
  uint32_t words[8], zword;
  u32x4 sraw;
  auto load_b = [&](int k0) {
    const int k = min(k0 + 8 * o, K - 8);
#pragma unroll
    for (int r = 0; r < 8; ++r) words[r] = qweight[(int64_t)(k + r) * NW + pw];
    const int gi = k / p.g;
    zword = qzeros[(int64_t)gi * NW + pw];
    sraw = *reinterpret_cast<const u32x4*>(scales + ((int64_t)gi * NW + pw) * 8);
  };
  const UnpackConsts uk = unpack_consts();
  auto stage_b = [&] {
    // Columns with a scale of zero (either sign) keep zeros instead of (q - z).
    uint32_t nil = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = sraw[i] & 0x7FFF7FFFu;
      nil |= (v - 0x00010001u) & ~v & 0x80008000u;
    }
    const bool any_nil = __builtin_amdgcn_ballot_w64(nil != 0) != 0;
    auto put = [&](int c, half2v (&v)[4]) {
      u32x4 d;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = BF16 ? pack_bf16x2((float)v[i][0], (float)v[i][1]) : as_u32(v[i]);
      if (any_nil && ((sraw[c >> 1] >> (16 * (c & 1))) & 0x7FFFu) == 0) d = u32x4{0u, 0u, 0u, 0u};
      const int col = 8 * w + c;
      *reinterpret_cast<u32x4*>(&Bs[b_row(col) * kBK + 8 * (o ^ b_swz(col))]) = d;
    };
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t zl = 0xE400u | zero_code(zword, lo_col(t)), zh = 0xD400u | (zero_code(zword, hi_col(t)) << 4);
      const half2v offl = as_h2(zl | (zl << 16)), offh = as_h2(zh | (zh << 16));
      half2v lo[4], hi[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t pb;
        if (t == 0) pb = pair_byte<0>(words[2 * i], words[2 * i + 1]);
        else if (t == 1) pb = pair_byte<1>(words[2 * i], words[2 * i + 1]);
        else if (t == 2) pb = pair_byte<2>(words[2 * i], words[2 * i + 1]);
        else pb = pair_byte<3>(words[2 * i], words[2 * i + 1]);
        lo[i] = lo_minus_zero(pb, offl, uk);
        hi[i] = hi_minus_zero(pb, offh, uk);
      }
      put(lo_col(t), lo);
      put(hi_col(t), hi);
    }
  };

  // This wave's columns: block j, column of the tile tcol(j) + lc.
  auto tcol = [&](int j) {
    if constexpr (GATED) return (j >= kFN / 2 ? kCols / 2 : 0) + 32 * (wn * (kFN / 2) + j % (kFN / 2));
    else return 32 * (wn * kFN + j);
  };
  int scol[kFN];  // column of the scales
#pragma unroll
  for (int j = 0; j < kFN; ++j) {
    if constexpr (GATED) scol[j] = min(n0 + 32 * (wn * (kFN / 2) + j % (kFN / 2)) + lc, N - 1) + (j >= kFN / 2 ? N : 0);
    else scol[j] = min(n0 + tcol(j) + lc, N - 1);
  }
  uint16_t s_next[kFN];
  auto load_scales = [&](int gi) {
#pragma unroll
    for (int j = 0; j < kFN; ++j) s_next[j] = scales[(int64_t)min(gi, G - 1) * NW * 8 + scol[j]];
  };

  floatx16 acc[kFM][kFN];
  float unit[kFN];
#pragma unroll
  for (int j = 0; j < kFN; ++j) {
    unit[j] = 1.f;
#pragma unroll
    for (int i = 0; i < kFM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  }

  load_scales(0);
  load_b(0);
  load_a(0, 0);
  int group = 0, boundary = 0;
  const int KT = (K + kBK - 1) / kBK;
  for (int kt = 0; kt < KT; ++kt) {
    const int k0 = kt * kBK;
    stage_b();
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (kt + 1 < KT) {
      load_a((kt + 1) & 1, k0 + kBK);
      load_b(k0 + kBK);
    }
    const uint16_t* A = As[kt & 1];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int kk = k0 + 32 * hf;
      if (kk >= K) break;  // uniform: the last k-tile may hold 32 rows
      if (kk == boundary) {
        boundary += p.g;
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
          const float s = act_to_float<false>(s_next[j]);
          const float u = s == 0.f ? unit[j] : s;
          const float ratio = unit[j] * __builtin_amdgcn_rcpf(u);
          if (group > 0) {
#pragma unroll
            for (int i = 0; i < kFM; ++i)
#pragma unroll
              for (int r = 0; r < 16; ++r) acc[i][j][r] *= ratio;
          }
          unit[j] = u;
        }
        ++group;
        load_scales(group);
      }
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const int ch = 4 * hf + 2 * st + (lane >> 5);
        half8v a[kFM], b[kFN];
#pragma unroll
        for (int i = 0; i < kFM; ++i) {
          const int r = wm * kWaveRows + 32 * i + lc;
          a[i] = *reinterpret_cast<const half8v*>(&A[r * kBK + 8 * (ch ^ ((r >> 1) & 7))]);
        }
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
          const int c = tcol(j) + lc;
          b[j] = *reinterpret_cast<const half8v*>(&Bs[b_row(c) * kBK + 8 * (ch ^ b_swz(c))]);
        }
#pragma unroll
        for (int i = 0; i < kFM; ++i)
#pragma unroll
          for (int j = 0; j < kFN; ++j) acc[i][j] = mfma32<BF16>(a[i], b[j], acc[i][j]);
      }
    }
    __syncthreads();
  }

  // 32 x 32 block: register r of lane l holds row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.
#pragma unroll
  for (int i = 0; i < kFM; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = wm * kWaveRows + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
      if (row >= rows) continue;
      const int64_t slot = slots[row];
      if constexpr (GATED) {
#pragma unroll
        for (int j = 0; j < kFN / 2; ++j) {
          const int n = n0 + tcol(j) + lc;
          if (n < N)
            p.h[slot * N + n] =
                float_to_act<BF16>(gated(acc[i][j][r] * unit[j], acc[i][j + kFN / 2][r] * unit[j + kFN / 2]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
          const int n = n0 + tcol(j) + lc;
          if (n < N) p.sums[slot * N + n] = acc[i][j][r] * unit[j];
        }
      }
    }
}

hipError_t launch_expert_tiles(const ExpertProduct& p, const ExpertPlan& tp, const int32_t* sorted,
                               const int32_t* table, hipStream_t stream) {
  const int cols = p.gated ? kCols / 2 : kCols;
  const int n_tiles = (p.N + cols - 1) / cols;
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)tp.grid), dim3(kThreads), 0, stream, p, n_tiles, (int)tp.tiles, sorted,
                       table);
  };
  if (p.gated) {
    if (p.bf16) go(expert_tile_kernel<true, true>);
    else go(expert_tile_kernel<true, false>);
  } else {
    if (p.bf16) go(expert_tile_kernel<false, true>);
    else go(expert_tile_kernel<false, false>);
  }
  return hipGetLastError();
}

// y[t] = sum over j of weights[t, j] * (sum over splits of sums[split][t topk + j]).  A
// workgroup takes 256 / PARTS groups of four columns; PARTS threads share one, each adding
// every PARTS-th (slot, split) term in order, and meet in LDS in order: the bits do not
// depend on the schedule.  PARTS > 1 where there are few columns in all, so that the loads of
// a column group are in flight together.
template <bool BF16, int PARTS>
__global__ __launch_bounds__(256) void expert_combine_kernel(const float* __restrict__ sums,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ weights, int64_t quads, int S,
                                                             int topk, int E, int N, int splits,
                                                             uint16_t* __restrict__ y) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  __shared__ floatx4 meet[PARTS > 1 ? 256 : 1];
  const int part = threadIdx.x % PARTS;
  const int64_t q_raw = (int64_t)blockIdx.x * (256 / PARTS) + threadIdx.x / PARTS;
  const int64_t q = q_raw < quads ? q_raw : quads - 1;
  const int64_t t = q / (N / 4);
  const int n = 4 * (int)(q - t * (N / 4));
  floatx4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = part; i < topk * splits; i += PARTS) {
    const int j = i / splits, sp = i - j * splits;
    const int64_t s = t * topk + j;
    const int e = ids[s];
    if (e >= 0 && e < E) a += weights[s] * *reinterpret_cast<const floatx4*>(sums + ((int64_t)sp * S + s) * N + n);
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

hipError_t launch_expert_combine(const float* sums, const int32_t* ids, const float* weights, int T, int topk, int E,
                                 int N, int splits, bool bf16, uint16_t* y, hipStream_t stream) {
  const int64_t quads = (int64_t)T * (N / 4);
  auto go = [&](auto kern, int parts) {
    const int64_t per = 256 / parts;
    hipLaunchKernelGGL(kern, dim3((unsigned)((quads + per - 1) / per)), dim3(256), 0, stream, sums, ids, weights,
                       quads, T * topk, topk, E, N, splits, y);
  };
  const bool few = quads * 8 <= 65536 && topk * splits > 2;  // fewer threads than the card holds
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
