// Few rows per routed expert: bandwidth-bound streaming of the experts' packed weights.
//
// A workgroup takes up to 16 or 32 routed rows of one expert (an entry), 256 columns (gated:
// the same 256 of both halves) and one K split.  Its four waves each take a run of 32-row
// k-steps; gated, even waves take the gate's columns and odd ones the up projection's (a wave's
// part is in awq_stream.h).
// The waves meet in LDS.  With one split a gated workgroup writes h; otherwise fp32 sums
// [split][slot][column] leave for the next kernel, which adds the splits in order.
//
// Which rows a workgroup has: up to 64 slots, every wave ranks them itself (one slot per
// lane); above, the table of launch_moe_align in blocks of 16 or 32 rows.
//
// Bound by HBM from a few rows on (medians of 27 calls): one token's two experts of 4096 -> 2 x
// 14336, 117 MB, 28.2 us (4.2 TB/s; a copy of 2 GiB 4.96, of which half are writes); 19 rows of
// 14336 -> 4096 over 8 experts, 235 MB, 46.7 us (5.0).  By latency below that (8 slots of 2048 -> 2 x
// 1408, 23 MB, 13.3 us), and by unpacking beside HBM at 32 rows and in bfloat16 (16 tokens' 8 x
// 4096 -> 2 x 14336, 470 MB, 109 us, 4.3 TB/s; 101 at best).
#include "awq_stream.h"

namespace awq {

using namespace stream;

// RB: blocks of 16 rows.  RL: lanes whose sums are kept, 16 per four rows (an entry of one block
// never has more than RL / 4 rows).  REST: rows of two terms, x and x_rest.
template <bool GATED, bool BF16, int RB, int RL, bool REST>
__global__ __launch_bounds__(kThreads, 2) void expert_stream_kernel(const ExpertProduct p, int by_xcd, int tiles,
                                                                    int splits, int steps,
                                                                    const int32_t* __restrict__ sorted,
                                                                    const int32_t* __restrict__ table) {
  constexpr int PARTS = kParts<GATED>;  // waves along K
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
    const int id = lane < p.S ? p.ids[lane] : -1;
    en = entry_of<16 * RB>(rank_slots<16 * RB>(id, p.E), id, entry, lane, slots);
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
  const int G = K / p.g;
  const uint32_t* qweight = p.qweight + (int64_t)en.expert * K * NW;
  const uint32_t* qzeros = p.qzeros + (int64_t)en.expert * G * NW;
  const uint16_t* scales = p.scales + (int64_t)en.expert * G * NW * 8;

  // Columns past N read the tile's first ones and are not stored.
  const int wc_in = tile * (kExpertStreamCols / 8) + 2 * c;
  const int wc = (wc_in < (N >> 3) ? wc_in : tile * (kExpertStreamCols / 8)) + half * (N >> 3);
  Share<RB> share{qweight, qzeros, scales, NW, K, p.g, wc, p.x, p.x_rest, {}, 0, 0};
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int r = 16 * rb + c;
    const int xrow = slots[r < en.rows ? r : 0] / p.row_div;
    share.x_off[rb] = ((uint32_t)xrow * (uint32_t)K + 8u * q) * 2u;
  }
  const int T = K / 32;
  const int s0 = split * PARTS * steps;
  share.kb = min(T, s0 + part_of * steps);
  share.ke = min(T, share.kb + steps);

  floatx4 part[RB][16];
  half8v unit[2];
  stream_sums<BF16, RB, REST>(share, Now{}, part, unit);

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
    floatx4 sum[SLOTS][HALVES];
    wave_sums<GATED, RL>(sh.red, part[rb], unit, sum);
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
