// Row tiles of routed experts: x . dequant(W[e]) over slots sorted by expert, with the gated
// activation or the fp32 sums as its epilogue.
//
// A tile's product is in awq_expert_tile.h.
//
// Bound by the matrix cores and what does not hide behind them.  2048 rows of 4096 -> 2 x 4096,
// g 128, take 127 us: 1.08 PFLOP/s (a large dense product 1.19; the MFMAs alone 79 us), 13 us of
// it the launch, the first k-tiles and the epilogue.  Groups of 32 take 175: the rescaling, 128
// vector multiplications per 16 MFMAs of a wave, no longer hides.  A tile of 64, 128, 192 rows
// takes 0.60, 0.70, 0.83 of a tile of 256: unpacking and staging the weights is the same for all,
// so experts' last, short entries add 24 to 36% to a prompt's products.
#include "awq_expert_tile.h"

namespace awq {

using namespace tile;

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
