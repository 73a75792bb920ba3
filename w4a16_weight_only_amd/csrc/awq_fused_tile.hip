// A dense product with its epilogue, many rows: row tiles on the matrix cores.
//
//   y = residual + scale * f(x . W + bias), gated f(x . Wg + bg) * (x . Wu + bu)
//
// A tile's product and its epilogue are in awq_expert_tile.h; here a workgroup takes up to `height`
// rows and 256 weight columns (gated: 128 of each half).
#include "awq_expert_tile.h"

namespace awq {

using namespace tile;

template <bool GATED, bool BF16, int BEGINS>
__global__ __launch_bounds__(kThreads, 2) void fused_tile_kernel(const DenseProduct d, const Epilogue epi, int n_tiles,
                                                                 int height) {
  __shared__ __attribute__((aligned(1024))) char lds[kLdsBytes];
  int block = blockIdx.x;
  if constexpr (GATED) {
    // Tiles that share 128-byte lines of the weight's rows on one XCD (as in expert_tile_kernel).
    if (block < ((int)gridDim.x & ~15)) block = (block & ~15) | ((block & 7) << 1) | ((block >> 3) & 1);
  }
  const int tile = block % n_tiles;
  const int first = block / n_tiles * height;
  const int rows = min(height, d.M - first);
  ExpertProduct p{};
  p.x = d.x;
  p.qweight = d.qweight;
  p.qzeros = d.qzeros;
  p.scales = d.scales;
  p.K = d.K;
  p.ldx = d.K;
  p.N = d.N;
  p.g = d.g;
  if (rows > 192) return expert_tile<4, GATED, BF16, BEGINS, false, true>(p, lds, 0, first, rows, tile, nullptr, &epi);
  if (rows > 128) return expert_tile<3, GATED, BF16, BEGINS, false, true>(p, lds, 0, first, rows, tile, nullptr, &epi);
  if constexpr (BEGINS > 0) {
    if (p.K % kBK == 0) {
      if (rows > 64) return expert_tile<2, GATED, BF16, BEGINS, true, true>(p, lds, 0, first, rows, tile, nullptr, &epi);
      return expert_tile<1, GATED, BF16, BEGINS, true, true>(p, lds, 0, first, rows, tile, nullptr, &epi);
    }
  }
  if (rows > 64) return expert_tile<2, GATED, BF16, BEGINS, false, true>(p, lds, 0, first, rows, tile, nullptr, &epi);
  expert_tile<1, GATED, BF16, BEGINS, false, true>(p, lds, 0, first, rows, tile, nullptr, &epi);
}

hipError_t launch_fused_tiles(const DenseProduct& p, const Epilogue& e, const DensePlan& d, hipStream_t stream) {
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)d.grid), dim3(kThreads), 0, stream, p, e, d.col_tiles, d.rows);
  };
  auto pick = [&](auto gated, auto bf16) {
    constexpr bool G = decltype(gated)::value, B = decltype(bf16)::value;
    if (p.g % (2 * kBK) == 0 || p.g == p.K) go(fused_tile_kernel<G, B, 2>);
    else if (p.g % kBK == 0) go(fused_tile_kernel<G, B, 1>);
    else go(fused_tile_kernel<G, B, 0>);
  };
  using yes = std::true_type;
  using no = std::false_type;
  if (p.gated) p.bf16 ? pick(yes{}, yes{}) : pick(yes{}, no{});
  else p.bf16 ? pick(no{}, yes{}) : pick(no{}, no{});
  return hipGetLastError();
}

}  // namespace awq
