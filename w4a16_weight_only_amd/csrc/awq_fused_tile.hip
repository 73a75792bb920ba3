// A dense product with its epilogue, many rows: row tiles on the matrix cores.
//
//   y = residual + scale * f(x . W + bias), gated f(x . Wg + bg) * (x . Wu + bu)
//
// A tile's product and its epilogue are in awq_expert_tile.h; here a workgroup takes up to `height`
// rows, 256 weight columns (gated: 128 of each half) and one K split.  Several splits leave fp32 sums,
// which a second kernel adds, in order, with the epilogue: 64 tiles of 1000 x 11008 -> 4096 would leave three
// compute units of four idle (143 us; four splits 102, of which the join of 66 MB of sums 12).  The join is a
// kernel more rather than the last workgroup's: 64 workgroups of the card's 256 would add them.
// Bound: the matrix cores together with the LDS reads that feed them; 2048 rows through 4096 -> 2 x 11008 366 us,
// 1.01 PFLOP/s, 0.85 of a large plain product's rate.
#include "awq_expert_tile.h"

namespace awq {

using namespace tile;

template <bool GATED, bool BF16, int BEGINS>
__global__ __launch_bounds__(kThreads, 2) void fused_tile_kernel(const DenseProduct d, const Epilogue epi, int n_tiles,
                                                                 int row_tiles, int height, int kps) {
  __shared__ __attribute__((aligned(1024))) char lds[kLdsBytes];
  int block = blockIdx.x;
  if constexpr (GATED) {
    // Tiles that share 128-byte lines of the weight's rows on one XCD (as in expert_tile_kernel).
    if (block < ((int)gridDim.x & ~15)) block = (block & ~15) | ((block & 7) << 1) | ((block >> 3) & 1);
  }
  const int tile = block % n_tiles;
  const int first = block / n_tiles % row_tiles * height;
  const int split = block / n_tiles / row_tiles;
  const int rows = min(height, d.M - first);
  // The split's rows of the weight as a weight of its own: kps is whole groups, or K is one group.
  const int k0 = split * kps, NW = (GATED ? 2 * d.N : d.N) >> 3;
  ExpertProduct p{};
  p.x = d.x + k0;
  p.qweight = d.qweight + (int64_t)k0 * NW;
  p.qzeros = d.qzeros + (int64_t)(k0 / d.g) * NW;
  p.scales = d.scales + (int64_t)(k0 / d.g) * NW * 8;
  p.K = min(kps, d.K - k0);
  p.ldx = d.K;
  p.N = d.N;
  p.g = d.g == d.K ? p.K : d.g;
  p.sums = kps < d.K ? d.sums + (int64_t)split * d.M * (NW * 8) : nullptr;
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

// y of eight adjacent columns from the splits' sums [splits][M][C], C = N or, gated, 2 N.
template <bool GATED, bool BF16>
__global__ __launch_bounds__(256) void fused_join_kernel(const float* __restrict__ sums, const Epilogue e, int64_t pieces,
                                                         int N, int splits) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= pieces) return;
  const int64_t row = i / (N / 8);
  const int n = 8 * (int)(i - row * (N / 8));
  const int C = GATED ? 2 * N : N;
  const float* at = sums + row * C + n;
  const int64_t stride = pieces / (N / 8) * C, out = row * N + n;
  u32x4 res{};
  if (e.residual != nullptr) res = *reinterpret_cast<const u32x4*>(e.residual + out);
  float v[GATED ? 2 : 1][8];
#pragma unroll
  for (int hf = 0; hf < (GATED ? 2 : 1); ++hf) {
    u32x4 raw{};
    if (e.bias != nullptr) raw = *reinterpret_cast<const u32x4*>(e.bias + hf * N + n);
    float b[8];
    unpack8<BF16>(raw, b);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const floatx4 s = sum_splits<4>(at + hf * N + 4 * h, stride, splits);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[hf][4 * h + j] = s[j] + b[4 * h + j];
    }
  }
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[j] = activate(e.act, v[0][j]);
    if constexpr (GATED) f[j] *= v[1][j];
  }
  finish8<BF16>(e, out, f, res);
}

hipError_t launch_fused_tiles(const DenseProduct& p, const Epilogue& e, const DensePlan& d, hipStream_t stream) {
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)d.grid), dim3(kThreads), 0, stream, p, e, d.col_tiles,
                       (p.M + d.rows - 1) / d.rows, d.rows, d.kps);
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
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || d.splits == 1) return err;
  const int64_t pieces = (int64_t)p.M * (p.N / 8);
  auto join = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, stream, p.sums, e, pieces, p.N,
                       d.splits);
  };
  if (p.gated) p.bf16 ? join(fused_join_kernel<true, true>) : join(fused_join_kernel<true, false>);
  else p.bf16 ? join(fused_join_kernel<false, true>) : join(fused_join_kernel<false, false>);
  return hipGetLastError();
}

}  // namespace awq
