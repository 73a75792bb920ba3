// A dense product with its epilogue, few rows: bandwidth-bound streaming of the packed weight.
//
//   y = residual + scale * f(x . W + bias), gated f(x . Wg + bg) * (x . Wu + bu)
//
// A workgroup takes up to 16 or 32 rows, 256 columns (gated: the same 256 of both halves) and one K
// split; a wave's part is in awq_stream.h.  The splits of a tile meet in one launch: each leaves
// its fp32 sums in the workspace, in the order its threads hold them, and counts itself in; the one
// that arrives last adds all of them in split order (the same bits whatever the order of arrival)
// and applies the epilogue.  Each XCD has its own L2: sums and counters go through to, and come
// from, where all of them see the same.  The counters are zero between calls.
#include "awq_epilogue.h"
#include "awq_stream.h"

namespace awq {

using namespace stream;

// RB: blocks of 16 rows; RL: lanes whose rows are kept, 16 per four rows.
template <bool GATED, bool BF16, int RB, int RL>
__global__ __launch_bounds__(kThreads, 2) void fused_stream_kernel(const DenseProduct p, const Epilogue e, int tiles,
                                                                   int splits, int steps) {
  constexpr int PARTS = kParts<GATED>;
  constexpr int SLOTS = 16 * RL / kThreads, HALVES = GATED ? 2 : 1;
  __shared__ union {
    floatx4 red[kWaves][16][RL];
    float ys[RL / 4][HALVES][kYld];
  } sh;
  __shared__ uint32_t last_arrival;

  // Splits fastest, then column tiles, then row blocks.
  const int split = blockIdx.x % splits;
  const int tile = blockIdx.x / splits % tiles;
  const int block = blockIdx.x / splits / tiles;
  const int row0 = block * 16 * RB;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, c = lane & 15;
  const int K = p.K, N = p.N;
  const int half = GATED ? (wave & 1) : 0;
  const int part_of = GATED ? wave >> 1 : wave;

  // Columns past N read the tile's first ones and are not stored; rows past M read the block's
  // first.
  const int wc_in = tile * (kExpertStreamCols / 8) + 2 * c;
  const int wc = (wc_in < (N >> 3) ? wc_in : tile * (kExpertStreamCols / 8)) + half * (N >> 3);
  Share<RB> share{p.qweight, p.qzeros, p.scales, (GATED ? 2 * N : N) >> 3, K, p.g, wc, p.x, nullptr, {}, 0, 0};
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int row = row0 + 16 * rb + c;
    share.x_off[rb] = ((uint32_t)(row < p.M ? row : row0) * (uint32_t)K + 8u * q) * 2u;
  }
  const int T = K / 32;
  share.kb = min(T, (split * PARTS + part_of) * steps);
  share.ke = min(T, share.kb + steps);
  floatx4 part[RB][16];
  half8v unit[2];
  stream_sums<BF16, RB, false>(share, Now{}, part, unit);

  // Sums of block rb in registers -> y.
  const int n0 = tile * kExpertStreamCols;
  auto finish = [&](int rb, const floatx4 (&sum)[SLOTS][HALVES]) {
    const int rows = min(p.M - row0 - 16 * rb, 16);
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
      const int s = tid + k * kThreads;
      const int col = slot_col(s), row = slot_row(s);
      const int n = n0 + col;
#pragma unroll
      for (int hf = 0; hf < HALVES; ++hf) {
        const float b = e.bias != nullptr && n < N ? act_to_float<BF16>(e.bias[hf * N + n]) : 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) sh.ys[row + r][hf][col] = sum[k][hf][r] + b;
      }
    }
    __syncthreads();
    for (int i = tid; i < rows * (kExpertStreamCols / 8); i += kThreads) {
      const int row = i / (kExpertStreamCols / 8), cp = 8 * (i % (kExpertStreamCols / 8));
      if (n0 + cp >= N) continue;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[j] = activate(e.act, sh.ys[row][0][cp + j]);
        if constexpr (GATED) f[j] *= sh.ys[row][HALVES - 1][cp + j];
      }
      finish8<BF16>(e, (int64_t)(row0 + 16 * rb + row) * N + n0 + cp, f);
    }
  };

  // Sums in the workspace: [row block][tile][split][rb][half][slot][thread] of four rows.
  constexpr uint32_t kShareBytes = (uint32_t)(RB * HALVES * SLOTS * kThreads * 16);
  const int64_t tile_at = (int64_t)block * tiles + tile;
  const __amdgpu_buffer_rsrc_t prs = __builtin_amdgcn_make_buffer_rsrc(
      p.sums + tile_at * splits * (kShareBytes / 4), (short)0, (int)(kShareBytes * (uint32_t)splits), 0x00020000);
  auto share_at = [&](int sp, int rb, int hf, int k) {
    return (uint32_t)sp * kShareBytes + (uint32_t)(((rb * HALVES + hf) * SLOTS + k) * kThreads + tid) * 16u;
  };
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    if (row0 + 16 * rb >= p.M) break;  // the same in every wave
    if (rb > 0) __syncthreads();       // the last block's LDS has been read
    floatx4 sum[SLOTS][HALVES];
    wave_sums<GATED, RL>(sh.red, part[rb], unit, sum);
    if (splits == 1) {
      __syncthreads();  // the sums are in registers: their LDS takes the output rows
      finish(rb, sum);
    } else {
#pragma unroll
      for (int k = 0; k < SLOTS; ++k)
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sum[k][hf]), prs, share_at(split, rb, hf, k), 0,
                                                 kCpolDevice);
    }
  }
  if (splits == 1) return;
  // Every wave's stores are complete before the workgroup counts itself in.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    uint32_t* count = p.counters + tile_at;
    const bool last = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                      (uint32_t)splits - 1u;
    if (last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last_arrival = last;
  }
  __syncthreads();
  if (!last_arrival) return;
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    if (row0 + 16 * rb >= p.M) break;
    if (rb > 0) __syncthreads();
    floatx4 sum[SLOTS][HALVES];
#pragma unroll
    for (int k = 0; k < SLOTS; ++k)
#pragma unroll
      for (int hf = 0; hf < HALVES; ++hf) {
        sum[k][hf] = floatx4{0.f, 0.f, 0.f, 0.f};
        // Eight loads at a time; those past the last split read it again and are dropped.
        for (int s0 = 0; s0 < splits; s0 += 8) {
          floatx4 v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[j] = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(
                                                   prs, share_at(min(s0 + j, splits - 1), rb, hf, k), 0, kCpolDevice));
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (s0 + j < splits) sum[k][hf] += v[j];
        }
      }
    finish(rb, sum);
  }
}

hipError_t launch_fused_stream(const DenseProduct& p, const Epilogue& e, const DensePlan& d, hipStream_t stream) {
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)d.grid), dim3(kThreads), 0, stream, p, e, d.col_tiles, d.splits, d.steps);
  };
#define AWQ_FUSED(GATED, BF16)                                            \
  do {                                                                    \
    if (d.rows == 4) go(fused_stream_kernel<GATED, BF16, 1, 16>);         \
    else if (d.rows == 8) go(fused_stream_kernel<GATED, BF16, 1, 32>);    \
    else if (d.rows == 16) go(fused_stream_kernel<GATED, BF16, 1, 64>);   \
    else go(fused_stream_kernel<GATED, BF16, 2, 64>);                     \
  } while (0)
  if (p.gated) {
    if (p.bf16) AWQ_FUSED(true, true);
    else AWQ_FUSED(true, false);
  } else {
    if (p.bf16) AWQ_FUSED(false, true);
    else AWQ_FUSED(false, false);
  }
#undef AWQ_FUSED
  return hipGetLastError();
}

}  // namespace awq
