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
//
// Eight waves, one workgroup to a compute unit, rather than two of four: half the shares to join (us in
// a graph, four / eight waves: 1 x 4096 -> 4096 fp16 12.1 / 8.3, with its splits; 19 x 4096 -> 2 x 11008
// bfloat16 36 / 28).  256 columns a wave, so that 16 lanes read whole 128-byte lines of a row.
// Bound: one row of 4096 x 4096 (8.0 us, 8.7 MB) by this form, one after another of the weights, the waves' and the
// splits' sums, on half of the compute units (awq_decode.hip, lighter workgroups and no sums read back, takes 4.6
// there, without the epilogue); 19 rows through 4096 -> 2 x 11008 (25.3 us, 47 MB, 172 workgroups) and 200 rows of 2048 -> 8192
// (20.2 us) by unpacking: VALU 60% and the matrix cores 25% of a busy compute unit's time.  Whether these or
// row tiles take a call: choose_tiles.
#include "awq_epilogue.h"
#include "awq_stream.h"

namespace awq {

using namespace stream;

// RB: blocks of 16 rows; RL: lanes whose rows are kept, 16 per four rows; R: 1 for one row in all.
template <bool GATED, bool BF16, int RB, int RL, int R>
__global__ __launch_bounds__(64 * kStreamWaves, 2) void fused_stream_kernel(const DenseProduct p, const Epilogue e, int tiles,
                                                                     int splits, int steps) {
  constexpr int WAVES = kStreamWaves, THREADS = 64 * WAVES;
  constexpr int PARTS = kParts<GATED, WAVES>;
  constexpr int SLOTS = kSlots<RL, WAVES>, HALVES = GATED ? 2 : 1;
  constexpr int kPieces = R == 1 ? 1 : (RL / 4 * (kExpertStreamCols / 8) + THREADS - 1) / THREADS;
  __shared__ union {
    Rows<R> red[WAVES][16][RL];
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

  // What the epilogue reads is asked for before the splits meet: the biases of the slots' columns, and
  // the residual of the row pieces that this thread writes (one row: of its column).
  const int n0 = tile * kExpertStreamCols;
  uint16_t braw[SLOTS][HALVES];
#pragma unroll
  for (int k = 0; k < SLOTS; ++k)
#pragma unroll
    for (int hf = 0; hf < HALVES; ++hf) {
      const int n = n0 + slot_col(tid + k * THREADS);
      braw[k][hf] = e.bias != nullptr && n < N ? e.bias[hf * N + n] : 0;
    }
  auto piece = [&](int i, int rb, int& row, int& col) {  // piece i of this thread: whether it is one
    const int at = tid + i * THREADS;
    row = row0 + 16 * rb + at / (kExpertStreamCols / 8);
    col = n0 + 8 * (at % (kExpertStreamCols / 8));
    return at < RL / 4 * (kExpertStreamCols / 8) && row < p.M && col < N;
  };
  struct Residual {
    u32x4 w[kPieces];
    uint16_t one;
  };
  auto ask_residual = [&](int rb, Residual& r) {
    if (e.residual == nullptr) return;
    if constexpr (R == 1) {
      const int n = n0 + slot_col(tid);
      r.one = tid < 16 * RL && n < N ? e.residual[n] : 0;
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        int row, col;
        if (piece(i, rb, row, col)) r.w[i] = *reinterpret_cast<const u32x4*>(e.residual + (int64_t)row * N + col);
      }
    }
  };
  // Sums of block rb in registers -> y.
  auto finish = [&](int rb, const Rows<R> (&sum)[SLOTS][HALVES], const Residual& res) {
    if constexpr (R == 1) {
      const int n = n0 + slot_col(tid);
      if (tid >= 16 * RL || n >= N) return;
      float f = activate(e.act, sum[0][0] + act_to_float<BF16>(braw[0][0]));
      if constexpr (GATED) f *= sum[0][HALVES - 1] + act_to_float<BF16>(braw[0][HALVES - 1]);
      e.y[n] = float_to_act<BF16>((e.residual != nullptr ? act_to_float<BF16>(res.one) : 0.f) + e.scale * f);
    } else {
#pragma unroll
      for (int k = 0; k < SLOTS; ++k) {
        const int s = tid + k * THREADS;
        if (THREADS > 16 * RL && s >= 16 * RL) continue;
        const int col = slot_col(s), row = slot_row(s);
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            sh.ys[row + r][hf][col] = row_of<R>(sum[k][hf], r) + act_to_float<BF16>(braw[k][hf]);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        int row, col;
        if (!piece(i, rb, row, col)) continue;
        const int at = row - row0 - 16 * rb, cp = col - n0;
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[j] = activate(e.act, sh.ys[at][0][cp + j]);
          if constexpr (GATED) f[j] *= sh.ys[at][HALVES - 1][cp + j];
        }
        finish8<BF16>(e, (int64_t)row * N + col, f, res.w[i]);
      }
    }
  };

  // Sums in the workspace: [row block][tile][split][rb][half][slot][thread] of R rows.
  constexpr uint32_t kOne = 4u * R;
  constexpr uint32_t kShareBytes = (uint32_t)(RB * HALVES * 16 * RL) * kOne;
  const int64_t tile_at = (int64_t)block * tiles + tile;
  const __amdgpu_buffer_rsrc_t prs = __builtin_amdgcn_make_buffer_rsrc(
      p.sums + tile_at * splits * (kShareBytes / 4), (short)0, (int)(kShareBytes * (uint32_t)splits), 0x00020000);
  // (Threads past the last slot, and slots of rows past M, reach past the buffer: nothing moves.)
  auto share_at = [&](int sp, int rb, int hf, int k) {
    const int s = tid + k * THREADS;
    const uint32_t at = (uint32_t)sp * kShareBytes + (uint32_t)((rb * HALVES + hf) * 16 * RL + s) * kOne;
    const bool none = (THREADS > 16 * RL && s >= 16 * RL) || row0 + 16 * rb + slot_row(s) >= p.M;
    return none ? kShareBytes * (uint32_t)splits : at;
  };
  Residual res;
  if (splits == 1) ask_residual(0, res);
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    if (row0 + 16 * rb >= p.M) break;  // the same in every wave
    if (rb > 0) {
      if (splits == 1) ask_residual(rb, res);
      __syncthreads();  // the last block's LDS has been read
    }
    Rows<R> sum[SLOTS][HALVES];
    wave_sums<GATED, RL, WAVES, R>(sh.red, part[rb], unit, sum);
    if (splits == 1) {
      __syncthreads();  // the sums are in registers: their LDS takes the output rows
      finish(rb, sum, res);
    } else {
#pragma unroll
      for (int k = 0; k < SLOTS; ++k)
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) device_store<R>(prs, share_at(split, rb, hf, k), sum[k][hf]);
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
  if (__builtin_amdgcn_readfirstlane((int)last_arrival) == 0) return;
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    if (row0 + 16 * rb >= p.M) break;
    ask_residual(rb, res);
    Rows<R> flat[SLOTS * HALVES], sum[SLOTS][HALVES];
    device_sums<R>(prs, splits, [&](int sp, int i) { return share_at(sp, rb, i % HALVES, i / HALVES); }, flat);
#pragma unroll
    for (int i = 0; i < SLOTS * HALVES; ++i) sum[i / HALVES][i % HALVES] = flat[i];
    if (rb > 0) __syncthreads();
    finish(rb, sum, res);
  }
}

hipError_t launch_fused_stream(const DenseProduct& p, const Epilogue& e, const DensePlan& d, hipStream_t stream) {
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)d.grid), dim3(64 * kStreamWaves), 0, stream, p, e, d.col_tiles, d.splits,
                       d.steps);
  };
#define AWQ_FUSED(GATED, BF16)                                             \
  do {                                                                     \
    if (d.rows == 1) go(fused_stream_kernel<GATED, BF16, 1, 16, 1>);       \
    else if (d.rows == 4) go(fused_stream_kernel<GATED, BF16, 1, 16, 4>);  \
    else if (d.rows == 8) go(fused_stream_kernel<GATED, BF16, 1, 32, 4>);  \
    else if (d.rows == 16) go(fused_stream_kernel<GATED, BF16, 1, 64, 4>); \
    else go(fused_stream_kernel<GATED, BF16, 2, 64, 4>);                   \
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
