// Routed experts: alignment of routed slots by expert, for the tile kernel's grouped
// mode (vLLM article, section 5.4: a routed-expert layer runs a 4-bit WNA16 MoE
// kernel over per-expert qweight / qzeros / scales).
//
// One workgroup counts the slots of each expert in LDS (each atomic's old count is the slot's
// place within its expert), scans the counts into offsets (and the per-expert tile counts into
// table positions), writes one table entry (expert, first sorted row, rows, 0) per tile of
// block_rows rows, and stores every slot at its expert's offset plus its place.  Within an
// expert the slot order depends on the atomics' order; every row of the grouped product
// depends only on its own slot, so the product does not.
// Latency is all there is to it, so up to 16 slots a thread are loaded at once and stay in
// registers with their places (16384 slots over 64 experts 15.8 -> 9.3 us, against a loop of
// single loads and a scan by one thread); more slots are read and counted a second time.
#include "awq_device.h"
#include "awq_kernels.h"

namespace awq {

constexpr int kAlignThreads = 1024;
constexpr int kAlignMaxExperts = 1024;

__global__ __launch_bounds__(kAlignThreads) void moe_align_kernel(const int32_t* __restrict__ ids, int S, int E,
                                                                 int block_rows, int tiles,
                                                                 int32_t* __restrict__ offsets,
                                                                 int32_t* __restrict__ sorted_slots,
                                                                 int32_t* __restrict__ table) {
  constexpr int kHeld = 16;  // slots a thread holds in registers
  constexpr int kWaves = kAlignThreads / 64;
  __shared__ int cnt[kAlignMaxExperts];
  __shared__ int off[kAlignMaxExperts + 1];
  __shared__ int tstart[kAlignMaxExperts + 1];
  __shared__ int wave_rows[kWaves], wave_tiles[kWaves];
  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = tid >> 6;
  cnt[tid] = 0;
  int id[kHeld], place[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int s = tid + i * kAlignThreads;
    id[i] = s < S ? ids[s] : -1;
  }
  __syncthreads();
  // Slots whose expert id is outside [0, E) are not routed anywhere.
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    if (id[i] >= E) id[i] = -1;
    if (id[i] >= 0) place[i] = atomicAdd(&cnt[id[i]], 1);
  }
  if (S > kHeld * kAlignThreads) {
    __syncthreads();  // the held slots' places are below their experts' held counts
    for (int s = tid + kHeld * kAlignThreads; s < S; s += kAlignThreads) {
      const int e = ids[s];
      if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
    }
  }
  __syncthreads();
  // Inclusive sums of rows and tiles over the experts, one per thread: within the wave, then
  // over the waves before it.
  const int rows = cnt[tid];
  const int blocks = (rows + block_rows - 1) / block_rows;
  int r = rows, t = blocks;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int ur = __shfl_up(r, d), ut = __shfl_up(t, d);
    if (lane >= d) {
      r += ur;
      t += ut;
    }
  }
  if (lane == 63) {
    wave_rows[wave] = r;
    wave_tiles[wave] = t;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w)
    if (w < wave) {
      r += wave_rows[w];
      t += wave_tiles[w];
    }
  off[tid + 1] = r;  // experts past E have no rows: every sum from E on is the total
  tstart[tid + 1] = t;
  if (tid == 0) off[0] = tstart[0] = 0;
  __syncthreads();
  for (int e = tid; e <= E; e += kAlignThreads) offsets[e] = off[e];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (id[i] >= 0) sorted_slots[off[id[i]] + place[i]] = tid + i * kAlignThreads;
  // Table entry i belongs to the expert e with tstart[e] <= i < tstart[e + 1].
  for (int i = tid; i < tiles; i += kAlignThreads) {
    int4 ent = {-1, 0, 0, 0};
    if (i < tstart[E]) {
      int lo = 0, hi = E - 1;  // last e with tstart[e] <= i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tstart[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      const int j = i - tstart[lo];
      ent = int4{lo, off[lo] + j * block_rows, min(block_rows, off[lo + 1] - off[lo] - j * block_rows), 0};
    }
    reinterpret_cast<int4*>(table)[i] = ent;
  }
  if (S <= kHeld * kAlignThreads) return;
  // The slots beyond the held ones go behind them: an expert's cursor starts at its held count.
  __syncthreads();
  cnt[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (id[i] >= 0) atomicAdd(&cnt[id[i]], 1);
  __syncthreads();
  for (int s = tid + kHeld * kAlignThreads; s < S; s += kAlignThreads) {
    const int e = ids[s];
    if (e >= 0 && e < E) sorted_slots[off[e] + atomicAdd(&cnt[e], 1)] = s;
  }
}

hipError_t launch_moe_align(const int32_t* expert_ids, int S, int E, int block_rows, int tiles,
                            int32_t* offsets, int32_t* sorted_slots, int32_t* table, hipStream_t stream) {
  hipLaunchKernelGGL(moe_align_kernel, dim3(1), dim3(kAlignThreads), 0, stream, expert_ids, S, E, block_rows, tiles,
                     offsets, sorted_slots, table);
  return hipGetLastError();
}

}  // namespace awq
