// A whole routed layer for few tokens (at most 64 slots), in two kernels:
//   y[t] = residual[t] + sum over j of weights[t, j] * down[e](silu(gate[e](x[t])) * up[e](x[t])),
//   e and weights of slot (t, j) from the logits x . router^T
//
// layer_router_kernel: a wave per expert (up to eight for few experts) forms the logits of eight tokens;
// the workgroup that finishes last routes those tokens, a wave per token (awq_route.h), where the
// next kernel does not.
//
// layer_kernel: both products, streamed (awq_stream.h) in items of (up to 16 slots of one expert, 256
// columns, K split).  Workgroups take the items of the gated product first, then those of the
// second, by tickets.  h is two terms, rounded and what that leaves out, as in awq_moe_mlp.
//   - Splits of a gated tile meet in the workspace; the last to arrive adds them in order and writes h.
//   - An item of the second product waits until h of its slots is whole, with its first weights already
//     on their way.
//   - One token: no one joins the splits for all; an item of the second product adds and gates what it
//     multiplies.
//   - The last item of a column tile of the second product adds the slots and splits of every token in a fixed
//     order, and the residual, and writes y.
// What workgroups hand to each other goes through to, and comes from, where every XCD's L2 sees the
// same (kCpolDevice), and is counted in after it is complete.
//
// Every wait ends, whatever else runs on the card and however many workgroups are resident: a ticket
// is taken by a workgroup that runs, a gated item waits for nothing, and a workgroup begins with items
// of the second product only after it has seen that all gated items are taken (it may hold a ticket
// before: nobody waits for those).  So does a bound on the polls, behind which y is NaN.
// Tickets are eight lists, one per XCD as blocks go round them (one list: 18 ns for each workgroup in
// turn); who finds his own empty takes from the others.
//
// Bound (us, router and layer kernel): one token through 64 x 2048 -> 1408 top 8 (3 + 28, 36 MB) latency,
// of six steps that wait for each other: logits, routing, the gated product, its sums, the second
// product, its sums; one token
// through 8 x 4096 -> 14336 top 2 (5 + 53, 183 MB), 7 tokens of 64 x 2048 -> 1408 (8 + 53, 182 MB) and 16 of
// 8 x 4096 -> 14336 (6 + 152, 730 MB) HBM, at 3.4, 3.4 and 4.8 TB/s with the fill and drain of each phase;
// bfloat16 unpacks beside it.
#include "awq_epilogue.h"
#include "awq_route.h"
#include "awq_stream.h"

namespace awq {

using namespace stream;

namespace {

constexpr int kRouterWaves = kLayerTokens;  // a token each to route
constexpr int kRouterThreads = 64 * kRouterWaves;

constexpr uint32_t kMaxPolls = 1u << 18;  // a fifth of a second or more

__device__ __forceinline__ uint32_t load_count(const uint32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t count_in(uint32_t* p) {
  return __hip_atomic_fetch_add(p, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Stores of this wave are complete where every XCD sees them.
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A lane's share of the logits of TOKENS tokens (those past the last: the last again, so that no load
// waits behind a branch).
template <bool BF16, bool R32, int TOKENS>
__device__ __forceinline__ void dots(const LayerArgs& a, int e, int t0, int first, int step, float (&acc)[kLayerTokens]) {
  const char* row = static_cast<const char*>(a.router) + (int64_t)e * a.K * (R32 ? 4 : 2);
  const uint16_t* x[TOKENS];
#pragma unroll
  for (int t = 0; t < TOKENS; ++t) x[t] = a.x + (int64_t)min(t0 + t, a.T - 1) * a.K;
#pragma unroll 2
  for (int k = first; k < a.K; k += step) {
    u32x4 v[TOKENS];
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) v[t] = *reinterpret_cast<const u32x4*>(x[t] + k);
    float w[8];
    if constexpr (R32) {
      const floatx4* p = reinterpret_cast<const floatx4*>(row + 4 * (int64_t)k);
      const floatx4 lo = p[0], hi = p[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = lo[i], w[4 + i] = hi[i];
    } else {
      unpack8<BF16>(*reinterpret_cast<const u32x4*>(row + 2 * (int64_t)k), w);
    }
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
      float f[8];
      unpack8<BF16>(v[t], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[t] = fmaf(f[i], w[i], acc[t]);
    }
  }
}

template <bool BF16, bool R32>
__device__ __forceinline__ void dots(const LayerArgs& a, int e, int t0, int nt, int first, int step,
                                     float (&acc)[kLayerTokens]) {
  if (nt == 1) dots<BF16, R32, 1>(a, e, t0, first, step, acc);
  else dots<BF16, R32, kLayerTokens>(a, e, t0, first, step, acc);
}

}  // namespace

template <typename Key, typename Worth, int VPL, bool GROUPS>
__global__ __launch_bounds__(64 * kRouterWaves) void layer_router_kernel(const LayerArgs a, const RouteArgs r) {
  constexpr float kInf = __builtin_inff();
  __shared__ union {
    float part[kRouterWaves][kLayerTokens];
    struct {
      float l[64 * VPL];
      route::Scratch<Worth, 64, VPL, GROUPS> scratch;
    } of[kRouterWaves];
  } sh;
  __shared__ uint32_t last_arrival;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.y * kLayerTokens;
  const int nt = min(a.T - t0, kLayerTokens);
  // The other kernel's counts.
  for (int64_t i = (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * kRouterThreads + tid; i < a.n_counts;
       i += (int64_t)gridDim.x * gridDim.y * kRouterThreads)
    a.counts[i] = 0;

  const int per = kRouterWaves / a.router_waves;  // experts of a workgroup
  const int e = blockIdx.x * per + wave / a.router_waves, part = wave % a.router_waves;
  const int el = min(e, a.E - 1);
  float acc[kLayerTokens];
#pragma unroll
  for (int t = 0; t < kLayerTokens; ++t) acc[t] = 0.f;
  const int first = 8 * (part * 64 + lane), step = 512 * a.router_waves;
  if (a.bf16) a.router32 ? dots<true, true>(a, el, t0, nt, first, step, acc) : dots<true, false>(a, el, t0, nt, first, step, acc);
  else a.router32 ? dots<false, true>(a, el, t0, nt, first, step, acc) : dots<false, false>(a, el, t0, nt, first, step, acc);
#pragma unroll
  for (int t = 0; t < kLayerTokens; ++t) acc[t] = lanes_sum<64>(acc[t]);
  if (lane == 0) {
#pragma unroll
    for (int t = 0; t < kLayerTokens; ++t) sh.part[wave][t] = acc[t];
  }
  __syncthreads();
  if (part == 0 && lane < nt && e < a.E) {
    float v = sh.part[wave][lane];
    for (int w = 1; w < a.router_waves; ++w) v += sh.part[wave + w][lane];
    if (a.round_logits) v = a.bf16 ? act_to_float<true>(float_to_act<true>(v)) : act_to_float<false>(float_to_act<false>(v));
    __hip_atomic_store(a.logits + (int64_t)(t0 + lane) * a.E + e, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (a.route_inside) return;
  stores_done();
  __syncthreads();
  if (tid == 0) {
    const bool last = count_in(a.arrivals + blockIdx.y) == gridDim.x - 1;
    if (last) __hip_atomic_store(a.arrivals + blockIdx.y, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last_arrival = last;
  }
  __syncthreads();
  if (!last_arrival) return;

  // The LDS accesses of a wave are its own and in order; the compiler keeps them so.
  auto sync = [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); };
  for (int i = wave; i < nt; i += kRouterWaves) {
    const int t = t0 + i;
    float l[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int f = lane * VPL + j;
      const float v = __hip_atomic_load(a.logits + (int64_t)t * a.E + min(f, a.E - 1), __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
      l[j] = f < a.E ? v : -kInf;
    }
    sync();
#pragma unroll
    for (int j = 0; j < VPL; ++j) sh.of[wave].l[lane * VPL + j] = l[j];
    sync();
    route::route_tokens<Key, Worth, 64, VPL, GROUPS>(
        r, l, [&](int f) { return sh.of[wave].l[f]; }, sync, sh.of[wave].scratch, true, [&](int j, int id, float weight) {
          a.ids[t * a.topk + j] = id;
          a.weights[t * a.topk + j] = weight;
        });
    __builtin_amdgcn_wave_barrier();  // the lanes go round together
  }
}

// RL: lanes whose rows are kept, 16 per four rows; R: 1 for one token.
template <bool BF16, int RL, int R>
__global__ __launch_bounds__(64 * kStreamWaves, 2) void layer_kernel(const LayerArgs a, const RouteArgs r) {
  constexpr int WAVES = kStreamWaves, THREADS = 64 * WAVES;
  constexpr int SLOTS = kSlots<RL, WAVES>;
  constexpr int kEntryRows = 16;
  __shared__ union {
    Rows<R> red[WAVES][16][RL];
    float ys[RL / 4][kYld];
  } sh;
  __shared__ __attribute__((aligned(16))) uint16_t hs[2][R == 1 ? kLayerCols : 8];
  __shared__ int32_t slots[kEntryRows], ids[kExpertRankSlots];
  __shared__ float weights[kExpertRankSlots];
  __shared__ route::Scratch<float, 64, 1, false> chosen[WAVES];
  __shared__ int taken;
  __shared__ uint32_t last_arrival;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, c = lane & 15;
  const int S = a.T * a.topk;
  const int home = blockIdx.x & 7;
  uint32_t* const up_tickets = a.counts;
  uint32_t* const down_tickets = up_tickets + 8 * kLayerStride;
  uint32_t* const ready = down_tickets + 8 * kLayerStride;
  uint32_t* const down_counts = ready + kExpertRankSlots * kLayerStride;
  uint32_t* const up_counts = down_counts + a.down_tiles;

  // A ticket of one's own list, and how far the lists are, asked for ahead of when they are needed.
  struct Ticket {
    uint32_t mine, seen;  // (lane 0; lanes 0 to 7) of wave 0
  };
  auto ask = [&](uint32_t* tickets) {
    Ticket t{0, 0};
    if (wave == 0) {
      if (lane == 0) t.mine = count_in(tickets + kLayerStride * home);
      if (lane < 8) t.seen = load_count(tickets + kLayerStride * lane);
    }
    return t;
  };
  // The item of a ticket, of what the other lists have left if one's own is empty, or -1 when all of
  // them are.  Item i is in list i % 8.
  auto settle = [&](const Ticket& ticket, uint32_t* tickets, int total) {
    if (wave == 0) {
      int got = -1, list = home;
      uint32_t v = __builtin_amdgcn_readfirstlane(ticket.mine), seen = ticket.seen;
      for (;;) {
        const int n = (total - list + 7) >> 3;  // items of this list
        if (n > 0 && v < (uint32_t)n) {
          got = (int)v * 8 + list;
          break;
        }
        const uint64_t left = __ballot(lane < 8 && lane != list && (int64_t)seen < (int64_t)((total - lane + 7) >> 3));
        if (left == 0) break;
        // The next list after one's own that has something left.
        const uint32_t turned = (uint32_t)((left | left << 8) >> home) & 0xFFu;
        list = (home + __builtin_ctz(turned)) & 7;
        v = 0;
        if (lane == 0) v = count_in(tickets + kLayerStride * list);
        v = __builtin_amdgcn_readfirstlane(v);
        seen = lane < 8 ? load_count(tickets + kLayerStride * lane) : 0u;
      }
      if (lane == 0) taken = got;
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(taken);
  };
  // Each round of the loops below ends in a barrier.  It keeps the LDS of one item from the next, and
  // it keeps the lanes together: without one the compiler may carry a branch of thread 0's from a
  // round's end into the next round, and lanes that have to act as one no longer do.

  // Last of n arrivals at a count (the same answer in every thread); the workgroup's stores precede.
  auto last_of = [&](uint32_t* count, int n) {
    stores_done();
    __syncthreads();
    if (tid == 0) last_arrival = count_in(count) == (uint32_t)n - 1u;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane((int)last_arrival) != 0;
  };

  // Slots by expert, one per lane, in every wave: blocks of 16 slots of one expert are entries.
  // What routing needs is asked for first: loads come back in order, and the tickets' atomics take longer.
  Ticket ticket;
  int id;
  if (a.route_inside) {
    // A wave per token; the LDS accesses of a wave are its own and in order.  (Where the first kernel
    // routes, us: one token 64 x 2048 -> 1408 33.4, here 32.6; one of 8 x 4096 -> 14336 64.1, 63.4.)
    if (wave < a.T) {
      auto route = [&](auto vpl) {
        constexpr int VPL = decltype(vpl)::value;
        float l[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const int e = lane * VPL + j;
          l[j] = a.logits[(int64_t)wave * a.E + min(e, a.E - 1)];
        }
        ticket = ask(up_tickets);
#pragma unroll
        for (int j = 0; j < VPL; ++j) l[j] = lane * VPL + j < a.E ? l[j] : -__builtin_inff();
        route::route_tokens<float, float, 64, VPL, false>(
            r, l, [&](int e) { return a.logits[(int64_t)wave * a.E + e]; },
            [] { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); },
            chosen[wave], true,
            [&](int j, int e, float weight) {
              ids[wave * a.topk + j] = e;
              weights[wave * a.topk + j] = weight;
            });
      };
      if (a.E <= 64) route(std::integral_constant<int, 1>{});
      else route(std::integral_constant<int, 4>{});
    }
    __syncthreads();
    id = lane < S ? ids[lane] : -1;
  } else {
    id = lane < S ? a.ids[lane] : -1;
    const float weight = lane < S ? a.weights[lane] : 0.f;
    ticket = ask(up_tickets);
    if (wave == 0 && lane < S) {
      ids[lane] = id;
      weights[lane] = weight;
    }
  }
  const Ranks ranks = rank_slots<kEntryRows>(id, a.E);
  const int entries = ranks.entries;
  const int up_items = entries * a.up_tiles * a.up_splits, down_items = entries * a.down_tiles * a.down_splits;
  __syncthreads();

  // y of a column tile: every token's slots and splits, in order.  P threads share four columns, each
  // adding every P-th term.
  auto combine = [&](int tile) {
    int P = 1;
    while (P < 8 && 2 * P * a.T * (kExpertStreamCols / 4) <= THREADS) P *= 2;
    const int part = tid & (P - 1), terms = entries > 0 ? a.topk * a.down_splits : 0;
    const float per = 1.f / (float)a.down_splits;
    auto slot_of = [&](int term) { return (int)(((float)term + 0.5f) * per); };  // term / down_splits (< 2^12)
    const __amdgpu_buffer_rsrc_t srs = __builtin_amdgcn_make_buffer_rsrc(
        a.down_sums, (short)0, (int)((uint32_t)a.down_splits * (uint32_t)S * (uint32_t)a.N * 4u), 0x00020000);
    for (int i = tid / P; i < a.T * (kExpertStreamCols / 4); i += THREADS / P) {
      const int t = i / (kExpertStreamCols / 4);
      const int n = tile * kExpertStreamCols + 4 * (i % (kExpertStreamCols / 4));
      const bool live = n < a.N;
      const int64_t at = (int64_t)t * a.N + n;
      u32x2 res = {0u, 0u};
      if (a.residual != nullptr && live) res = *reinterpret_cast<const u32x2*>(a.residual + at);
      floatx4 sum = {0.f, 0.f, 0.f, 0.f};
      // Terms' loads by the eight, or four, at a time, routed or not (what no one wrote is dropped).
      auto add = [&](auto count, int i0) {
        constexpr int B = decltype(count)::value;
        floatx4 v[B];
        int s[B];
#pragma unroll
        for (int u = 0; u < B; ++u) {
          const int term = min(i0 + u * P, terms - 1);
          const int j = slot_of(term), sp = term - j * a.down_splits;
          s[u] = t * a.topk + j;
          v[u] = device_read<4>(srs, ((uint32_t)(sp * S + s[u]) * (uint32_t)a.N + (uint32_t)(live ? n : 0)) * 4u);
        }
#pragma unroll
        for (int u = 0; u < B; ++u)
          if (i0 + u * P < terms && ids[s[u]] >= 0) sum += weights[s[u]] * v[u];
      };
      int i0 = part;
      for (; i0 - part + 4 * P < terms; i0 += 8 * P) add(std::integral_constant<int, 8>{}, i0);
      if (i0 - part < terms) add(std::integral_constant<int, 4>{}, i0);
      for (int m = 1; m < P; m *= 2)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += __shfl_xor(sum[j], m);
      // A token without scores has NaN weights and no experts.
      const float lost = weights[t * a.topk] != weights[t * a.topk] ? weights[t * a.topk] : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += lost + act_to_float<BF16>((uint16_t)(res[j >> 1] >> (16 * (j & 1))));
      if (part == 0 && live)
        *reinterpret_cast<u32x2*>(a.y + at) = u32x2{pack_act2<BF16>(sum[0], sum[1]), pack_act2<BF16>(sum[2], sum[3])};
    }
  };
  if (entries == 0) {  // nobody goes anywhere
    for (int tile = blockIdx.x; tile < a.down_tiles; tile += gridDim.x) combine(tile);
    return;
  }
  const __amdgpu_buffer_rsrc_t hrs = __builtin_amdgcn_make_buffer_rsrc(
      a.h, (short)0, (int)(2u * (uint32_t)S * (uint32_t)a.inner * 2u), 0x00020000);
  const uint32_t rest_at = (uint32_t)S * (uint32_t)a.inner * 2u;  // the second term's bytes
  // One token: the gated product's sums, [slot][split][half][column].
  const __amdgpu_buffer_rsrc_t grs = __builtin_amdgcn_make_buffer_rsrc(
      a.up_sums, (short)0, (int)((uint32_t)(S * a.up_splits) * 2u * (uint32_t)a.inner * 4u), 0x00020000);
  auto gate_at = [&](int slot, int split, int hf, int n) {
    return ((uint32_t)((slot * a.up_splits + split) * 2 + hf) * (uint32_t)a.inner + (uint32_t)n) * 4u;
  };

  // ---- The gated product.
  Ticket next;  // of the second product
  bool asked = false;
  for (;;) {
    const int item = settle(ticket, up_tickets, up_items);
    if (item < 0) break;
    const int split = item % a.up_splits, tile = item / a.up_splits % a.up_tiles;
    const int entry = item / a.up_splits / a.up_tiles;
    const Entry en = entry_of<kEntryRows>(ranks, id, entry, lane, slots);
    __syncthreads();
    const int K = a.K, N = a.inner, half = wave & 1, NW = N >> 2, G = K / a.g_up;
    const int wc_in = tile * (kExpertStreamCols / 8) + 2 * c;
    const int wc = (wc_in < (N >> 3) ? wc_in : tile * (kExpertStreamCols / 8)) + half * (N >> 3);
    Share<1> share{a.up_qweight + (int64_t)en.expert * K * NW, a.up_qzeros + (int64_t)en.expert * G * NW,
                   a.up_scales + (int64_t)en.expert * G * NW * 8, NW, K, a.g_up, wc, a.x, nullptr, {}, 0, 0};
    share.x_off[0] = ((uint32_t)(slots[c < en.rows ? c : 0] / a.topk) * (uint32_t)K + 8u * q) * 2u;
    share.kb = min(K / 32, (split * kParts<true, WAVES> + (wave >> 1)) * a.up_steps);
    share.ke = min(K / 32, share.kb + a.up_steps);
    floatx4 part[1][16];
    half8v unit[2];
    stream_sums<BF16, 1, false>(share, Now{}, part, unit);
    ticket = ask(up_tickets);
    if (!asked) next = ask(down_tickets);
    asked = true;
    Rows<R> sum[SLOTS][2];
    wave_sums<true, RL, WAVES, R>(sh.red, part[0], unit, sum);
    if constexpr (R == 1) {
      // One token: its sums leave as they are, by column, and whoever takes a part of the second product
      // joins what it needs of them.
      const int n = tile * kExpertStreamCols + slot_col(tid);
      if (tid < 16 * RL && n < N) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) device_store<1>(grs, gate_at(slots[0], split, hf, n), sum[0][hf]);
      }
      stores_done();
      __syncthreads();
      if (tid == 0) count_in(ready + kLayerStride * entry);
      __syncthreads();
      continue;
    }
    bool mine = true;
    if (a.up_splits > 1) {
      constexpr uint32_t kShare = 2u * 16 * RL * 4u * R;
      const int64_t tile_at = (int64_t)entry * a.up_tiles + tile;
      const __amdgpu_buffer_rsrc_t prs = __builtin_amdgcn_make_buffer_rsrc(
          a.up_sums + tile_at * a.up_splits * (kShare / 4), (short)0, (int)(kShare * (uint32_t)a.up_splits), 0x00020000);
      // (Threads past the last slot, and slots of rows past the entry's, reach past the buffer.)
      auto at = [&](int sp, int k, int hf) {
        const int s = tid + k * THREADS;
        const bool none = (THREADS > 16 * RL && s >= 16 * RL) || slot_row(s) >= en.rows;
        return none ? kShare * (uint32_t)a.up_splits : (uint32_t)sp * kShare + (uint32_t)(hf * 16 * RL + s) * 4u * R;
      };
#pragma unroll
      for (int k = 0; k < SLOTS; ++k)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) device_store<R>(prs, at(split, k, hf), sum[k][hf]);
      mine = last_of(up_counts + tile_at, a.up_splits);
      if (mine) {
        Rows<R> flat[2 * SLOTS];
        device_sums<R>(prs, a.up_splits, [&](int sp, int i) { return at(sp, i / 2, i % 2); }, flat);
#pragma unroll
        for (int i = 0; i < 2 * SLOTS; ++i) sum[i / 2][i % 2] = flat[i];
      }
    } else {
      __syncthreads();  // the sums are in registers: their LDS takes h
    }
    if (mine) {
#pragma unroll
      for (int k = 0; k < SLOTS; ++k) {
        const int s = tid + k * THREADS;
        if (THREADS > 16 * RL && s >= 16 * RL) continue;
#pragma unroll
        for (int r = 0; r < R; ++r)
          sh.ys[slot_row(s) + r][slot_col(s)] = gated(row_of<R>(sum[k][0], r), row_of<R>(sum[k][1], r));
      }
      __syncthreads();
      const int n0 = tile * kExpertStreamCols;
      for (int i = tid; i < en.rows * (kExpertStreamCols / 8); i += THREADS) {
        const int row = i / (kExpertStreamCols / 8), cp = 8 * (i % (kExpertStreamCols / 8));
        if (n0 + cp >= N) continue;
        const float* v = &sh.ys[row][cp];
        u32x4 term, rest;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          term[j] = pack_act2<BF16>(v[2 * j], v[2 * j + 1]);
          rest[j] = pack_act2<BF16>(rest_of<BF16>(v[2 * j]), rest_of<BF16>(v[2 * j + 1]));
        }
        const uint32_t at = ((uint32_t)slots[row] * (uint32_t)N + (uint32_t)(n0 + cp)) * 2u;
        __builtin_amdgcn_raw_buffer_store_b128(term, hrs, at, 0, kCpolDevice);
        __builtin_amdgcn_raw_buffer_store_b128(rest, hrs, at + rest_at, 0, kCpolDevice);
      }
      stores_done();
      __syncthreads();
      if (tid == 0) count_in(ready + kLayerStride * entry);
    }
    __syncthreads();
  }
  if (!asked) next = ask(down_tickets);
  __syncthreads();  // `taken` has been read

  // ---- The second product.
  for (;;) {
    const int item = settle(next, down_tickets, down_items);
    if (item < 0) break;
    const int split = item % a.down_splits, tile = item / a.down_splits % a.down_tiles;
    const int entry = item / a.down_splits / a.down_tiles;
    const Entry en = entry_of<kEntryRows>(ranks, id, entry, lane, slots);
    __syncthreads();
    const int K = a.inner, N = a.N, NW = N >> 3, G = K / a.g_down;
    const int wc_in = tile * (kExpertStreamCols / 8) + 2 * c;
    const int wc = wc_in < NW ? wc_in : tile * (kExpertStreamCols / 8);
    Share<1> share{a.down_qweight + (int64_t)en.expert * K * NW, a.down_qzeros + (int64_t)en.expert * G * NW,
                   a.down_scales + (int64_t)en.expert * G * NW * 8, NW, K, a.g_down, wc, a.h,
                   a.h + (int64_t)S * a.inner, {}, 0, 0};
    share.x_off[0] = ((uint32_t)slots[c < en.rows ? c : 0] * (uint32_t)K + 8u * q) * 2u;
    share.kb = min(K / 32, (split * kParts<false, WAVES> + wave) * a.down_steps);
    share.ke = min(K / 32, share.kb + a.down_steps);
    bool whole = true;
    const uint32_t parts_of_h = (uint32_t)(R == 1 ? a.up_tiles * a.up_splits : a.up_tiles);
    auto wait = [&] {
      uint32_t polls = 0;
      while (load_count(ready + kLayerStride * entry) < parts_of_h) {
        if (++polls == kMaxPolls) {
          whole = false;
          break;
        }
        __builtin_amdgcn_s_sleep(1);
      }
      asm volatile("" ::: "memory");  // nothing of h is read before
    };
    floatx4 part[1][16];
    half8v unit[2];
    if constexpr (R == 1) {
      // This split's part of h, joined and gated into LDS; four columns a thread at a time.
      const int k0 = split * WAVES * a.down_steps * 32, cols = min(K - k0, WAVES * a.down_steps * 32);
      const int slot = slots[0];
      auto join = [&] {
        wait();
        for (int c0 = tid; c0 < cols; c0 += 4 * THREADS) {
          float flat[8];
          device_sums<1>(grs, a.up_splits, [&](int sp, int i) {
            return gate_at(slot, sp, i & 1, k0 + min(c0 + (i >> 1) * THREADS, cols - 1));
          }, flat);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = c0 + j * THREADS;
            const float h = gated(flat[2 * j], flat[2 * j + 1]);
            if (at < cols) {
              hs[0][at] = float_to_act<BF16>(h);
              hs[1][at] = float_to_act<BF16>(rest_of<BF16>(h));
            }
          }
        }
        __syncthreads();
      };
      stream_sums<BF16, 1, true>(share, join, part, unit, [&](int k, bool rest) {
        return *reinterpret_cast<const half8v*>(&hs[rest][k - k0]);
      });
    } else {
      stream_sums<BF16, 1, true>(share, wait, part, unit);
    }
    next = ask(down_tickets);
    if (!whole) {
#pragma unroll
      for (int v = 0; v < 16; ++v) part[0][v] = floatx4{__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
    }
    Rows<R> sum[SLOTS][1];
    wave_sums<false, RL, WAVES, R>(sh.red, part[0], unit, sum);
    __syncthreads();  // the sums are in registers: their LDS takes the output rows
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
      const int s = tid + k * THREADS;
      if (THREADS > 16 * RL && s >= 16 * RL) continue;
#pragma unroll
      for (int r = 0; r < R; ++r) sh.ys[slot_row(s) + r][slot_col(s)] = row_of<R>(sum[k][0], r);
    }
    __syncthreads();
    const int n0 = tile * kExpertStreamCols;
    const __amdgpu_buffer_rsrc_t srs = __builtin_amdgcn_make_buffer_rsrc(
        a.down_sums, (short)0, (int)((uint32_t)a.down_splits * (uint32_t)S * (uint32_t)N * 4u), 0x00020000);
    for (int i = tid; i < en.rows * (kExpertStreamCols / 4); i += THREADS) {
      const int row = i / (kExpertStreamCols / 4), cp = 4 * (i % (kExpertStreamCols / 4));
      if (n0 + cp >= N) continue;
      device_store<4>(srs, ((uint32_t)(split * S + slots[row]) * (uint32_t)N + (uint32_t)(n0 + cp)) * 4u,
                      *reinterpret_cast<const floatx4*>(&sh.ys[row][cp]));
    }
    if (last_of(down_counts + tile, entries * a.down_splits)) combine(tile);
    __syncthreads();
  }
}

hipError_t launch_layer(LayerArgs a, const RouteArgs& r, const LayerPlan& p, hipStream_t stream) {
  if (a.router_waves < 1 || kRouterWaves % a.router_waves != 0) return hipErrorInvalidValue;  // whole experts a workgroup
  const dim3 grid((unsigned)((a.E * a.router_waves + kRouterWaves - 1) / kRouterWaves), (unsigned)((a.T + kLayerTokens - 1) / kLayerTokens));
  // Routing by the logits alone, of few tokens and experts, takes every workgroup of the second kernel
  // less time than handing the ids over takes the first.
  a.route_inside = r.bias == nullptr && r.groups == 1 && a.E <= 256 && a.T <= kStreamWaves;
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(kRouterThreads), 0, stream, a, r); };
  auto sized = [&](auto key, auto worth, auto groups) {
    using Key = decltype(key);
    using Worth = decltype(worth);
    constexpr bool G = decltype(groups)::value;
    if (a.E <= 64) go(layer_router_kernel<Key, Worth, 1, G>);
    else if (a.E <= 256) go(layer_router_kernel<Key, Worth, 4, G>);
    else go(layer_router_kernel<Key, Worth, 16, G>);
  };
  using yes = std::true_type;
  using no = std::false_type;
  // Which keys need fp64: awq_route.h.
  if (r.bias != nullptr) r.groups > 1 ? sized(double{}, double{}, yes{}) : sized(double{}, double{}, no{});
  else if (r.groups > 1 && r.group_top == 2) sized(float{}, double{}, yes{});
  else r.groups > 1 ? sized(float{}, float{}, yes{}) : sized(float{}, float{}, no{});
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  auto main_kernel = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)p.workgroups), dim3(64 * kStreamWaves), 0, stream, a, r);
  };
  auto by_rows = [&](auto bf16) {
    constexpr bool B = decltype(bf16)::value;
    if (p.rows == 1) main_kernel(layer_kernel<B, 16, 1>);
    else if (p.rows == 4) main_kernel(layer_kernel<B, 16, 4>);
    else if (p.rows == 8) main_kernel(layer_kernel<B, 32, 4>);
    else main_kernel(layer_kernel<B, 64, 4>);
  };
  a.bf16 ? by_rows(yes{}) : by_rows(no{});
  return hipGetLastError();
}

}  // namespace awq
