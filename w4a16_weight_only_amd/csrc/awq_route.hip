// Routing of tokens to experts: scores, a balancing bias, groups, top-k, weights.
//
// Per token, over its E logits l:
//   score   s_e = exp(l_e) / sum_f exp(l_f)  or  1 / (1 + exp(-l_e))
//   choice  c_e = s_e + bias_e; an expert with l_e = -inf or c_e = -inf is never chosen
//   groups  of E / G consecutive experts, worth their largest c or the sum of their two
//           largest (of the one, where only one can be chosen); the best topk_groups stay
//   ids     the topk experts by c, largest first, ties to the lowest index (groups too);
//           -1 where nothing is left to choose
//   weight  s of the chosen (without the bias), divided by their sum on request, times scale
//
// Order.  Without a bias and with groups worth their best expert, every comparison is one
// of scores, and s rises strictly with l: the logits themselves are the keys, exact in
// fp32, and two experts tie exactly when their logits do.  A bias or a sum of two scores
// has to be added up, and in fp32 the sum's rounding (2^-25 of a score near 1) would swap
// experts that close together: those keys are formed in fp64.
// Weights.  Renormalised scores are quotients, so a common factor is taken out first:
// exp(l - max over the chosen) instead of the softmax, and exp(min(l, 0) - min(max, 0)) /
// (1 + exp(-|l|)) for the sigmoid, so that scores too small for fp32 still divide.
//
// One token per LPT lanes, each lane holding VPL consecutive experts in registers (lanes in
// index order, so a tie goes to the lowest lane); topk rounds of a maximum over the lanes.
#include "awq_device.h"
#include "awq_kernels.h"

namespace awq {

namespace {

constexpr int kRouteThreads = 256;

__device__ __forceinline__ float load_logit(const void* p, int type, int64_t i) {
  if (type == 2) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return type == 1 ? bf16_bits_to_float(b) : act_to_float<false>(b);
}

template <int LPT, typename V>
__device__ __forceinline__ V lanes_max(V v) {
#pragma unroll
  for (int d = LPT / 2; d > 0; d /= 2) {
    const V o = __shfl_xor(v, d, LPT);
    v = o > v ? o : v;
  }
  return v;
}
template <int LPT, typename V>
__device__ __forceinline__ V lanes_sum(V v) {
#pragma unroll
  for (int d = LPT / 2; d > 0; d /= 2) v += __shfl_xor(v, d, LPT);
  return v;
}

}  // namespace

// Key: float (keys are the logits) or double (keys are choices).  GROUPS: expert groups.
template <typename Key, int LPT, int VPL, bool GROUPS>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const RouteArgs a) {
  constexpr int TOKENS = kRouteThreads / LPT;  // tokens per workgroup
  constexpr bool kChoice = sizeof(Key) == 8;
  __shared__ Key keys_lds[GROUPS ? TOKENS * LPT * VPL : 1];
  const Key kNone = -(Key)__builtin_inff();
  const int lane = threadIdx.x & 63;
  const int p = threadIdx.x % LPT;  // lane within the token
  const int slot = threadIdx.x / LPT;
  const int64_t t_raw = (int64_t)blockIdx.x * TOKENS + slot;
  const bool live = t_raw < a.T;
  const int64_t t = live ? t_raw : a.T - 1;  // lanes past the last token redo it and store nothing
  const int64_t row = t * a.row_stride;
  const int lane0 = lane & ~(LPT - 1);
  auto vote = [&](bool b) {
    return (uint64_t)(__ballot(b) >> lane0) & (LPT == 64 ? ~0ull : (1ull << (LPT & 63)) - 1);
  };

  float l[VPL];
  float top = -__builtin_inff();
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = p * VPL + i;
    l[i] = e < a.E ? load_logit(a.logits, a.type, row + e) : -__builtin_inff();
    bad |= l[i] != l[i] || (a.softmax && l[i] == __builtin_inff());
    top = fmaxf(top, l[i]);
  }
  // A row with a NaN (or, for the softmax, +inf) has no scores: it goes nowhere.
  const bool lost = vote(bad) != 0;
  top = lanes_max<LPT>(top);

  Key key[VPL];
  if constexpr (kChoice) {
    double z = 0.0, s[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const double d = (double)l[i];
      s[i] = l[i] == -__builtin_inff() ? 0.0 : a.softmax ? exp(d - (double)top) : 1.0 / (1.0 + exp(-d));
      z += s[i];
    }
    z = lanes_sum<LPT>(z);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = p * VPL + i;
      const double c = (a.softmax ? s[i] / z : s[i]) + (a.bias != nullptr && e < a.E ? (double)a.bias[e] : 0.0);
      key[i] = l[i] == -__builtin_inff() || c != c ? kNone : c;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = l[i];
  }

  if constexpr (GROUPS) {
    // Lane g < G scans group g's keys in LDS; then the best groups are drawn like experts.
    Key* mine = keys_lds + slot * LPT * VPL;
#pragma unroll
    for (int i = 0; i < VPL; ++i) mine[p * VPL + i] = key[i];
    __syncthreads();
    const int per = a.E / a.groups;
    uint64_t keep = 0;  // groups that stay, one bit each
    Key worth[64 / LPT];
#pragma unroll
    for (int r = 0; r < 64 / LPT; ++r) {
      const int g = r * LPT + p;
      Key b1 = kNone, b2 = kNone;
      if (g < a.groups)
        for (int i = 0; i < per; ++i) {
          const Key k = mine[g * per + i];
          b2 = k > b1 ? b1 : (k > b2 ? k : b2);
          b1 = k > b1 ? k : b1;
        }
      worth[r] = a.group_top == 2 && b2 != kNone ? b1 + b2 : b1;
    }
    for (int j = 0; j < a.topk_groups; ++j) {
      Key m = kNone;
#pragma unroll
      for (int r = 0; r < 64 / LPT; ++r) m = worth[r] > m ? worth[r] : m;
      m = lanes_max<LPT>(m);
      if (m == kNone) break;
      bool taken = false;
#pragma unroll
      for (int r = 0; r < 64 / LPT; ++r) {
        const uint64_t who = vote(!taken && worth[r] == m);
        if (who != 0) {
          const int w = __builtin_ctzll(who);
          if (!taken) keep |= 1ull << (r * LPT + w);
          if (!taken && p == w) worth[r] = kNone;
          taken = true;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = p * VPL + i;
      if (e >= a.E || ((keep >> (e / per)) & 1) == 0) key[i] = kNone;
    }
  }

  // topk rounds; lane j % LPT of the token keeps the expert of rounds j = lane, lane + LPT, ...
  int got[64 / LPT];
#pragma unroll
  for (int r = 0; r < 64 / LPT; ++r) got[r] = -1;
  if (!lost)
    for (int j = 0; j < a.topk; ++j) {
      Key m = key[0];
      int at = 0;
#pragma unroll
      for (int i = 1; i < VPL; ++i)
        if (key[i] > m) {
          m = key[i];
          at = i;
        }
      const Key best = lanes_max<LPT>(m);
      if (best == kNone) break;
      const int w = __builtin_ctzll(vote(m == best));
      const int e = __shfl(p * VPL + at, w, LPT);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (p == w && i == at) key[i] = kNone;
#pragma unroll
      for (int r = 0; r < 64 / LPT; ++r)
        if (j == r * LPT + p) got[r] = e;
    }

  // Weights.
  float lj[64 / LPT];
  float far = -__builtin_inff();
#pragma unroll
  for (int r = 0; r < 64 / LPT; ++r) {
    lj[r] = got[r] >= 0 ? load_logit(a.logits, a.type, row + got[r]) : -__builtin_inff();
    far = fmaxf(far, lj[r]);
  }
  far = lanes_max<LPT>(far);
  float w[64 / LPT];
  float sum = 0.f;
  // What the exponent is taken relative to: the largest chosen logit where the weights are
  // divided by their sum, else the softmax's own maximum (and nothing for the sigmoid).
  const float ref = a.softmax ? (a.renormalize ? far : top) : (a.renormalize ? fminf(far, 0.f) : 0.f);
#pragma unroll
  for (int r = 0; r < 64 / LPT; ++r) {
    const float v = a.softmax ? expf(lj[r] - ref) : expf(fminf(lj[r], 0.f) - ref) / (1.f + expf(-fabsf(lj[r])));
    w[r] = got[r] >= 0 ? v : 0.f;
    sum += w[r];
  }
  if (a.renormalize) {
    sum = lanes_sum<LPT>(sum);
  } else {
    sum = 1.f;
    if (a.softmax) {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) z += l[i] == -__builtin_inff() ? 0.f : expf(l[i] - top);
      sum = lanes_sum<LPT>(z);
    }
  }
#pragma unroll
  for (int r = 0; r < 64 / LPT; ++r) {
    const int j = r * LPT + p;
    if (live && j < a.topk) {
      a.ids[t * a.topk + j] = got[r];
      a.weights[t * a.topk + j] =
          lost ? __builtin_nanf("") : got[r] >= 0 ? w[r] / sum * a.scale : 0.f;
    }
  }
}

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  // Keys need fp64 where scores are added to something (see the top of the file).
  const bool choice = a.bias != nullptr || (a.groups > 1 && a.group_top == 2);
  auto go = [&](auto kern, int lpt) {
    const int64_t tokens = kRouteThreads / lpt;
    hipLaunchKernelGGL(kern, dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(kRouteThreads), 0, stream, a);
  };
#define AWQ_ROUTE(KEY, LPT, VPL)                              \
  do {                                                        \
    if (a.groups > 1) go(route_kernel<KEY, LPT, VPL, true>, LPT); \
    else go(route_kernel<KEY, LPT, VPL, false>, LPT);         \
  } while (0)
#define AWQ_ROUTE_E(KEY)                          \
  do {                                            \
    if (a.E <= 64) AWQ_ROUTE(KEY, 64, 1);         \
    else if (a.E <= 128) AWQ_ROUTE(KEY, 64, 2);   \
    else if (a.E <= 256) AWQ_ROUTE(KEY, 64, 4);   \
    else if (a.E <= 512) AWQ_ROUTE(KEY, 64, 8);   \
    else AWQ_ROUTE(KEY, 64, 16);                  \
  } while (0)
  if (choice) AWQ_ROUTE_E(double);
  else AWQ_ROUTE_E(float);
#undef AWQ_ROUTE_E
#undef AWQ_ROUTE
  return hipGetLastError();
}

}  // namespace awq
