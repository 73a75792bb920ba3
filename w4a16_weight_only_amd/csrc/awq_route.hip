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
// Order.  Without a bias the comparison of experts is one of scores, and s rises strictly with l:
// the logits themselves are the keys, exact in fp32, and two experts tie exactly when their
// logits do.  A bias has to be added up, and in fp32 the sum's rounding (2^-25 of a score near 1)
// would swap experts that close together: those keys are formed in fp64.  So are the sums of two
// scores that groups may be worth, whose experts then still go by their logits without a bias.
// Weights.  Renormalised scores are quotients, so a common factor is taken out first:
// exp(l - max over the chosen) instead of the softmax, and exp(min(l, 0) - min(max, 0)) /
// (1 + exp(-|l|)) for the sigmoid, so that scores too small for fp32 still divide.  They are formed
// in fp32, their type: off by 6e-8 of their size on the measured cases, where one rounding is 3e-8
// (in fp64, us fp32 / fp64: 16384 tokens of 128 experts 7.7 / 8.5, not divided 8.5 / 10.8).
//
// One token per LPT lanes (16: four tokens a wave, for many tokens; else 64), each lane
// holding VPL consecutive experts in registers, lanes in index order, so a tie goes to the
// lowest lane; topk rounds of a maximum over the lanes, which never leaves the registers
// (rotations within 16 lanes, row swaps across them).  The winning lane alone notes its
// expert, in LDS, and strikes it out.  Groups are ranked by counting the better ones.
#include <type_traits>

#include "awq_device.h"
#include "awq_kernels.h"
#include "awq_lanes.h"

namespace awq {

namespace {

constexpr int kRouteThreads = 64;
constexpr int64_t kRouteFewTokens = 2048;

template <int TYPE>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (TYPE == 2) return static_cast<const float*>(p)[i];
  else return act_to_float<TYPE == 1>(static_cast<const uint16_t*>(p)[i]);
}

// The two largest keys seen.
template <typename Key>
struct Two {
  Key first, second;
  __device__ void add(Key k) {
    second = larger(second, k < first ? k : first);
    first = larger(first, k);
  }
  __device__ void add(const Two& o) {
    add(o.first);
    second = larger(second, o.second);
  }
};

}  // namespace

// Key: float (keys are the logits) or double (keys are choices).  Worth, of groups: float (their
// best logit) or double (choices).  GROUPS: expert groups.  TYPE of the logits: 0 fp16, 1
// bfloat16, 2 fp32.
template <typename Key, typename Worth, int LPT, int VPL, bool GROUPS, int TYPE>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const RouteArgs a) {
  constexpr int TOKENS = kRouteThreads / LPT;  // tokens per workgroup (one wave)
  constexpr bool kChoice = sizeof(Key) == 8, kScores = sizeof(Worth) == 8;
  constexpr int kOut = 64 / LPT;  // experts a lane stores, LPT apart
  constexpr float kInf = __builtin_inff();
  __shared__ Worth keys_lds[GROUPS ? TOKENS * LPT * VPL : 1];
  __shared__ Worth worth[GROUPS ? TOKENS : 1][kRouteMaxGroups];
  __shared__ int chosen[TOKENS][kRouteMaxTopk];
  const Key kNone = -(Key)kInf;
  const int lane = threadIdx.x;
  const int p = lane % LPT;  // lane within the token
  const int slot = lane / LPT;
  const int64_t t_raw = (int64_t)blockIdx.x * TOKENS + slot;
  const bool live = t_raw < a.T;
  const int64_t t = live ? t_raw : a.T - 1;  // lanes past the last token redo it and store nothing
  const int64_t row = t * a.row_stride;
  const int lane0 = lane & ~(LPT - 1);
  auto vote = [&](bool b) {
    return (uint64_t)(__ballot(b) >> lane0) & (LPT == 64 ? ~0ull : (1ull << (LPT & 63)) - 1);
  };
  for (int j = p; j < a.topk; j += LPT) chosen[slot][j] = -1;

  float l[VPL];
  constexpr int kSize = TYPE == 2 ? 4 : 2;
  constexpr int kPiece = VPL * kSize < 16 ? VPL * kSize : 16;  // bytes of a wide load
  if (a.wide && kPiece >= 4) {  // every lane's experts lie on whole pieces, all inside or all outside
    const bool in = p * VPL < a.E;
    const char* at = static_cast<const char*>(a.logits) + (row + (in ? p * VPL : 0)) * kSize;
    struct alignas(kPiece < 4 ? 4 : kPiece) Piece {
      uint32_t w[kPiece < 4 ? 1 : kPiece / 4];
    };
#pragma unroll
    for (int c = 0; c < VPL * kSize / kPiece; ++c) {
      const Piece d = reinterpret_cast<const Piece*>(at)[c];
#pragma unroll
      for (int i = 0; i < kPiece / kSize; ++i) {
        const uint32_t w = d.w[i * kSize / 4];
        const float v = TYPE == 2 ? __builtin_bit_cast(float, w)
                                  : act_to_float<TYPE == 1>((uint16_t)(w >> (16 * (i & 1))));
        l[c * (kPiece / kSize) + i] = in ? v : -kInf;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = p * VPL + i;
      const float v = load_logit<TYPE>(a.logits, row + (e < a.E ? e : 0));
      l[i] = e < a.E ? v : -kInf;
    }
  }
  float top = -kInf;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    bad |= l[i] != l[i] || (a.softmax && l[i] == kInf);
    top = fmaxf(top, l[i]);
  }
  // A row with a NaN (or, for the softmax, +inf) has no scores: it goes nowhere.
  const bool lost = vote(bad) != 0;
  top = lanes_max<LPT>(top);

  Key key[VPL];
  Worth val[VPL];  // what groups are worth the largest of
  if constexpr (kScores) {
    double z = 0.0, s[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const double d = (double)l[i];
      s[i] = l[i] == -kInf ? 0.0 : a.softmax ? exp(d - (double)top) : 1.0 / (1.0 + exp(-d));
      z += s[i];
    }
    z = a.softmax ? 1.0 / lanes_sum<LPT>(z) : 1.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = p * VPL + i;
      const double c = s[i] * z + (a.bias != nullptr && e < a.E ? (double)a.bias[e] : 0.0);
      val[i] = l[i] == -kInf || c != c ? -(Worth)kInf : c;
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if constexpr (kChoice) key[i] = val[i];
    else key[i] = lost ? kNone : l[i];
    if constexpr (!kScores) val[i] = key[i];
  }

  if constexpr (GROUPS) {
    // Worths.  Groups of whole lanes, a power of two of them within 16: the lanes' two largest
    // meet in registers.  Otherwise lane g (and g + LPT, ...) scans group g's keys in LDS.
    const int per = a.E / a.groups;
    const int width = per / VPL;  // lanes of a group
    const bool whole = per % VPL == 0 && width <= 16 && (width & (width - 1)) == 0;
    const Worth kNothing = -(Worth)kInf;
    auto value = [&](const Two<Worth>& b) {
      return a.group_top == 2 && b.second != kNothing ? b.first + b.second : b.first;
    };
    if (whole) {
      Two<Worth> b{kNothing, kNothing};
#pragma unroll
      for (int i = 0; i < VPL; ++i) b.add(val[i]);
      auto meet = [&](auto ctrl) {
        constexpr int C = decltype(ctrl)::value;
        b.add(Two<Worth>{rotated<C>(b.first), rotated<C>(b.second)});
      };
      if (width >= 2) meet(std::integral_constant<int, 0xB1>{});   // lane ^ 1
      if (width >= 4) meet(std::integral_constant<int, 0x4E>{});   // lane ^ 2
      if (width >= 8) meet(std::integral_constant<int, 0x141>{});  // mirrored in 8: the other four
      if (width >= 16) meet(std::integral_constant<int, 0x140>{});  // mirrored in 16: the other eight
      if (p % width == 0 && p / width < a.groups) worth[slot][p / width] = value(b);
    } else {
      Worth* mine = keys_lds + slot * LPT * VPL;
#pragma unroll
      for (int i = 0; i < VPL; ++i) mine[p * VPL + i] = val[i];
      __syncthreads();
      for (int g = p; g < a.groups; g += LPT) {
        Two<Worth> b{kNothing, kNothing};
#pragma unroll 8
        for (int i = 0; i < per; ++i) b.add(mine[g * per + i]);
        worth[slot][g] = value(b);
      }
    }
    __syncthreads();
    uint64_t keep = 0;  // groups that stay, one bit each: fewer than topk_groups are better
#pragma unroll
    for (int r = 0; r < kOut; ++r) {
      const int g = r * LPT + p;
      const Worth mine = worth[slot][g < a.groups ? g : 0];
      int better = 0;
      for (int o = 0; o < a.groups; ++o) {
        const Worth k = worth[slot][o];
        better += k > mine || (k == mine && o < g) ? 1 : 0;
      }
      keep |= vote(g < a.groups && better < a.topk_groups) << (r * LPT);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = p * VPL + i;
      if (e >= a.E || ((keep >> (e / per)) & 1) == 0) key[i] = kNone;
    }
  }
  __syncthreads();  // the slots of `chosen` are cleared

  // topk rounds.  A token without a choice left keeps -1 in the rest.
  if (!lost)
    for (int j = 0; j < a.topk; ++j) {
      Key m = key[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) m = larger(m, key[i]);
      const Key best = lanes_max<LPT>(m);
      const int w = __builtin_ctzll(vote(m == best));
      if (best != kNone && p == w) {
        int at = 0;
        bool struck = false;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const bool hit = !struck && key[i] == best;
          at = hit ? i : at;
          key[i] = hit ? kNone : key[i];
          struck |= hit;
        }
        chosen[slot][j] = p * VPL + at;
      }
    }
  __syncthreads();

  // Weights: lane j % LPT of the token has the experts of rounds j = lane, lane + LPT, ...
  int got[kOut];
  float lj[kOut];
  float far = -kInf;
#pragma unroll
  for (int r = 0; r < kOut; ++r) {
    const int j = r * LPT + p;
    got[r] = j < a.topk ? chosen[slot][j] : -1;
    lj[r] = got[r] >= 0 ? load_logit<TYPE>(a.logits, row + got[r]) : -kInf;
    far = fmaxf(far, lj[r]);
  }
  far = lanes_max<LPT>(far);
  float w[kOut];
  float sum = 0.f;
  // What the exponent is taken relative to: the largest chosen logit where the weights are
  // divided by their sum, else the softmax's own maximum (and nothing for the sigmoid).
  const float ref = a.softmax ? (a.renormalize ? far : top) : (a.renormalize ? fminf(far, 0.f) : 0.f);
#pragma unroll
  for (int r = 0; r < kOut; ++r) {
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
      for (int i = 0; i < VPL; ++i) z += l[i] == -kInf ? 0.f : expf(l[i] - top);
      sum = lanes_sum<LPT>(z);
    }
  }
#pragma unroll
  for (int r = 0; r < kOut; ++r) {
    const int j = r * LPT + p;
    if (live && j < a.topk) {
      a.ids[t * a.topk + j] = got[r];
      a.weights[t * a.topk + j] = lost ? __builtin_nanf("") : got[r] >= 0 ? w[r] / sum * a.scale : 0.f;
    }
  }
}

hipError_t launch_route(RouteArgs a, hipStream_t stream) {
  // Keys and worths need fp64 where scores are added to something (see the top of the file).
  const bool choice = a.bias != nullptr, scores = choice || (a.groups > 1 && a.group_top == 2);
  auto go = [&](auto kern, int lpt, int vpl) {
    const int64_t tokens = kRouteThreads / lpt;
    // Wide loads: rows and lanes start on whole pieces, and E ends on one.
    const int size = a.type == 2 ? 4 : 2;
    const int piece = vpl * size < 16 ? vpl * size : 16;
    a.wide = a.E % vpl == 0 && reinterpret_cast<uintptr_t>(a.logits) % piece == 0 &&
             (a.T == 1 || a.row_stride * size % piece == 0);
    hipLaunchKernelGGL(kern, dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(kRouteThreads), 0, stream, a);
  };
  auto typed = [&](auto key, auto worth_of, auto groups, auto lpt, auto vpl) {
    using Key = decltype(key);
    using Worth = decltype(worth_of);
    constexpr bool G = decltype(groups)::value;
    constexpr int L = decltype(lpt)::value, V = decltype(vpl)::value;
    if (a.type == 2) go(route_kernel<Key, Worth, L, V, G, 2>, L, V);
    else if (a.type == 1) go(route_kernel<Key, Worth, L, V, G, 1>, L, V);
    else go(route_kernel<Key, Worth, L, V, G, 0>, L, V);
  };
  auto sized = [&](auto key, auto worth, auto groups) {
    using I4 = std::integral_constant<int, 4>;
    using I8 = std::integral_constant<int, 8>;
    using I16 = std::integral_constant<int, 16>;
    using I64 = std::integral_constant<int, 64>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    // Few tokens: a wave each, the shortest way through; many: four a wave, the fewest
    // instructions.  Measured, us, a wave each / four a wave: 512 tokens of 128 experts 4.5 / 5.2,
    // 4096 6.4 / 5.5, 16384 14.6 / 7.5 (a third of a copy's rate); 16 fp64 keys a lane do not
    // pay: 512 tokens of 256 experts in 8 groups 7.4 / 15.6, 16384 32.4 / 36.5.
    if (a.T <= kRouteFewTokens || (sizeof(worth) == 8 && a.E > 128)) {
      if (a.E <= 64) typed(key, worth, groups, I64{}, I1{});
      else if (a.E <= 128) typed(key, worth, groups, I64{}, I2{});
      else if (a.E <= 256) typed(key, worth, groups, I64{}, I4{});
      else if (a.E <= 512) typed(key, worth, groups, I64{}, I8{});
      else typed(key, worth, groups, I64{}, I16{});
    } else {
      if (a.E <= 64) typed(key, worth, groups, I16{}, I4{});
      else if (a.E <= 128) typed(key, worth, groups, I16{}, I8{});
      else if (a.E <= 256) typed(key, worth, groups, I16{}, I16{});
      else if (a.E <= 512) typed(key, worth, groups, I64{}, I8{});
      else typed(key, worth, groups, I64{}, I16{});
    }
  };
  using yes = std::true_type;
  using no = std::false_type;
  if (choice) a.groups > 1 ? sized(double{}, double{}, yes{}) : sized(double{}, double{}, no{});
  else if (scores) sized(float{}, double{}, yes{});
  else a.groups > 1 ? sized(float{}, float{}, yes{}) : sized(float{}, float{}, no{});
  return hipGetLastError();
}

}  // namespace awq
