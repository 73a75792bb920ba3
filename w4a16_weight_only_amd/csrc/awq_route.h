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
#pragma once

#include <type_traits>

#include "awq_device.h"
#include "awq_kernels.h"
#include "awq_lanes.h"

namespace awq {
namespace route {

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

// LDS of the tokens of one wave.
template <typename Worth, int LPT, int KEYS>
struct ScratchOf {
  static constexpr int kTokens = 64 / LPT;
  Worth keys[KEYS > 1 ? kTokens : 1][KEYS];
  Worth worth[KEYS > 1 ? kTokens : 1][kRouteMaxGroups];
  int chosen[kTokens][kRouteMaxTopk];
};
template <typename Worth, int LPT, int VPL, bool GROUPS>
using Scratch = ScratchOf<Worth, LPT, GROUPS ? LPT * VPL : 1>;

// Key: float (keys are the logits) or double (keys are choices).  Worth, of groups: float (their
// best logit) or double (choices).  GROUPS: expert groups.  One token per LPT lanes of a wave: l holds
// this lane's VPL experts (-inf past the last), logit(e) is that of expert e, put(j, id, weight) takes
// slot j's result, where live; sync() orders the wave's LDS accesses.
template <typename Key, typename Worth, int LPT, int VPL, bool GROUPS, typename Logit, typename Sync, typename Put>
__device__ __forceinline__ void route_tokens(const RouteArgs& a, const float (&l)[VPL], Logit logit, Sync sync,
                                             Scratch<Worth, LPT, VPL, GROUPS>& lds, bool live, Put put) {
  constexpr bool kChoice = sizeof(Key) == 8, kScores = sizeof(Worth) == 8;
  constexpr int kOut = 64 / LPT;  // experts a lane stores, LPT apart
  constexpr float kInf = __builtin_inff();
  const Key kNone = -(Key)kInf;
  const int lane = threadIdx.x & 63;
  const int p = lane % LPT;  // lane within the token
  const int slot = lane / LPT;
  const int lane0 = lane & ~(LPT - 1);
  auto vote = [&](bool b) {
    return (uint64_t)(__ballot(b) >> lane0) & (LPT == 64 ? ~0ull : (1ull << (LPT & 63)) - 1);
  };
  for (int j = p; j < a.topk; j += LPT) lds.chosen[slot][j] = -1;
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
      if (p % width == 0 && p / width < a.groups) lds.worth[slot][p / width] = value(b);
    } else {
      Worth* mine = lds.keys[slot];
#pragma unroll
      for (int i = 0; i < VPL; ++i) mine[p * VPL + i] = val[i];
      sync();
      for (int g = p; g < a.groups; g += LPT) {
        Two<Worth> b{kNothing, kNothing};
#pragma unroll 8
        for (int i = 0; i < per; ++i) b.add(mine[g * per + i]);
        lds.worth[slot][g] = value(b);
      }
    }
    sync();
    uint64_t keep = 0;  // groups that stay, one bit each: fewer than topk_groups are better
#pragma unroll
    for (int r = 0; r < kOut; ++r) {
      const int g = r * LPT + p;
      const Worth mine = lds.worth[slot][g < a.groups ? g : 0];
      int better = 0;
      for (int o = 0; o < a.groups; ++o) {
        const Worth k = lds.worth[slot][o];
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
  sync();  // the slots of `chosen` are cleared

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
        lds.chosen[slot][j] = p * VPL + at;
      }
    }
  sync();

  // Weights: lane j % LPT of the token has the experts of rounds j = lane, lane + LPT, ...
  int got[kOut];
  float lj[kOut];
  float far = -kInf;
#pragma unroll
  for (int r = 0; r < kOut; ++r) {
    const int j = r * LPT + p;
    got[r] = j < a.topk ? lds.chosen[slot][j] : -1;
    lj[r] = got[r] >= 0 ? logit(got[r]) : -kInf;
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
      put(j, got[r], lost ? __builtin_nanf("") : got[r] >= 0 ? w[r] / sum * a.scale : 0.f);
    }
  }
}

}  // namespace route
}  // namespace awq
