// Routing of tokens to experts (awq_moe_route): the kernel over rows of logits.  What it computes,
// and how, is in awq_route.h.
#include "awq_route.h"

namespace awq {

using namespace route;

namespace {

constexpr int kRouteThreads = 64;
constexpr int64_t kRouteFewTokens = 2048;

template <int TYPE>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (TYPE == 2) return static_cast<const float*>(p)[i];
  else return act_to_float<TYPE == 1>(static_cast<const uint16_t*>(p)[i]);
}

}  // namespace

// TYPE of the logits: 0 fp16, 1 bfloat16, 2 fp32.
template <typename Key, typename Worth, int LPT, int VPL, bool GROUPS, int TYPE>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const RouteArgs a) {
  constexpr int TOKENS = kRouteThreads / LPT;  // tokens per workgroup (one wave)
  constexpr float kInf = __builtin_inff();
  __shared__ Scratch<Worth, LPT, VPL, GROUPS> lds;
  const int lane = threadIdx.x;
  const int p = lane % LPT;  // lane within the token
  const int slot = lane / LPT;
  const int64_t t_raw = (int64_t)blockIdx.x * TOKENS + slot;
  const bool live = t_raw < a.T;
  const int64_t t = live ? t_raw : a.T - 1;  // lanes past the last token redo it and store nothing
  const int64_t row = t * a.row_stride;

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
  route_tokens<Key, Worth, LPT, VPL, GROUPS>(
      a, l, [&](int e) { return load_logit<TYPE>(a.logits, row + e); }, [] { __syncthreads(); }, lds, live,
      [&](int j, int id, float weight) {
        a.ids[t * a.topk + j] = id;
        a.weights[t * a.topk + j] = weight;
      });
}

hipError_t launch_route(RouteArgs a, hipStream_t stream) {
  // Keys and worths need fp64 where scores are added to something (awq_route.h).
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
