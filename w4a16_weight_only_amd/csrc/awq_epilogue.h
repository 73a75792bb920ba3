// Epilogue of a product: y = residual + scale * f(v + bias), or f(v + bias) * (u + bias_u), in fp32.
#pragma once

#include "awq_device.h"
#include "awq_kernels.h"

namespace awq {

// f of the epilogue.  The quotients are reciprocals good to one step.  gelu by erfc, and its tanh
// form as v times a logistic function, keep their digits where 1 + erf or 1 + tanh would cancel.
__device__ __forceinline__ float activate(int kind, float v) {
  switch (kind) {
    case kActRelu: return v < 0.f ? 0.f : v;  // (NaN stays)
    case kActSilu: return v * __builtin_amdgcn_rcpf(1.f + __expf(-v));
    case kActGelu: return 0.5f * v * erfcf(-0.70710678f * v);
    case kActGeluTanh: {
      const float u = 0.79788456f * (v + 0.044715f * v * v * v);
      return v * __builtin_amdgcn_rcpf(1.f + __expf(-2.f * u));
    }
    default: return v;
  }
}

// Eight 16-bit values of a row in 16 bytes.
template <bool BF16>
__device__ __forceinline__ void unpack8(const u32x4& w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = act_to_float<BF16>((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
}

// y of eight adjacent columns whose f is formed: joined with the residual (raw), rounded once.
template <bool BF16>
__device__ __forceinline__ void finish8(const Epilogue& e, int64_t at, const float (&f)[8], const u32x4& raw) {
  float r[8];
  if (e.residual != nullptr) {
    unpack8<BF16>(raw, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] += e.scale * f[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = e.scale * f[i];
  }
  *reinterpret_cast<u32x4*>(e.y + at) = u32x4{pack_act2<BF16>(r[0], r[1]), pack_act2<BF16>(r[2], r[3]),
                                              pack_act2<BF16>(r[4], r[5]), pack_act2<BF16>(r[6], r[7])};
}

}  // namespace awq
