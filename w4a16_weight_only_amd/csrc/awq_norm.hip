// Norms on the residual stream, before and after a block:
//   z = x, or norm(x) * post_weight + post_bias
//   r = residual + scale * gate * z          (written in the stream's type)
//   y = norm(r) * weight + bias              (of r before its rounding)
//   norm(v) = v / sqrt(mean(v^2) + eps), or with the mean taken off v first
//
// A row stays in registers from its one read to its one write, so that the sums of a second
// norm, or of squares about the mean, cost no memory.  A row is one wave's, or 4 to 16 waves'
// that meet in LDS, once per sum.  All of a row's loads go out before the first sum waits.
// Everything is fp32 from the loads on; y and r are rounded once.
//
// Bound by HBM for many rows: 8192 x 4096 with a gate, on a stream in fp32 (402 MB), 76.8 us, 5.2 TB/s, where a
// large copy reaches 5.0.  By latency for few: one row of 4096 2.8 us, an empty launch 1.7.
#include <type_traits>

#include "awq_device.h"
#include "awq_kernels.h"
#include "awq_lanes.h"

namespace awq {

namespace {

// Eight elements of a row per lane and piece: 16 adjacent bytes (WIDE), or one element of every
// TPR, so that neighbouring lanes read neighbouring elements.
template <bool WIDE, int TPR>
struct Place {
  int at, H;  // WIDE: first element; else element 0 of 8, TPR apart
  __device__ Place(int piece, int lane, int H_) : at(WIDE ? 8 * (piece * TPR + lane) : 8 * piece * TPR + lane), H(H_) {}
  __device__ int element(int i) const { return WIDE ? at + i : at + i * TPR; }
  __device__ bool in(int i) const { return WIDE ? at < H : element(i) < H; }
  // Places outside the row read its first element and are masked by the caller.
  __device__ u32x4 load16(const uint16_t* row) const {
    if constexpr (WIDE) {
      return *reinterpret_cast<const u32x4*>(row + (at < H ? at : 0));
    } else {
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = (uint32_t)row[in(2 * i) ? element(2 * i) : 0] | (uint32_t)row[in(2 * i + 1) ? element(2 * i + 1) : 0] << 16;
      return v;
    }
  }
  __device__ void load32(const float* row, float (&v)[8]) const {
    if constexpr (WIDE) {
      const float* p = row + (at < H ? at : 0);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const floatx4 f = reinterpret_cast<const floatx4*>(p)[h];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = f[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = row[in(i) ? element(i) : 0];
    }
  }
  template <bool BF16>
  __device__ void store16(uint16_t* row, const float (&v)[8]) const {
    if constexpr (WIDE) {
      if (at < H)
        *reinterpret_cast<u32x4*>(row + at) = u32x4{pack_act2<BF16>(v[0], v[1]), pack_act2<BF16>(v[2], v[3]),
                                                    pack_act2<BF16>(v[4], v[5]), pack_act2<BF16>(v[6], v[7])};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in(i)) row[element(i)] = float_to_act<BF16>(v[i]);
    }
  }
  __device__ void store32(float* row, const float (&v)[8]) const {
    if constexpr (WIDE) {
      if (at < H) {
        reinterpret_cast<floatx4*>(row + at)[0] = floatx4{v[0], v[1], v[2], v[3]};
        reinterpret_cast<floatx4*>(row + at)[1] = floatx4{v[4], v[5], v[6], v[7]};
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in(i)) row[element(i)] = v[i];
    }
  }
};

template <bool BF16>
__device__ __forceinline__ float half_of(const u32x4& w, int i) {
  return act_to_float<BF16>((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
}

}  // namespace

// WAVES of a row (1: four rows per workgroup), PIECES of 8 elements per lane.  R32: the stream
// is fp32.  first: the launch's first row.
template <bool BF16, bool R32, int WAVES, int PIECES, bool WIDE>
__global__ __launch_bounds__(norm_threads(WAVES)) void norm_kernel(const NormArgs a, int64_t first) {
  constexpr int TPR = 64 * WAVES;
  constexpr int ROWS = norm_rows(WAVES);
  __shared__ float red[4][WAVES];
  const int lane = threadIdx.x % TPR;
  const int64_t t = first + (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  if (t >= a.T) return;  // whole waves, and with several waves a row there is one row
  const int H = a.H;
  auto sum_row = [&](float v, int which) {
    v = lanes_sum<64>(v);
    if constexpr (WAVES > 1) {
      if ((lane & 63) == 0) red[which][lane >> 6] = v;
      __syncthreads();
      v = red[which][0];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v += red[which][w];
    }
    return v;
  };

  const bool has_res = a.residual != nullptr, has_gate = a.gate != nullptr, has_post = a.post_weight != nullptr;
  const bool has_pb = a.post_bias != nullptr, has_bias = a.bias != nullptr;
  u32x4 xw[PIECES], gw[PIECES], pw[PIECES], pb[PIECES], ww[PIECES], bw[PIECES];
  float r[PIECES][8];
  const uint16_t* x = a.x + t * a.x_stride;
  const uint16_t* gate = has_gate ? a.gate + t / a.gate_rows * H : nullptr;
#pragma unroll
  for (int p = 0; p < PIECES; ++p) {
    const Place<WIDE, TPR> at(p, lane, H);
    xw[p] = at.load16(x);
    if (has_res) {
      if constexpr (R32) {
        at.load32(static_cast<const float*>(a.residual) + t * a.residual_stride, r[p]);
      } else {
        const u32x4 w = at.load16(static_cast<const uint16_t*>(a.residual) + t * a.residual_stride);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[p][i] = half_of<BF16>(w, i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[p][i] = 0.f;
    }
    if (has_post) pw[p] = at.load16(a.post_weight);
    if (has_pb) pb[p] = at.load16(a.post_bias);
    if (has_gate) gw[p] = at.load16(gate);
    if (a.y != nullptr) ww[p] = at.load16(a.weight);
    if (has_bias) bw[p] = at.load16(a.bias);
  }
  __builtin_amdgcn_sched_barrier(0);

  const float each = 1.f / (float)H, off = a.unit_offset ? 1.f : 0.f;
  // (mean, 1 / spread) of the row's values.
  auto statistics = [&](const float (&v)[PIECES][8], int which, float& mean, float& inv) {
    mean = 0.f;
    if (a.layer) {
      float s = 0.f;
#pragma unroll
      for (int p = 0; p < PIECES; ++p) {
        const Place<WIDE, TPR> at(p, lane, H);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += at.in(i) ? v[p][i] : 0.f;
      }
      mean = sum_row(s, which) * each;
    }
    float s = 0.f;
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const Place<WIDE, TPR> at(p, lane, H);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = v[p][i] - mean;
        s += at.in(i) ? d * d : 0.f;
      }
    }
    inv = 1.f / sqrtf(sum_row(s, which + 1) * each + a.eps);
  };

  float z[PIECES][8];
#pragma unroll
  for (int p = 0; p < PIECES; ++p)
#pragma unroll
    for (int i = 0; i < 8; ++i) z[p][i] = half_of<BF16>(xw[p], i);
  if (has_post) {
    float mean, inv;
    statistics(z, 0, mean, inv);
#pragma unroll
    for (int p = 0; p < PIECES; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        z[p][i] = (z[p][i] - mean) * inv * (off + half_of<BF16>(pw[p], i)) + (has_pb ? half_of<BF16>(pb[p], i) : 0.f);
  }
#pragma unroll
  for (int p = 0; p < PIECES; ++p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[p][i] += a.scale * (has_gate ? z[p][i] * half_of<BF16>(gw[p], i) : z[p][i]);
    if (a.r != nullptr) {
      const Place<WIDE, TPR> at(p, lane, H);
      if constexpr (R32) at.store32(static_cast<float*>(a.r) + t * H, r[p]);
      else at.template store16<BF16>(static_cast<uint16_t*>(a.r) + t * H, r[p]);
    }
  }
  if (a.y == nullptr) return;
  float mean, inv;
  statistics(r, 2, mean, inv);
#pragma unroll
  for (int p = 0; p < PIECES; ++p) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      y[i] = (r[p][i] - mean) * inv * (off + half_of<BF16>(ww[p], i)) + (has_bias ? half_of<BF16>(bw[p], i) : 0.f);
    Place<WIDE, TPR>(p, lane, H).template store16<BF16>(a.y + t * H, y);
  }
}

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  // Wide pieces: every row of every tensor starts on 16 bytes and ends on a whole piece.
  auto wide16 = [&](const void* p, int64_t stride_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.T == 1 || stride_bytes % 16 == 0);
  };
  const int64_t row = 2 * (int64_t)a.H, stream_size = a.r32 ? 4 : 2;
  const bool wide = a.H % 8 == 0 && wide16(a.x, 2 * a.x_stride) && wide16(a.residual, stream_size * a.residual_stride) &&
                    wide16(a.gate, row) && wide16(a.post_weight, row) && wide16(a.post_bias, row) &&
                    wide16(a.weight, row) && wide16(a.bias, row) && wide16(a.y, row) &&
                    wide16(a.r, stream_size * a.H);
  auto go = [&](auto bf16, auto r32, auto waves, auto pieces, auto w) {
    constexpr int W = decltype(waves)::value;
    constexpr int64_t most = norm_launch_rows(W);
    for (int64_t first = 0; first < a.T; first += most) {
      const int64_t rows = a.T - first < most ? a.T - first : most;
      hipLaunchKernelGGL((norm_kernel<decltype(bf16)::value, decltype(r32)::value, W, decltype(pieces)::value,
                                      decltype(w)::value>),
                         dim3((unsigned)((rows + norm_rows(W) - 1) / norm_rows(W))), dim3(norm_threads(W)), 0, stream,
                         a, first);
    }
  };
  auto sized = [&](auto bf16, auto r32, auto w) {
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I4 = std::integral_constant<int, 4>;
    using I8 = std::integral_constant<int, 8>;
    using I16 = std::integral_constant<int, 16>;
    switch (norm_waves(a.H)) {
      case 1: return a.H <= 512 ? go(bf16, r32, I1{}, I1{}, w) : go(bf16, r32, I1{}, I2{}, w);
      case 4:
        if (a.H <= 2048) return go(bf16, r32, I4{}, I1{}, w);
        return a.H <= 4096 ? go(bf16, r32, I4{}, I2{}, w) : go(bf16, r32, I4{}, I4{}, w);
      case 8: return go(bf16, r32, I8{}, I4{}, w);
      default: return go(bf16, r32, I16{}, I4{}, w);
    }
  };
  auto typed = [&](auto bf16, auto r32) { wide ? sized(bf16, r32, std::true_type{}) : sized(bf16, r32, std::false_type{}); };
  using yes = std::true_type;
  using no = std::false_type;
  if (a.bf16) a.r32 ? typed(yes{}, yes{}) : typed(yes{}, no{});
  else a.r32 ? typed(no{}, yes{}) : typed(no{}, no{});
  return hipGetLastError();
}

}  // namespace awq
