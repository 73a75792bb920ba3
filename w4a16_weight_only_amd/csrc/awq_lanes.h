// Reductions over the lanes of a wave that never leave the registers (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace awq {

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }

template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL, typename V>
__device__ __forceinline__ V rotated(V v) {
  if constexpr (sizeof(V) == 4) {
    return __builtin_bit_cast(V, dpp<CTRL>(__builtin_bit_cast(int, v)));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)dpp<CTRL>((int)(uint32_t)u), hi = (uint32_t)dpp<CTRL>((int)(uint32_t)(u >> 32));
    return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
  }
}
// The other operand of a fold across rows of 16 lanes: ROWS 1 pairs rows (0, 1) and (2, 3),
// ROWS 2 rows (0, 2) and (1, 3).  The swap of a register with a copy of itself leaves, in the
// two results, each lane's own value and its partner's.
template <int ROWS>
__device__ __forceinline__ int across(int v, int& own) {
  const auto r = ROWS == 1 ? __builtin_amdgcn_permlane16_swap((unsigned)v, (unsigned)v, false, false)
                           : __builtin_amdgcn_permlane32_swap((unsigned)v, (unsigned)v, false, false);
  own = (int)r[0];
  return (int)r[1];
}
template <int ROWS, typename V, typename F>
__device__ __forceinline__ V fold_rows(V v, F f) {
  int own, other;
  if constexpr (sizeof(V) == 4) {
    other = across<ROWS>(__builtin_bit_cast(int, v), own);
    return f(__builtin_bit_cast(V, own), __builtin_bit_cast(V, other));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    int own_hi, other_hi;
    other = across<ROWS>((int)(uint32_t)u, own);
    other_hi = across<ROWS>((int)(uint32_t)(u >> 32), own_hi);
    return f(__builtin_bit_cast(V, (uint64_t)(uint32_t)own_hi << 32 | (uint32_t)own),
             __builtin_bit_cast(V, (uint64_t)(uint32_t)other_hi << 32 | (uint32_t)other));
  }
}
// f (commutative) over the token's lanes, in every one of them: rotations by 8, 4, 2, 1 within
// 16 lanes, then across the rows.
template <int LPT, typename V, typename F>
__device__ __forceinline__ V lanes_fold(V v, F f) {
  v = f(v, rotated<0x128>(v));
  v = f(v, rotated<0x124>(v));
  v = f(v, rotated<0x122>(v));
  v = f(v, rotated<0x121>(v));
  if constexpr (LPT == 64) {
    v = fold_rows<1>(v, f);
    v = fold_rows<2>(v, f);
  }
  return v;
}
template <int LPT, typename V>
__device__ __forceinline__ V lanes_max(V v) {
  return lanes_fold<LPT>(v, [](V a, V b) { return larger(a, b); });
}
template <int LPT, typename V>
__device__ __forceinline__ V lanes_sum(V v) {
  return lanes_fold<LPT>(v, [](V a, V b) { return a + b; });
}

}  // namespace awq
