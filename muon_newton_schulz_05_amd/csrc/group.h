// group.h -- reductions over aligned groups of L lanes, L a power of two up to 64.  Every lane of a group gets the
// same result, added in the same order.
#pragma once
#include "device_common.h"

namespace muon {

// The value of the lane that step S of a butterfly pairs with this one, where the 2^S lanes before agree: quad
// permutations, mirrored half rows and rows, and gfx950's swaps of rows and of halves.
template <int S>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  if constexpr (S < 4) {
    constexpr int ctrl = S == 0 ? 0xB1 : S == 1 ? 0x4E : S == 2 ? 0x141 : 0x140;
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, true);
  } else {
    // Of the two swapped registers one holds the group's own half in every lane, the other the other half.
    const bool upper = (threadIdx.x >> S) & 1;
    if constexpr (S == 4) {
      const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
      return upper ? r[0] : r[1];
    } else {
      const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
      return upper ? r[0] : r[1];
    }
  }
}
template <int S>
__device__ __forceinline__ float partner(float v) {
  return __uint_as_float(partner<S>(__float_as_uint(v)));
}

template <int L, int S = 0>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr ((1 << S) < L) return group_sum<L, S + 1>(v + partner<S>(v));
  else return v;
}
// The largest value, NaN left out.
template <int L, int S = 0>
__device__ __forceinline__ float group_max(float v) {
  if constexpr ((1 << S) < L) return group_max<L, S + 1>(fmaxf(v, partner<S>(v)));
  else return v;
}

template <int L, int S = 0>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr ((1 << S) < L) return group_max<L, S + 1>(max(v, partner<S>(v)));
  else return v;
}
template <int L, int S = 0>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  if constexpr ((1 << S) < L) return group_min<L, S + 1>(min(v, partner<S>(v)));
  else return v;
}

}  // namespace muon
