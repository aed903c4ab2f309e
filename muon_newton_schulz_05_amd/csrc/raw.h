// raw.h -- pieces of eight elements held as they lie in memory.
#pragma once
#include "act.h"

namespace muon {

// Eight elements as they lie in memory, so that a load can be in flight while other work goes on.
template <typename T> struct Raw {
  u32x4_t r[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, int n) {
    if (n >= 8) {
#pragma unroll
      for (int q = 0; q < (int)sizeof(T) / 2; ++q) r[q] = load16(p + q * (16 / sizeof(T)));
      return;
    }
#pragma unroll
    for (int q = 0; q < (int)sizeof(T) / 2; ++q) r[q] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 4) r[i >> 2][i & 3] = __float_as_uint(p[i]);
        else r[0][i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
      }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(r[i >> 2][i & 3]);
    else return i & 1 ? bf16_hi(r[0][i >> 1]) : bf16_lo(r[0][i >> 1]);
  }
};

}  // namespace muon
