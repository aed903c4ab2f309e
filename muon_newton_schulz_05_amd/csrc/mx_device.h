// mx_device.h -- values to e2m1 in blocks of 32 with an e8m0 scale, on the device.
#pragma once
#include "act.h"
#include "mx.h"

namespace muon {

constexpr int kNanScale = 255;

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// The scale of a block whose magnitudes' largest bits are m.
__device__ __forceinline__ int scale_of(uint32_t m) {
  return m >= 0x7f800000u ? kNanScale : max((int)(m >> 23) - 2, 0);
}
// Eight values as e2m1 in that scale, the first in the lowest bits.
__device__ __forceinline__ uint32_t pack8(const float (&v)[8], int scale) {
  const int up = 127 - scale;
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, ldexpf(v[0], up), ldexpf(v[1], up), 1.f, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, ldexpf(v[2], up), ldexpf(v[3], up), 1.f, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, ldexpf(v[4], up), ldexpf(v[5], up), 1.f, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, ldexpf(v[6], up), ldexpf(v[7], up), 1.f, 3);
  return scale == kNanScale ? 0u : q;
}

}  // namespace muon
