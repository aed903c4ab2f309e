// act.h -- activations, their derivatives, and the blocks of grouped rows.
#pragma once
#include "device_common.h"
#include "ops.h"

namespace muon {

// act(z) in float32.  Each is z times a factor in [0, 1] that keeps its relative
// accuracy where it falls to zero: the tanh form of gelu uses (1 + tanh u) / 2 =
// sigmoid(2 u).  Exponentials and reciprocals are the hardware's (about one unit in the
// last place, and what the exponent's rounding makes of it: about as much as one rounding
// of z itself does); subnormal values are zero.  NaN stays NaN.
__device__ __forceinline__ float sigmoid_f(float v) { return __builtin_amdgcn_rcpf(1.f + __expf(-v)); }
// sigmoid(v) and, in rest, 1 - sigmoid(v), each to its own relative accuracy: slopes
// multiply the second by as much as z^3, and with it the error of a difference from
// one (33 2^-24 of dy at z = 5 in gelu_tanh, where this is 4 off at most).
__device__ __forceinline__ float sigmoid_f(float v, float& rest) {
  const float t = __expf(-fabsf(v)), d = __builtin_amdgcn_rcpf(1.f + t);
  rest = v < 0.f ? d : t * d;
  return v < 0.f ? t * d : d;
}
constexpr float kGeluC = 0.7978845608028654f, kGeluA = 0.044715f;  // sqrt(2 / pi); the cubic term

// The normal distribution function: Phi(-x) = e^(-x^2 / 2) t P(t) with t = 1 / (1 + 0.37 x),
// P a polynomial of degree 8 fitted here (weighted least squares, the weights moved until the relative
// error levels) to erfcx(x / sqrt 2) / (2 t), which is smooth over all of t = 0 .. 1.  Relative to itself
// the tail is off by at most 2.1e-7 from the fit, about 3e-7 from its float32 steps and 1.5 x^2 2^-24
// from the exponent (one rounding of z itself moves it by x^2 2^-24), down to 1e-37, where it is
// taken as zero.  (A published formula of four terms fewer that bounds the absolute error, by
// 1.5e-7, was 4.7e-4 off at -4 and 2e-2 at -10; [8192, 4096] x [4096, 16384] with gelu took
// 935 us with it and takes 949.)  e = e^(-z^2 / 2), which the slope needs too.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.37f, 1.f));
  e = __builtin_amdgcn_exp2f(z * z * (-0.5f * 1.4426950408889634f));
  float p = fmaf(t, -0.03132685f, 0.13513201f);
  p = fmaf(t, p, -0.19429737f);
  p = fmaf(t, p, 0.06451427f);
  p = fmaf(t, p, 0.0134073235f);
  p = fmaf(t, p, 0.0901829f);
  p = fmaf(t, p, 0.12716383f);
  p = fmaf(t, p, 0.14761533f);
  p = fmaf(t, p, 0.14760861f);
  const float q = t * p * e;
  return z < 0.f ? q : 1.f - q;
}
__device__ __forceinline__ float act_f(float z, int act) {
  switch (act) {
    case MUON_ACT_RELU: return z <= 0.f ? 0.f : z;
    case MUON_ACT_SILU: return z * sigmoid_f(z);
    case MUON_ACT_GELU: {
      float e;
      return z * normal_cdf(z, e);
    }
    case MUON_ACT_GELU_TANH: return z * sigmoid_f(2.f * kGeluC * (z + kGeluA * z * z * z));
    default: return z;
  }
}
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case MUON_ACT_RELU: return z <= 0.f ? 0.f : 1.f;
    case MUON_ACT_SILU: {
      float r;
      const float q = sigmoid_f(z, r);
      return q + z * q * r;
    }
    case MUON_ACT_GELU: {
      float e;
      const float c = normal_cdf(z, e);
      return fmaf(z * 0.3989422804014327f, e, c);
    }
    case MUON_ACT_GELU_TANH: {
      float r;
      const float q = sigmoid_f(2.f * kGeluC * (z + kGeluA * z * z * z), r);
      // z^2 is bounded so that its overflow does not meet r = 0.
      return q + z * q * r * 2.f * kGeluC * (1.f + 3.f * kGeluA * fminf(z * z, 1e30f));
    }
    default: return 1.f;
  }
}

// Orders this wave's LDS accesses: lanes exchange values through LDS that no
// other wave touches (the LDS itself serves a wave's accesses in order).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Row range [lo, hi) of group e; group `groups` is the rows past the last
// one.  The first group starts at row 0, and offsets are clamped into
// [0, rows], so whatever they hold, every row read or written lies inside
// the tensors.
__device__ __forceinline__ void group_range(const int32_t* offsets, int groups, int64_t rows, int e, int& lo, int& hi) {
  const int r = (int)rows;
  lo = e == 0 ? 0 : min(max(offsets[e], 0), r);
  hi = e == groups ? r : max(lo, min(offsets[e + 1], r));
}

// A sum of block counts.  Groups that overlap, by offsets that do not ascend, can
// have more blocks than 32 bits hold: the sum then stays at a bound that no valid
// offsets reach.
__device__ __forceinline__ int add_blocks(int a, int b) { return min(a + b, (1 << 30) - 1); }

// Every group's rows cut into blocks of `block`: each lane counts its share of the
// groups' blocks, and a wave-wide prefix sum places the shares.  Results are
// uniform over the wave.
struct GroupBlocks {
  int e0, e1;         // this lane's groups
  int before, count;  // blocks ahead of them, and theirs
  int total;

  __device__ __forceinline__ GroupBlocks(const int32_t* offsets, int groups, int64_t rows, int block) {
    const int lane = threadIdx.x & 63, per = (groups + 64) / 64;  // groups + 1 ranges over 64 lanes
    e0 = lane * per;
    e1 = min(e0 + per, groups + 1);
    count = 0;
    for (int i = e0; i < e1; ++i) {
      int lo, hi;
      group_range(offsets, groups, rows, i, lo, hi);
      count = add_blocks(count, (hi - lo + block - 1) / block);
    }
    int incl = count;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl = add_blocks(incl, v);
    }
    before = incl - count;
    total = __builtin_amdgcn_readlane(incl, 63);
  }

  // The group e of block b (0 <= b < total), its first row and its group's end; no rows
  // where offsets that do not ascend leave the block without a group.
  __device__ __forceinline__ void find(const int32_t* offsets, int groups, int64_t rows, int block, int b, int& e,
                                       int& row0, int& end) const {
    int left = b - before, fe = 0, f0 = 0, f1 = 0;
    const bool mine = left >= 0 && left < count;
    const uint64_t hit = __ballot(mine);
    if (mine) {
      for (int i = e0; i < e1; ++i) {
        int lo, hi;
        group_range(offsets, groups, rows, i, lo, hi);
        const int c = (hi - lo + block - 1) / block;
        if (left < c) {
          fe = i;
          f0 = lo + left * block;
          f1 = hi;
          break;
        }
        left -= c;
      }
    }
    const int src = hit ? __builtin_ctzll(hit) : 0;
    e = __builtin_amdgcn_readlane(fe, src);
    row0 = __builtin_amdgcn_readlane(f0, src);
    end = __builtin_amdgcn_readlane(f1, src);
  }
};

// Eight consecutive elements as float32, n of them inside the row (the others
// are zero).  Whole groups move as 16-byte accesses at any alignment of
// their elements, which the hardware splits where it has to.
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));  // at any alignment of 16-bit elements
template <typename T, bool NT = false>
__device__ __forceinline__ u32x4_t load16(const T* p) {
  const MUON_GLOBAL u32x4_any_t* q = (const MUON_GLOBAL u32x4_any_t*)as_global(p);
  if constexpr (NT) return __builtin_nontemporal_load(q);
  else return *q;
}
template <bool NT = false, typename T>
__device__ __forceinline__ void store16(T* p, u32x4_t w) {
  MUON_GLOBAL u32x4_any_t* q = (MUON_GLOBAL u32x4_any_t*)as_global(p);
  if constexpr (NT) __builtin_nontemporal_store(w, q);
  else *q = w;
}
template <typename T, bool NT = false>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
  if (n >= 8) {
    if constexpr (sizeof(T) == 2) {
      const u32x4_t w = load16<T, NT>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
      const f32x4_t w[2] = {__builtin_bit_cast(f32x4_t, load16<T, NT>(p)), __builtin_bit_cast(f32x4_t, load16<T, NT>(p + 4))};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = w[i >> 2][i & 3];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? x_to_f32(p[i]) : 0.f;
}
template <typename T, bool NT = false>
__device__ __forceinline__ void store8(T* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    if constexpr (sizeof(T) == 2) {
      store16<NT>(p, u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                             pack_bf16x2(v[6], v[7])});
    } else {
      store16<NT>(p, __builtin_bit_cast(u32x4_t, f32x4_t{v[0], v[1], v[2], v[3]}));
      store16<NT>(p + 4, __builtin_bit_cast(u32x4_t, f32x4_t{v[4], v[5], v[6], v[7]}));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = cvt_x<T>(v[i]);
}

}  // namespace muon
