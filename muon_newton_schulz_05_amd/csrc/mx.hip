// mx.hip -- values to four bits and back: e2m1 in blocks of 32 that share an e8m0 scale (the Open Compute Project's
// microscaling formats, version 1.0).
//
// A block's scale is 2^(floor(log2 of its largest magnitude) - 2), at least 2^-127; a value is divided by it, which
// is exact, and rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), to 6 from above. A block
// with an infinity or NaN has scale 255, which is NaN, and values of zero.  The matrix instructions take these scales
// as they are.
#include "act.h"
#include "mx.h"

namespace muon {
namespace {

constexpr int kNanScale = 255;

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
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ int64_t row_bytes(int64_t k) { return (k + kMxBlock - 1) / kMxBlock * (kMxBlock / 2); }
__device__ __forceinline__ int64_t slices(int64_t k) { return (k + kMxSlice - 1) / kMxSlice; }
// Where block b of row r has its scale.
__device__ __forceinline__ int64_t scale_place(int64_t rows, int64_t r, int64_t b) {
  return ((b >> 3) * rows + r) * 8 + 2 * (b & 3) + ((b >> 2) & 1);
}

// A thread's piece: eight values of a row, so that four lanes share a block and a wave's loads and stores are whole
// lines.  (The divisions by a row's pieces are 64 bits wide once a workgroup.)
struct Piece8 {
  int64_t row;
  int piece;
  __device__ __forceinline__ Piece8(int64_t pieces) {
    const int64_t at = (int64_t)blockIdx.x * 256, row0 = at / pieces;
    const uint32_t p = (uint32_t)(at - row0 * pieces) + threadIdx.x, per = (uint32_t)pieces;
    row = row0 + p / per;
    piece = (int)(p % per);
  }
};

template <typename T>
__global__ __launch_bounds__(256) void k_quantize_rows(MxArgs a) {
  const int64_t rb = row_bytes(a.k), pieces = rb / 4;
  const Piece8 p(pieces);
  // The rows of all groups, one behind the other; the last workgroup's lanes past them hold no block.
  if (p.row >= a.rows * a.groups) return;
  const int64_t e = a.groups > 1 ? p.row / a.rows : 0, r = p.row - e * a.rows;
  float v[8];
  const int col = p.piece * 8;
  load8(static_cast<const T*>(a.src) + e * a.step + r * a.ld + col, (int)max((int64_t)0, min((int64_t)8, a.k - col)), v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, magnitude(v[i]));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));  // lanes i and i ^ 1
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));  // and i ^ 2
  const int scale = scale_of(m);
  reinterpret_cast<uint32_t*>(a.values + p.row * rb)[p.piece] = pack8(v, scale);
  if ((p.piece & 3) != 0) return;
  uint8_t* scales = a.scales + e * slices(a.k) * a.rows * 8;
  scales[scale_place(a.rows, r, p.piece >> 2)] = (uint8_t)scale;
  // The last block's lane clears what is left of the slice.
  if (p.piece + 4 == pieces)
    for (int64_t b = pieces / 4; b & 7; ++b) scales[scale_place(a.rows, r, b)] = 0;
}

// Rows that lie across memory (a weight [K, N]): a lane takes 16 bytes of 32 lines, one block of each of its C rows; the
// wave 8 C rows of a slice of 256, so that loads are 128-byte lines and stores 128 bytes of a row.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize_cols(MxArgs a, int tiles) {
  constexpr int C = 16 / sizeof(T);
  const int lane = threadIdx.x & 63, b = lane >> 3;
  const int64_t rb = row_bytes(a.k), ns = slices(a.k);
  const int64_t tile = blockIdx.x % tiles, eq = blockIdx.x / tiles, e = eq / ns, q = eq - e * ns;
  const int64_t r0 = (tile * 4 + (threadIdx.x >> 6)) * 8 * C + (lane & 7) * C, k0 = q * kMxSlice + b * kMxBlock;
  const int n = (int)max((int64_t)0, min((int64_t)C, a.rows - r0));
  if (n == 0) return;
  uint8_t* scales = a.scales + e * ns * a.rows * 8;
  if (k0 >= a.k) {  // what is left of the last slice
    for (int c = 0; c < n; ++c) scales[scale_place(a.rows, r0 + c, k0 / kMxBlock)] = 0;
    return;
  }
  const T* src = static_cast<const T*>(a.src) + e * a.step + k0 * a.ld + r0;
  const int lines = (int)min((int64_t)kMxBlock, a.k - k0);
  u32x4_t raw[kMxBlock];
  if (n == C && lines == kMxBlock) {
#pragma unroll
    for (int j = 0; j < kMxBlock; ++j) raw[j] = load16(src + j * a.ld);
  } else {
#pragma unroll
    for (int j = 0; j < kMxBlock; ++j) {
      raw[j] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (j < lines && c < n) {
          const T v = src[j * a.ld + c];
          if constexpr (sizeof(T) == 4) raw[j][c] = __builtin_bit_cast(uint32_t, v);
          else raw[j][c / 2] |= (uint32_t)v << (16 * (c & 1));
        }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    auto value = [&](int j) {
      if constexpr (sizeof(T) == 4) return __uint_as_float(raw[j][c]);
      else return c & 1 ? bf16_hi(raw[j][c / 2]) : bf16_lo(raw[j][c / 2]);
    };
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kMxBlock; ++j) m = max(m, magnitude(value(j)));
    const int scale = scale_of(m);
    u32x4_t out;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = value(8 * w + i);
      out[w] = pack8(v, scale);
    }
    if (c < n) {
      const int64_t r = r0 + c;
      *reinterpret_cast<u32x4_t*>(a.values + (e * a.rows + r) * rb + k0 / 2) = out;
      scales[scale_place(a.rows, r, k0 / kMxBlock)] = (uint8_t)scale;
    }
  }
}

// Eight values of a row from their four bits.
template <typename T>
__global__ __launch_bounds__(256) void k_dequantize(MxArgs a) {
  const int64_t rb = row_bytes(a.k), pieces = (a.k + 7) / 8;
  const Piece8 p(pieces);
  if (p.row >= a.rows * a.groups) return;
  const int64_t e = a.groups > 1 ? p.row / a.rows : 0, r = p.row - e * a.rows;
  const int scale = a.scales[e * slices(a.k) * a.rows * 8 + scale_place(a.rows, r, p.piece >> 2)];
  const uint32_t q = reinterpret_cast<const uint32_t*>(a.values + p.row * rb)[p.piece];
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2_t two = i == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 0)
                        : i == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 1)
                        : i == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 2)
                                 : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 3);
    v[2 * i] = two[0];
    v[2 * i + 1] = two[1];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = scale == kNanScale ? __builtin_nanf("") : ldexpf(v[i], scale - 127);
  store8(static_cast<T*>(a.dst) + p.row * a.k + p.piece * 8, (int)min((int64_t)8, a.k - p.piece * 8), v);
}

template <typename T>
hipError_t quantize(const MxArgs& a, hipStream_t s) {
  if (a.t) {
    constexpr int64_t kRows = 4 * 8 * 16 / sizeof(T);  // of a workgroup
    const int64_t tiles = (a.rows + kRows - 1) / kRows, blocks = tiles * ((a.k + kMxSlice - 1) / kMxSlice) * a.groups;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_quantize_cols<T>), dim3((unsigned)blocks), dim3(256), 0, s, a, (int)tiles);
  } else {
    const int64_t blocks = (a.rows * a.groups * (mx_row_bytes(a.k) / 4) + 255) / 256;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_quantize_rows<T>), dim3((unsigned)blocks), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const MxArgs& a, int dtype, hipStream_t s) {
  if (a.rows == 0 || a.k == 0 || a.groups == 0) return hipSuccess;
  return dtype == MUON_BF16 ? quantize<uint16_t>(a, s) : quantize<float>(a, s);
}

hipError_t launch_mx_dequantize(const MxArgs& a, int dtype, hipStream_t s) {
  if (a.rows == 0 || a.k == 0 || a.groups == 0) return hipSuccess;
  const int64_t blocks = (a.rows * a.groups * ((a.k + 7) / 8) + 255) / 256;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  if (dtype == MUON_BF16) hipLaunchKernelGGL(k_dequantize<uint16_t>, dim3((unsigned)blocks), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_dequantize<float>, dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
