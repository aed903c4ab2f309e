// mx.h -- launchers of the four-bit layers' kernels, and the layout of what is held in four bits.
#pragma once
#include "ops.h"

namespace muon {

// R rows of K values: e2m1 values two a byte (the lower bits first), rows of K rounded up to 32 values; and one
// e8m0 scale for each 32 of a row.  Scales lie by slices of 256 values, [slice][row][8], so that the rows of a
// tile are one stretch of a slice; byte 2 (b mod 4) + b / 4 of a row's eight is that of the slice's block b,
// which puts the two substeps of one lane group side by side.  What pads a row is zero.
constexpr int kMxBlock = 32, kMxSlice = 256;
inline int64_t mx_row_bytes(int64_t k) { return (k + kMxBlock - 1) / kMxBlock * (kMxBlock / 2); }
inline int64_t mx_scale_bytes(int64_t rows, int64_t k) { return (k + kMxSlice - 1) / kMxSlice * rows * 8; }

struct MxArgs {
  const void* src;       // element (r, j) at r ld + j, or where t at j ld + r; one group's `step` behind another's
  uint8_t* values;       // [groups][rows][row bytes]
  uint8_t* scales;       // [groups][slices][rows][8]
  void* dst;             // dequantised rows of k
  int64_t rows, k, ld, step;
  int32_t groups, t;
};
hipError_t launch_mx_quantize(const MxArgs& a, int dtype, hipStream_t s);
hipError_t launch_mx_dequantize(const MxArgs& a, int dtype, hipStream_t s);
hipError_t launch_gemm_mx(const GemmArgs& g, int dtype, int tile, hipStream_t s);

}  // namespace muon
