// mx.h -- launchers of the four-bit layers' kernels, and the layout of what is held in four bits.
#pragma once
#include "ops.h"

namespace muon {

// R rows of K values, by slices of 128 values (64 bytes) of every row: values [slice][row][64], e2m1 two a byte, the
// lower bits first; and by chunks of four slices the e8m0 scales, [chunk][row][16]: byte 4 g + s of a row is that
// of the 32 values g (0..3) of the chunk's slice s.  The rows of a tile are so one stretch of a slice, whole lines
// for any tile; 16 rows of a slice are, in order, what the lanes of a wave hand to a matrix
// instruction; and four bytes are a lane's scales for a chunk.  What pads K is zero.
constexpr int kMxBlock = 32, kMxSlice = 128, kMxSliceBytes = 64, kMxChunk = 512, kMxChunkBytes = 16;
inline __host__ __device__ int64_t mx_slices(int64_t k) { return (k + kMxSlice - 1) / kMxSlice; }
inline __host__ __device__ int64_t mx_chunks(int64_t k) { return (k + kMxChunk - 1) / kMxChunk; }
inline int64_t mx_value_bytes(int64_t rows, int64_t k) { return mx_slices(k) * rows * kMxSliceBytes; }
inline int64_t mx_scale_bytes(int64_t rows, int64_t k) { return mx_chunks(k) * rows * kMxChunkBytes; }

struct MxArgs {
  const void* src;       // element (r, j) at r ld + j, or where t at j ld + r; one group's `step` behind another's
  uint8_t* values;       // of each group
  uint8_t* scales;
  void* dst;             // dequantised rows of k, contiguous
  int64_t rows, k, ld, step;
  int32_t groups, t;
};
// Workgroups of the kernels over rows, and whether one launch holds them (2^32 threads).
inline int64_t mx_row_blocks(int64_t rows, int64_t k) { return (rows + 3) / 4 * mx_chunks(k); }
inline bool mx_rows_fit(int64_t rows, int64_t k) { return mx_row_blocks(rows, k) < (int64_t(1) << 24); }
// A weight's: with at least four rows a group, since the kernel across memory takes one group a workgroup.
inline bool mx_weight_fits(int64_t groups, int64_t n, int64_t k) { return mx_rows_fit(groups * (n > 4 ? n : 4), k); }
hipError_t launch_mx_quantize(const MxArgs& a, int dtype, hipStream_t s);
hipError_t launch_mx_dequantize(const MxArgs& a, int dtype, hipStream_t s);

// C = act(A B^T + bias) + res of A [m, k] and B [groups][n, k] in four bits; k and k_per of `g` count slices, k_per
// a multiple of four.
struct MxProduct {
  GemmArgs g;
  const uint8_t* sca;    // scales of A
  const uint8_t* scb;
  const void* x;         // kMxRowsOwn: A itself, taken to four bits on the way
  int64_t ldx, kx;
};
enum MxTile { kMx256x128 = 0, kMx128, kMx64, kMxRows32, kMxRows16, kMxRowsOwn };
inline int mx_tile_m(int tile) {
  constexpr int rows[] = {256, 128, 64, 32, 16, 16};
  return rows[tile];
}
// Columns of a workgroup: fixed for the tiles in LDS; for few rows, as few as it takes to occupy every compute unit.
inline int mx_tile_n(int tile, int64_t blocks_m, int64_t n) {
  if (tile <= kMx64) return tile == kMx64 ? 64 : 128;
  int cols = 64;
  while (cols > 16 && blocks_m * ((n + cols - 1) / cols) < 256) cols /= 2;
  return cols;
}
hipError_t launch_mx_product(const MxProduct& a, int dtype, int tile, int cols, hipStream_t s);

}  // namespace muon
