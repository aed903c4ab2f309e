// mx.hip -- values to four bits and back: e2m1 in blocks of 32 that share an e8m0 scale (the Open Compute Project's
// microscaling formats, version 1.0).
//
// A block's scale is 2^(floor(log2 of its largest magnitude) - 2), at least 2^-127; a value is divided by it, which
// is exact, and rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), to 6 from above. A block
// with an infinity or NaN has scale 255, which is NaN, and values of zero.  The matrix instructions take these scales
// as they are.
//
// Bound by memory.  bf16, operands that come from HBM: a weight [4096, 16384] held [K, N] takes 38 us (4.4 TB/s over what is read
// and written), held [N, K] 39, back 46 (3.7), rows of [49152, 2048] 54 (4.8), of [8192, 4096] 23 (3.7).  Operands that the
// memory-side cache still holds: 29, 33, 27, 46 and 19.
#include "mx_device.h"

namespace muon {
namespace {

// Where the block of values 32 b .. of row r has its scale.
__device__ __forceinline__ int64_t scale_place(int64_t rows, int64_t r, int64_t b) {
  return ((b >> 4) * rows + r) * kMxChunkBytes + 4 * (b & 3) + ((b >> 2) & 3);
}
// Where eight values of row r lie.
__device__ __forceinline__ int64_t value_place(int64_t rows, int64_t r, int64_t piece) {
  return ((piece >> 4) * rows + r) * kMxSliceBytes + 4 * (piece & 15);
}

// A workgroup takes U sets of four rows by a chunk of 512 values, a wave one of its slices and a lane eight values of one
// row of each set: loads are 256 bytes of a row, stores 256 bytes of a slice, and four lanes share a block.
struct Piece8 {
  int64_t row, chunk;  // row of the first set; the next one's is four further
  int piece;           // of the chunk
  __device__ __forceinline__ Piece8(int64_t chunks, int sets) {
    const int64_t b = blockIdx.x, r = b / chunks;
    chunk = b - r * chunks;
    row = r * 4 * sets + ((threadIdx.x >> 4) & 3);
    piece = (threadIdx.x >> 6) * 16 + (threadIdx.x & 15);
  }
};

template <typename T, int U>
__global__ __launch_bounds__(256) void k_quantize_rows(MxArgs a) {
  const int64_t chunks = mx_chunks(a.k), slices = mx_slices(a.k), all = a.rows * a.groups;
  const Piece8 p(chunks, U);
  const int64_t at = p.chunk * 64 + p.piece, col = at * 8;
  const int n = (int)max((int64_t)0, min((int64_t)8, a.k - col));
  int64_t e[U], r[U];
  float v[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // The rows of all groups, one behind the other.
    const int64_t row = p.row + 4 * u;
    e[u] = a.groups > 1 ? row / a.rows : 0;
    r[u] = row - e[u] * a.rows;
    load8(static_cast<const T*>(a.src) + e[u] * a.step + r[u] * a.ld + col, row < all ? n : 0, v[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (p.row + 4 * u >= all) return;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, magnitude(v[u][i]));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));  // lanes i and i ^ 1
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));  // and i ^ 2
    const int scale = scale_of(m);
    if ((at >> 4) < slices)
      *reinterpret_cast<uint32_t*>(a.values + e[u] * slices * a.rows * kMxSliceBytes + value_place(a.rows, r[u], at)) =
          pack8(v[u], scale);
    if ((p.piece & 3) == 0)
      a.scales[e[u] * chunks * a.rows * kMxChunkBytes + scale_place(a.rows, r[u], at >> 2)] = (uint8_t)scale;
  }
}

// Rows that lie across memory (a weight [K, N]): a lane takes 16 bytes of 32 lines, one block of each of its C rows; the
// wave 16 C rows of a slice, and the workgroup's four waves the chunk's four slices.  Loads are 256 bytes of a line.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize_cols(MxArgs a, int tiles) {
  constexpr int C = 16 / sizeof(T);
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int64_t chunks = mx_chunks(a.k), slices = mx_slices(a.k);
  const int64_t tile = blockIdx.x % tiles, ec = blockIdx.x / tiles, e = ec / chunks, q = ec - e * chunks;
  const int64_t r0 = tile * 16 * C + (lane & 15) * C, b = q * 16 + (threadIdx.x >> 6) * 4 + g, k0 = b * kMxBlock;
  const int n = (int)max((int64_t)0, min((int64_t)C, a.rows - r0));
  const int lines = (int)max((int64_t)0, min((int64_t)kMxBlock, a.k - k0));
  if (n == 0) return;
  const T* src = static_cast<const T*>(a.src) + e * a.step + k0 * a.ld + r0;
  uint8_t* values = a.values + e * slices * a.rows * kMxSliceBytes;
  uint8_t* scales = a.scales + e * chunks * a.rows * kMxChunkBytes;
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
      if ((b >> 2) < slices) *reinterpret_cast<u32x4_t*>(values + value_place(a.rows, r0 + c, b * 4)) = out;
      scales[scale_place(a.rows, r0 + c, b)] = (uint8_t)scale;
    }
  }
}

// Eight values of a row from their four bits.
template <typename T>
__global__ __launch_bounds__(256) void k_dequantize(MxArgs a) {
  const int64_t chunks = mx_chunks(a.k);
  const Piece8 p(chunks, 1);
  const int64_t at = p.chunk * 64 + p.piece, col = at * 8;
  if (p.row >= a.rows * a.groups || col >= a.k) return;
  const int64_t e = a.groups > 1 ? p.row / a.rows : 0, r = p.row - e * a.rows;
  const int scale = a.scales[e * chunks * a.rows * kMxChunkBytes + scale_place(a.rows, r, at >> 2)];
  const uint32_t q = *reinterpret_cast<const uint32_t*>(a.values + e * mx_slices(a.k) * a.rows * kMxSliceBytes +
                                                        value_place(a.rows, r, at));
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
  store8(static_cast<T*>(a.dst) + p.row * a.k + col, (int)min((int64_t)8, a.k - col), v);
}

template <typename T>
hipError_t quantize(const MxArgs& a, hipStream_t s) {
  if (a.t) {
    constexpr int64_t kRows = 16 * 16 / sizeof(T);  // of a workgroup
    const int64_t tiles = (a.rows + kRows - 1) / kRows, blocks = tiles * mx_chunks(a.k) * a.groups;
    hipLaunchKernelGGL((k_quantize_cols<T>), dim3((unsigned)blocks), dim3(256), 0, s, a, (int)tiles);
  } else {
    const unsigned blocks = (unsigned)mx_row_blocks(a.rows * a.groups, a.k);
    // Four sets a workgroup where there are plenty.
    if (blocks < 8192) hipLaunchKernelGGL((k_quantize_rows<T, 1>), dim3(blocks), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_quantize_rows<T, 4>), dim3((unsigned)((a.rows * a.groups + 15) / 16 * mx_chunks(a.k))), dim3(256), 0, s, a);
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
  const unsigned blocks = (unsigned)mx_row_blocks(a.rows * a.groups, a.k);
  if (dtype == MUON_BF16) hipLaunchKernelGGL(k_dequantize<uint16_t>, dim3(blocks), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_dequantize<float>, dim3(blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
