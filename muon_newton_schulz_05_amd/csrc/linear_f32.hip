// linear_f32.hip -- the float32 products of the layer operators, the joining
// of split contractions, and the activation's gradient.
#include "gemm.h"

namespace muon {

hipError_t launch_gemm_f32(const GemmArgs& g, bool ta, bool tb, int loads, int tile, hipStream_t s) {
  if (loads == kDirect4) {
    if (tile == kTile32x64) return launch_tile<float, 32, 64, 1, 4, 1, 4, kDirect4>(g, ta, tb, s);
    return launch_tile<float, 64, 64, 2, 2, 1, 2, kDirect4>(g, ta, tb, s);
  }
  if (loads == kStaged) {
    if (tile == kTile32x64) return launch_tile<float, 32, 64, 1, 4, 1, 2, kStaged>(g, ta, tb, s);
    return launch_tile<float, 64, 64, 2, 2, 1, 2, kStaged>(g, ta, tb, s);
  }
  switch (tile) {
    case kTile32x64: return launch_tile<float, 32, 64, 1, 4, 1, 4, kDirect16>(g, ta, tb, s);
    case kTileRows32: return launch_tile<float, 32, 128, 1, 4, 1, 4, kDirect16>(g, ta, tb, s);
    case kTileRows32K: return launch_tile<float, 32, 64, 1, 2, 4, 3, kDirect16>(g, ta, tb, s);
    default: return launch_tile<float, 64, 64, 2, 2, 1, 2, kDirect16>(g, ta, tb, s);
  }
}

int gemm_tile_m(int tile) {
  switch (tile) {
    case kTile256:
    case kTile256x128: return 256;
    case kTile64: return 64;
    case kTile32x64:
    case kTileRows32:
    case kTileRows32K: return 32;
    default: return 128;
  }
}
int gemm_tile_n(int tile) {
  switch (tile) {
    case kTile256: return 256;
    case kTile64:
    case kTile32x64:
    case kTileRows32K: return 64;
    default: return 128;
  }
}

hipError_t launch_gemm(const GemmArgs& g, int dtype, bool ta, bool tb, int loads, int tile, hipStream_t s) {
  return dtype == MUON_BF16 ? launch_gemm_bf16(g, ta, tb, loads, tile, s)
                            : launch_gemm_f32(g, ta, tb, loads, tile, s);
}

hipError_t launch_gemm_join(const GemmArgs& g, int dtype, hipStream_t s) {
  const int64_t blocks = ((g.n + 7) / 8 * g.m * g.groups + 255) / 256;
  if (blocks <= 0) return hipSuccess;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  if (dtype == MUON_BF16) hipLaunchKernelGGL((k_gemm_join<uint16_t>), dim3((unsigned)blocks), dim3(256), 0, s, g);
  else hipLaunchKernelGGL((k_gemm_join<float>), dim3((unsigned)blocks), dim3(256), 0, s, g);
  return hipGetLastError();
}

namespace {

// dz = dy act'(z) for one block of a.block rows of one group and 512
// columns, and that block's column sums, in float32 before any rounding.
// Each lane holds 8 columns and each of the 4 waves every fourth row; the waves'
// sums meet in LDS in wave order.  Bound by memory: it reads dy and z and
// writes dz once ([8192, 16384] bf16 with gelu: 184 - 190 us, 4.2 - 4.4 TB/s; 192 with the column
// sums).
template <typename T, bool FULL>
__global__ __launch_bounds__(256) void k_act_grad(ActGradArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cols = (int)((a.n + 511) / 512);
  const int blk = blockIdx.x / cols, cb = blockIdx.x - blk * cols;
  int e = 0, lo = 0, hi = 0;
  if (a.offsets2 && blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.groups; i += 256) a.offsets2[i] = 2 * min(max(a.offsets[i], 0), (int)a.rows);
  if (a.offsets) {
    const GroupBlocks gb(a.offsets, a.groups, a.rows, a.block);
    if (blk >= gb.total) return;
    gb.find(a.offsets, a.groups, a.rows, a.block, blk, e, lo, hi);
    hi = min(hi, lo + a.block);
  } else {
    lo = blk * a.block;
    hi = (int)min((int64_t)lo + a.block, a.rows);
  }
  const int64_t col = (int64_t)cb * 512 + lane * 8;
  const int n = FULL ? (col < a.n ? 8 : 0) : (int)min((int64_t)8, a.n - col);
  float sum[8] = {};
  // Rows past the last group: their gradient is zero.
  const bool dead = a.offsets && e == a.groups;
  if (n > 0) {
    constexpr int U = 4;  // rows in flight; past the block's end the last row is read again, not used
    for (int r0 = lo + wave; r0 < hi; r0 += 4 * U) {
      float v[U][8], z[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = min(r0 + 4 * u, hi - 1);
        load8(static_cast<const T*>(a.dy) + r * a.lddy + col, FULL ? 8 : n, v[u]);
        if (a.z) load8(static_cast<const T*>(a.z) + r * a.ldz + col, FULL ? 8 : n, z[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + 4 * u;
        if (r >= hi) break;
        if (a.z) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[u][i] *= act_slope(z[u][i], a.act);
        }
        if (dead) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
        }
        if (a.dz) store8(static_cast<T*>(a.dz) + (int64_t)(r << a.pairs) * a.lddz + col, FULL ? 8 : n, v[u]);
        if constexpr (sizeof(T) == 2) {
          if (a.pairs) {
            float lost[8];  // nothing where the value, or its rounding, is not finite
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float d = v[u][i] - from_bf16(to_bf16(v[u][i]));
              lost[i] = fabsf(d) < __builtin_huge_valf() ? d : 0.f;
            }
            store8(static_cast<T*>(a.dz) + (int64_t)(2 * r + 1) * a.lddz + col, FULL ? 8 : n, lost);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[u][i];
      }
    }
  }
  if (!a.db || dead) return;  // uniform over the workgroup
  __shared__ float part[4][512];
#pragma unroll
  for (int i = 0; i < 8; ++i) part[wave][lane * 8 + i] = sum[i];
  __syncthreads();
  for (int c = threadIdx.x; c < 512; c += 256) {
    const int64_t cc = (int64_t)cb * 512 + c;
    if (cc < a.n) a.part[(int64_t)blk * a.n + cc] = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
  }
}

// db: the blocks' sums of each group.  64 columns a workgroup; its four waves
// take every fourth block each, eight loads in flight, and meet in LDS: the
// order of the sum is fixed.
template <typename T>
__global__ __launch_bounds__(256) void k_col_join(ActGradArgs a, int blocks) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const int e = blockIdx.y;
  int b0 = 0, b1 = blocks;
  if (a.offsets) {
    // Blocks of the groups ahead of e, counted by the wave's lanes.
    int before = 0, mine = 0;
    for (int i = lane; i <= e; i += 64) {
      int lo, hi;
      group_range(a.offsets, a.groups, a.rows, i, lo, hi);
      const int k = (hi - lo + a.block - 1) / a.block;
      if (i < e) before = add_blocks(before, k);
      else mine = k;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      before = add_blocks(before, __shfl_xor(before, d, 64));
      mine = add_blocks(mine, __shfl_xor(mine, d, 64));
    }
    b0 = min(before, blocks);
    b1 = min(add_blocks(before, mine), blocks);
  }
  float s = 0.f;
  if (c < a.n) {
    const float* p = a.part + c;
    int b = b0 + wave;
    for (; b + 28 < b1; b += 32) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = p[(int64_t)(b + 4 * u) * a.n];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    for (; b < b1; b += 4) s += p[(int64_t)b * a.n];
  }
  __shared__ float part[4][64];
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < a.n)
    store_from_f32(a.db, (int64_t)e * a.n + c, sizeof(T) == 2,
                   (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]));
}

// One thread moves eight elements of a row.  Bound by memory: 4001 x 4003 in 13 us (5 TB/s).
__global__ __launch_bounds__(256) void k_align(AlignArgs a) {
  const int64_t per = a.ld / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= per * a.rows * a.groups) return;
  const int64_t row = i / per, e = row / a.rows, col = (i - row * per) * 8;
  float v[8];  // bf16 to float and back is exact
  load8(static_cast<const uint16_t*>(a.src) + e * a.src_step + (row - e * a.rows) * a.src_ld + col,
        (int)min((int64_t)8, a.cols - col), v);
  if (a.pairs && (row & 1)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fabsf(v[i]) < __builtin_huge_valf() ? v[i] : 0.f;
  }
  store8(static_cast<uint16_t*>(a.dst) + row * a.ld + col, 8, v);
}

}  // namespace

hipError_t launch_align(const AlignArgs& a, hipStream_t s) {
  const int64_t blocks = (a.ld / 8 * a.rows * a.groups + 255) / 256;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL(k_align, dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

// 64 rows a block; 16 where that would leave most of the card without one.
int act_grad_block(int64_t rows, int64_t n) { return (rows + 63) / 64 * ((n + 511) / 512) < 1024 ? 16 : 64; }
int64_t act_grad_blocks(int64_t rows, int64_t n, int32_t groups, bool grouped) {
  return group_blocks(rows, groups, grouped, act_grad_block(rows, n));
}

hipError_t launch_act_grad(const ActGradArgs& args, int dtype, hipStream_t s) {
  ActGradArgs a = args;
  a.block = act_grad_block(a.rows, a.n);
  const int64_t blocks = act_grad_blocks(a.rows, a.n, a.groups, a.offsets != nullptr);
  const int64_t cols = (a.n + 511) / 512;
  if (cols <= 0) return hipSuccess;
  if (blocks * cols > 0x7fffffff || a.groups > 65535) return hipErrorInvalidValue;
  if (blocks > 0) {
    const dim3 grid((unsigned)(cols * blocks));
    const bool full = a.n % 8 == 0;
    if (dtype == MUON_BF16 && full) hipLaunchKernelGGL((k_act_grad<uint16_t, true>), grid, dim3(256), 0, s, a);
    else if (dtype == MUON_BF16) hipLaunchKernelGGL((k_act_grad<uint16_t, false>), grid, dim3(256), 0, s, a);
    else if (full) hipLaunchKernelGGL((k_act_grad<float, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_act_grad<float, false>), grid, dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.db) return hipSuccess;
  const dim3 grid((unsigned)((a.n + 63) / 64), (unsigned)a.groups);
  if (dtype == MUON_BF16) hipLaunchKernelGGL((k_col_join<uint16_t>), grid, dim3(256), 0, s, a, (int)blocks);
  else hipLaunchKernelGGL((k_col_join<float>), grid, dim3(256), 0, s, a, (int)blocks);
  return hipGetLastError();
}

}  // namespace muon
