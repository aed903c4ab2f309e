// norm.hip -- layer norm and root-mean-square norm of rows, with the residual added ahead of them, and their
// gradients.
//
//   s = x + r,  y = xhat w + b,  xhat = (s - mean) rstd,  rstd = 1 / sqrt(var + eps)
//   g = dy w,   dx = rstd (g - mean(g) - xhat mean(g xhat)) + ds,  dw = sum dy xhat,  db = sum dy
//
// (The root-mean-square norm takes mean = 0 and has no mean(g).)  A row stays in the registers of TPR threads, CH
// pieces of eight columns each, so that it is read once; the variance is taken of the
// differences from the mean, in a second reduction, and loses nothing to a large mean.  y comes from the
// float32 sum s, and the gradient adds x and r again: from s as it is stored, in bf16, dw would be 1.4 times as
// far off as its own rounding makes it (that reads one tensor less: about 110 us for 134 - 139 at 16384 x 4096).
//
// The gradient of w and b is a sum over rows: each thread adds up its columns over the rows that its
// workgroup walks, workgroups leave one row of partial sums each, and a second
// kernel adds those in order.
//
// Bound by memory.  16384 x 4096 bf16 with a residual: forward 93 - 105 us (5.1 - 5.8 TB/s over its four tensors),
// gradient 134 - 139 and 5 for the join (4.9 TB/s over five); a row of 4096 alone 3.6 us.  The gradient
// without the next row's loads in flight took 172 us.
#include "act.h"
#include "group.h"
#include "norm.h"
#include "raw.h"

#include <algorithm>
#include <type_traits>

namespace muon {
namespace {

constexpr int kThreads(int tpr) { return tpr > 256 ? tpr : 256; }

// Sums of N values over the TPR threads of a row; `red` is this row's and this call's own LDS of 16 N floats, or unused.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = group_sum<(TPR < 64 ? TPR : 64)>(v[i]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = (threadIdx.x % TPR) >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * 16 + wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = red[i * 16];
#pragma unroll
      for (int w = 1; w < W; ++w) v[i] += red[i * 16 + w];
    }
  }
}

template <typename T, int TPR, int CH>
__global__ __launch_bounds__(kThreads(TPR)) void k_norm(NormArgs a) {
  constexpr int NT = kThreads(TPR), RPB = NT / TPR;
  __shared__ float red[2][RPB][2][16];  // by the parity of the row, so that one barrier a reduction is enough
  const int l = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float per = 1.f / (float)a.cols;
  int n[CH];
  float w[CH][8], b[CH][8] = {};
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * TPR + l) * 8;
    n[c] = (int)max((int64_t)0, min((int64_t)8, a.cols - col));
#pragma unroll
    for (int i = 0; i < 8; ++i) w[c][i] = 1.f;
    if (a.w) load8(static_cast<const T*>(a.w) + col, n[c], w[c]);
    if (a.b) load8(static_cast<const T*>(a.b) + col, n[c], b[c]);
  }
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB, turn ^= 1) {
    const int64_t row = r0 + sub;
    const bool in = row < a.rows;
    float v[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * TPR + l) * 8, m = in ? n[c] : 0;
      load8(static_cast<const T*>(a.x) + row * a.ldx + col, m, v[c]);
      if (a.res) {
        float r[8];
        load8(static_cast<const T*>(a.res) + row * a.ldr + col, m, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] += r[i];
        store8(static_cast<T*>(a.s) + row * a.cols + col, m, v[c]);
      }
    }
    float mean = 0.f;
    if (a.layer) {
      float t[1] = {0.f};
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) t[0] += v[c][i];
      row_sum<TPR>(t, red[turn][sub][0]);
      mean = t[0] * per;
    }
    float t[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] = i < n[c] ? v[c][i] - mean : 0.f;
        t[0] += v[c][i] * v[c][i];
      }
    row_sum<TPR>(t, red[turn][sub][1]);
    const float rstd = 1.f / sqrtf(t[0] * per + a.eps);
    if (a.stats && in && l == 0) {
      a.stats[2 * row] = mean;
      a.stats[2 * row + 1] = rstd;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = fmaf(v[c][i] * rstd, w[c][i], b[c][i]);
      store8(static_cast<T*>(a.y) + row * a.cols + (c * TPR + l) * 8, in ? n[c] : 0, v[c]);
    }
  }
}

// Eight columns a thread; a workgroup walks its rows with the next one's loads in flight.
// a.part: [workgroups][2][cols], dw's sums and db's.
template <typename T, int TPR>
__global__ __launch_bounds__(kThreads(TPR)) void k_norm_grad(NormGradArgs a) {
  constexpr int NT = kThreads(TPR), RPB = NT / TPR;
  __shared__ float red[2][RPB][2 * 16];
  __shared__ float sums[RPB > 1 ? NT * 8 : 1];
  const int l = threadIdx.x % TPR, sub = threadIdx.x / TPR, col = l * 8;
  const float per = 1.f / (float)a.cols;
  const int n = (int)max((int64_t)0, min((int64_t)8, a.cols - col));
  float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, dw[8] = {}, db[8] = {};
  if (a.w) load8(static_cast<const T*>(a.w) + col, n, w);
  Raw<T> rx, rr, rg, rd;
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    const bool in = row < a.rows;
    const int m = in ? n : 0;
    rx.load(static_cast<const T*>(a.x) + row * a.ldx + col, m);
    if (a.res) rr.load(static_cast<const T*>(a.res) + row * a.ldr + col, m);
    rg.load(static_cast<const T*>(a.dy) + row * a.ldg + col, m);
    if (a.ds) rd.load(static_cast<const T*>(a.ds) + row * a.ldd + col, m);
    mean = in && a.layer ? a.stats[2 * row] : 0.f;
    rstd = in ? a.stats[2 * row + 1] : 0.f;
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int turn = 0;
  fetch((int64_t)blockIdx.x * RPB + sub);
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += step, turn ^= 1) {
    const int64_t row = r0 + sub;
    const bool in = row < a.rows;
    const Raw<T> cx = rx, cr = rr, cg = rg, cd = rd;
    const float mu = mean, rs = rstd;
    fetch(row + step);
    float x[8], g[8], t[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = in && i < n ? ((a.res ? cx.at(i) + cr.at(i) : cx.at(i)) - mu) * rs : 0.f;
      g[i] = cg.at(i);
      dw[i] += g[i] * x[i];
      db[i] += g[i];
      g[i] *= w[i];
      t[0] += g[i];
      t[1] += g[i] * x[i];
    }
    if (!a.dx) continue;  // uniform
    row_sum<TPR>(t, red[turn][sub]);
    const float m1 = a.layer ? t[0] * per : 0.f, m2 = t[1] * per;
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = rs * (g[i] - m1 - x[i] * m2);
    if (a.ds) {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] += cd.at(i);
    }
    store8(static_cast<T*>(a.dx) + row * a.cols + col, in ? n : 0, g);
  }
  if (!a.part) return;
  // The workgroup's rows of threads are added in order.
  auto leave = [&](const float (&v)[8], int which) {
    float* to = a.part + ((int64_t)blockIdx.x * 2 + which) * a.cols;
    if constexpr (RPB == 1) {
      store8(to + col, n, v);
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[sub * TPR * 8 + col + i] = v[i];
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += NT) {
        float t = 0.f;
        for (int q = 0; q < RPB; ++q) t += sums[q * TPR * 8 + c];
        to[c] = t;
      }
    }
  };
  if (a.dw) leave(dw, 0);
  if (a.db) leave(db, 1);
}

// Eight elements of s = x + r.
template <typename T, typename A>
__device__ __forceinline__ void load_sum(const A& a, int64_t row, int64_t col, int n, float (&v)[8]) {
  load8(static_cast<const T*>(a.x) + row * a.ldx + col, n, v);
  if (!a.res) return;
  float r[8];
  load8(static_cast<const T*>(a.res) + row * a.ldr + col, n, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += r[i];
}

// Rows longer than the registers of a workgroup hold: read three times, the gradient's twice and once more for the
// sums over rows (4096 x 16384 bf16: 117 + 86 + 5 us, 1.9 TB/s over what it has to read and write once; with residual and ds 181 +
// 124 + 5, 2.2 TB/s; rows of 8192, which one workgroup holds: 66 + 6 with both, 4.7).
constexpr int kWide = 1024, kWideCols = 16384, kWideGradCols = 8192;
constexpr int64_t kWideGrid = 1 << 20;  // a launch holds fewer than 2^32 threads

template <typename T>
__global__ __launch_bounds__(kWide) void k_norm_wide(NormArgs a) {
  __shared__ float red[2][16];
  const float per = 1.f / (float)a.cols;
  int64_t row = blockIdx.x;
  auto get = [&](int64_t col, float (&v)[8]) {
    const int n = (int)min((int64_t)8, a.cols - col);
    load_sum<T>(a, row, col, n, v);
    return n;
  };
  for (; row < a.rows; row += gridDim.x) {
    float v[8], mean = 0.f;
    if (a.layer) {
      float t[1] = {0.f};
      for (int64_t col = threadIdx.x * 8; col < a.cols; col += kWide * 8) {
        get(col, v);
        float u = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) u += v[i];
        t[0] += u;
      }
      row_sum<kWide>(t, red[0]);
      mean = t[0] * per;
    }
    float t[1] = {0.f};
    for (int64_t col = threadIdx.x * 8; col < a.cols; col += kWide * 8) {
      const int n = get(col, v);
      float u = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) u += i < n ? (v[i] - mean) * (v[i] - mean) : 0.f;
      t[0] += u;
    }
    row_sum<kWide>(t, red[1]);
    const float rstd = 1.f / sqrtf(t[0] * per + a.eps);
    if (a.stats && threadIdx.x == 0) {
      a.stats[2 * row] = mean;
      a.stats[2 * row + 1] = rstd;
    }
    for (int64_t col = threadIdx.x * 8; col < a.cols; col += kWide * 8) {
      const int n = get(col, v);
      if (a.res) store8(static_cast<T*>(a.s) + row * a.cols + col, n, v);
      float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, b[8] = {};
      if (a.w) load8(static_cast<const T*>(a.w) + col, n, w);
      if (a.b) load8(static_cast<const T*>(a.b) + col, n, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf((v[i] - mean) * rstd, w[i], b[i]);
      store8(static_cast<T*>(a.y) + row * a.cols + col, n, v);
    }
    __syncthreads();  // the sums have been read
  }
}

template <typename T>
__global__ __launch_bounds__(kWide) void k_norm_grad_wide(NormGradArgs a) {
  __shared__ float red[2 * 16];
  const float per = 1.f / (float)a.cols;
  int64_t row = blockIdx.x;
  float mean = 0.f, rstd = 0.f, x[8], g[8];
  auto get = [&](int64_t col) {
    const int n = (int)min((int64_t)8, a.cols - col);
    load_sum<T>(a, row, col, n, x);
    load8(static_cast<const T*>(a.dy) + row * a.ldg + col, n, g);
    float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (a.w) load8(static_cast<const T*>(a.w) + col, n, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = i < n ? (x[i] - mean) * rstd : 0.f;
      g[i] *= w[i];
    }
    return n;
  };
  for (; row < a.rows; row += gridDim.x) {
    mean = a.layer ? a.stats[2 * row] : 0.f;
    rstd = a.stats[2 * row + 1];
    float t[2] = {0.f, 0.f};
    for (int64_t col = threadIdx.x * 8; col < a.cols; col += kWide * 8) {
      get(col);
      float u[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[0] += g[i];
        u[1] += g[i] * x[i];
      }
      t[0] += u[0];
      t[1] += u[1];
    }
    row_sum<kWide>(t, red);
    const float m1 = a.layer ? t[0] * per : 0.f, m2 = t[1] * per;
    for (int64_t col = threadIdx.x * 8; col < a.cols; col += kWide * 8) {
      const int n = get(col);
      float d[8] = {};
      if (a.ds) load8(static_cast<const T*>(a.ds) + row * a.ldd + col, n, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] += rstd * (g[i] - m1 - x[i] * m2);
      store8(static_cast<T*>(a.dx) + row * a.cols + col, n, d);
    }
    __syncthreads();  // the sums have been read
  }
}

// The column sums of wide rows: a thread's eight columns over one stretch of rows.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_cols(NormGradArgs a, int64_t stretch) {
  const int64_t col = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (col >= a.cols) return;
  const int n = (int)min((int64_t)8, a.cols - col);
  const int64_t r0 = blockIdx.y * stretch, r1 = min(a.rows, r0 + stretch);
  float dw[8] = {}, db[8] = {};
  for (int64_t row = r0; row < r1; ++row) {
    const float mean = a.layer ? a.stats[2 * row] : 0.f, rstd = a.stats[2 * row + 1];
    float x[8], g[8];
    load_sum<T>(a, row, col, n, x);
    load8(static_cast<const T*>(a.dy) + row * a.ldg + col, n, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] += g[i] * ((x[i] - mean) * rstd);
      db[i] += g[i];
    }
  }
  float* to = a.part + (int64_t)blockIdx.y * 2 * a.cols + col;
  if (a.dw) store8(to, n, dw);
  if (a.db) store8(to + a.cols, n, db);
}

// dw and db (blockIdx.y) from the partial sums: 16 waves take a share of the partials each, for 64 columns.
template <typename T>
__global__ __launch_bounds__(1024) void k_norm_join(NormGradArgs a, int parts) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  const int which = a.dw ? blockIdx.y : 1;
  float t = 0.f;
  if (col < a.cols) {
    const int share = (parts + 15) / 16, p1 = min(parts, (wave + 1) * share);
#pragma unroll 4
    for (int p = wave * share; p < p1; ++p) t += a.part[((int64_t)p * 2 + which) * a.cols + col];
  }
  sums[wave][lane] = t;
  __syncthreads();
  if (wave > 0 || col >= a.cols) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) t += sums[w][lane];
  static_cast<T*>(which ? a.db : a.dw)[col] = cvt_x<T>(t);
}

// The fewest threads, a power of two from 8 on, that hold a row with `each` columns a thread.
int threads_of_row(int64_t cols, int each) {
  int t = 8;
  while ((int64_t)t * each < cols) t *= 2;
  return t;
}
template <typename F>
void by_threads(int threads, F&& f) {
  switch (threads) {
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    case 32: return f(std::integral_constant<int, 32>{});
    case 64: return f(std::integral_constant<int, 64>{});
    case 128: return f(std::integral_constant<int, 128>{});
    case 256: return f(std::integral_constant<int, 256>{});
    case 512: return f(std::integral_constant<int, 512>{});
    default: return f(std::integral_constant<int, 1024>{});
  }
}
// Workgroups that have a row each (or as many rows as they have sets of threads).
int64_t row_groups(int64_t rows, int threads) {
  const int per = kThreads(threads) / threads;
  return (rows + per - 1) / per;
}
// Columns a thread of the forward pass: eight up to 512 columns, then 16.
int forward_columns(int64_t cols) { return cols <= 512 ? 8 : 16; }

template <typename T>
hipError_t forward(const NormArgs& a, hipStream_t s) {
  if (a.cols > kWideCols) {
    hipLaunchKernelGGL((k_norm_wide<T>), dim3((unsigned)std::min<int64_t>(a.rows, kWideGrid)), dim3(kWide), 0, s, a);
    return hipGetLastError();
  }
  const int each = forward_columns(a.cols), threads = threads_of_row(a.cols, each);
  const unsigned grid = (unsigned)std::min<int64_t>(row_groups(a.rows, threads), 2048);
  by_threads(threads, [&](auto tpr) {
    constexpr int TPR = decltype(tpr)::value;
    const dim3 block(kThreads(TPR));
    if constexpr (TPR <= 64) {
      if (each == 8) hipLaunchKernelGGL((k_norm<T, TPR, 1>), dim3(grid), block, 0, s, a);
    }
    if constexpr (TPR >= 64) {
      if (each == 16) hipLaunchKernelGGL((k_norm<T, TPR, 2>), dim3(grid), block, 0, s, a);
    }
  });
  return hipGetLastError();
}

template <typename T>
hipError_t backward(const NormGradArgs& a, hipStream_t s) {
  const int64_t parts = norm_parts(a.rows, a.cols);
  hipError_t e = hipSuccess;
  if (a.cols > kWideGradCols) {
    if (a.dx && a.rows > 0)
      hipLaunchKernelGGL((k_norm_grad_wide<T>), dim3((unsigned)std::min<int64_t>(a.rows, kWideGrid)), dim3(kWide), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.part && parts > 0)
      hipLaunchKernelGGL((k_norm_cols<T>), dim3((unsigned)((a.cols + 2047) / 2048), (unsigned)parts), dim3(256), 0, s, a,
                         (a.rows + parts - 1) / parts);
  } else if (a.rows > 0) {
    by_threads(threads_of_row(a.cols, 8), [&](auto tpr) {
      constexpr int TPR = decltype(tpr)::value;
      hipLaunchKernelGGL((k_norm_grad<T, TPR>), dim3((unsigned)parts), dim3(kThreads(TPR)), 0, s, a);
    });
  }
  if ((e = hipGetLastError()) != hipSuccess || !(a.dw || a.db)) return e;
  hipLaunchKernelGGL((k_norm_join<T>), dim3((unsigned)((a.cols + 63) / 64), a.dw && a.db ? 2 : 1), dim3(1024), 0, s, a,
                     (int)parts);
  return hipGetLastError();
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t cols) {
  if (cols > kWideGradCols) return std::min<int64_t>((rows + 15) / 16, 64);
  const int threads = threads_of_row(cols, 8);
  return std::min<int64_t>(row_groups(rows, threads), 256 * 1024 / kThreads(threads));
}

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  return dtype == MUON_BF16 ? forward<uint16_t>(a, s) : forward<float>(a, s);
}

hipError_t launch_norm_grad(const NormGradArgs& a, int dtype, hipStream_t s) {
  if (a.cols == 0 || (a.rows == 0 && !a.dw && !a.db)) return hipSuccess;  // of no rows dw and db are zero
  return dtype == MUON_BF16 ? backward<uint16_t>(a, s) : backward<float>(a, s);
}

}  // namespace muon
