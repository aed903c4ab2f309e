// norm.hip -- layer norm and root-mean-square norm of rows, with the residual added ahead of them, and their
// gradients.
//
//   s = x + r,  y = xhat w + b,  xhat = (s - mean) rstd,  rstd = 1 / sqrt(var + eps)
//   g = dy w,   dx = rstd (g - mean(g) - xhat mean(g xhat)) + ds,  dw = sum dy xhat,  db = sum dy
//
// (The root-mean-square norm takes mean = 0 and has no mean(g).)  A row stays in the registers of TPR threads, CH
// pieces of eight columns each, so that it is read once; the variance is taken of the
// differences from the mean, in a second reduction, and loses nothing to a large mean.  y comes from the
// float32 sum s; what is kept of s for the gradient (and for the residual stream) has
// the tensors' type, so in bf16 xhat is there off by at most half a step of s times rstd.
//
// The gradient of w and b is a sum over rows: each thread adds up its columns over the rows that its
// workgroup walks, workgroups leave one row of partial sums each, and a second
// kernel adds those in order.
#include "act.h"
#include "group.h"
#include "norm.h"

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

// a.part: [workgroups][2][cols], dw's sums and db's.
template <typename T, int TPR, int CH>
__global__ __launch_bounds__(kThreads(TPR)) void k_norm_grad(NormGradArgs a) {
  constexpr int NT = kThreads(TPR), RPB = NT / TPR;
  __shared__ float red[2][RPB][2 * 16];
  __shared__ float sums[RPB > 1 ? NT * CH * 8 : 1];
  const int l = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float per = 1.f / (float)a.cols;
  int n[CH];
  float w[CH][8], dw[CH][8] = {}, db[CH][8] = {};
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (c * TPR + l) * 8;
    n[c] = (int)max((int64_t)0, min((int64_t)8, a.cols - col));
#pragma unroll
    for (int i = 0; i < 8; ++i) w[c][i] = 1.f;
    if (a.w) load8(static_cast<const T*>(a.w) + col, n[c], w[c]);
  }
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB, turn ^= 1) {
    const int64_t row = r0 + sub;
    const bool in = row < a.rows;
    const float mean = in && a.layer ? a.stats[2 * row] : 0.f, rstd = in ? a.stats[2 * row + 1] : 0.f;
    float x[CH][8], g[CH][8], d[CH][8] = {}, t[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (c * TPR + l) * 8, m = in ? n[c] : 0;
      load8(static_cast<const T*>(a.s) + row * a.lds + col, m, x[c]);
      load8(static_cast<const T*>(a.dy) + row * a.ldg + col, m, g[c]);
      if (a.ds) load8(static_cast<const T*>(a.ds) + row * a.ldd + col, m, d[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[c][i] = i < m ? (x[c][i] - mean) * rstd : 0.f;
        dw[c][i] += g[c][i] * x[c][i];
        db[c][i] += g[c][i];
        g[c][i] *= w[c][i];
        t[0] += g[c][i];
        t[1] += g[c][i] * x[c][i];
      }
    }
    if (!a.dx) continue;  // uniform
    row_sum<TPR>(t, red[turn][sub]);
    const float m1 = a.layer ? t[0] * per : 0.f, m2 = t[1] * per;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[c][i] += rstd * (g[c][i] - m1 - x[c][i] * m2);
      store8(static_cast<T*>(a.dx) + row * a.cols + (c * TPR + l) * 8, in ? n[c] : 0, d[c]);
    }
  }
  if (!a.part) return;
  // The workgroup's rows of threads are added in order.
  auto leave = [&](float (&v)[CH][8], int which) {
    float* to = a.part + ((int64_t)blockIdx.x * 2 + which) * a.cols;
    if constexpr (RPB == 1) {
#pragma unroll
      for (int c = 0; c < CH; ++c) store8(to + (c * TPR + l) * 8, n[c], v[c]);
    } else {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[sub * TPR * CH * 8 + (c * TPR + l) * 8 + i] = v[c][i];
      __syncthreads();
      for (int col = threadIdx.x; col < a.cols; col += NT) {
        float t = 0.f;
        for (int q = 0; q < RPB; ++q) t += sums[q * TPR * CH * 8 + col];
        to[col] = t;
      }
    }
  };
  if (a.dw) leave(dw, 0);
  if (a.db) leave(db, 1);
}

// Rows longer than the registers of a workgroup hold: read three times.
// (A gradient's row takes more registers: 1024 threads would not hold 16 of its columns each.)
constexpr int kWide = 1024, kWideCols = 16384, kWideGradCols = 8192;

template <typename T>
__global__ __launch_bounds__(kWide) void k_norm_wide(NormArgs a) {
  __shared__ float red[2][16];
  const int64_t row = blockIdx.x;
  const float per = 1.f / (float)a.cols;
  auto get = [&](int64_t col, float (&v)[8]) {
    const int n = (int)min((int64_t)8, a.cols - col);
    load8(static_cast<const T*>(a.x) + row * a.ldx + col, n, v);
    if (a.res) {
      float r[8];
      load8(static_cast<const T*>(a.res) + row * a.ldr + col, n, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    return n;
  };
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
}

template <typename T>
__global__ __launch_bounds__(kWide) void k_norm_grad_wide(NormGradArgs a) {
  __shared__ float red[2 * 16];
  const int64_t row = blockIdx.x;
  const float per = 1.f / (float)a.cols, mean = a.layer ? a.stats[2 * row] : 0.f, rstd = a.stats[2 * row + 1];
  float x[8], g[8], t[2] = {0.f, 0.f};
  auto get = [&](int64_t col) {
    const int n = (int)min((int64_t)8, a.cols - col);
    load8(static_cast<const T*>(a.s) + row * a.lds + col, n, x);
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
    load8(static_cast<const T*>(a.s) + row * a.lds + col, n, x);
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

// Threads of a row: enough for eight columns each up to 512, then 16 each.
int threads_of_row(int64_t cols) {
  int t = 8;
  while (t < 64 && (int64_t)t * 8 < cols) t *= 2;
  while (t * 16 < cols) t *= 2;
  return t;
}
template <int MOST, typename F>
void by_width(int64_t cols, F&& f) {
  switch (threads_of_row(cols)) {
    case 8: return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
    case 16: return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    case 32: return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
    case 64:
      if (cols <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
      return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    case 128: return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 2>{});
    case 256: return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    case 512: return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
    default:
      if constexpr (MOST > 8192) return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
  }
}
int64_t row_groups(int64_t rows, int64_t cols) {
  const int t = threads_of_row(cols), per = kThreads(t) / t;
  return (rows + per - 1) / per;
}

template <typename T>
hipError_t forward(const NormArgs& a, hipStream_t s) {
  if (a.cols > kWideCols) {
    hipLaunchKernelGGL((k_norm_wide<T>), dim3((unsigned)a.rows), dim3(kWide), 0, s, a);
    return hipGetLastError();
  }
  const unsigned grid = (unsigned)std::min<int64_t>(row_groups(a.rows, a.cols), 2048);
  by_width<kWideCols>(a.cols, [&](auto tpr, auto ch) {
    constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
    hipLaunchKernelGGL((k_norm<T, TPR, CH>), dim3(grid), dim3(kThreads(TPR)), 0, s, a);
  });
  return hipGetLastError();
}

template <typename T>
hipError_t backward(const NormGradArgs& a, hipStream_t s) {
  const int64_t parts = norm_parts(a.rows, a.cols);
  hipError_t e = hipSuccess;
  if (a.cols > kWideGradCols) {
    if (a.dx) hipLaunchKernelGGL((k_norm_grad_wide<T>), dim3((unsigned)a.rows), dim3(kWide), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.part && parts > 0)
      hipLaunchKernelGGL((k_norm_cols<T>), dim3((unsigned)((a.cols + 2047) / 2048), (unsigned)parts), dim3(256), 0, s, a,
                         (a.rows + parts - 1) / parts);
  } else if (a.rows > 0) {
    by_width<kWideGradCols>(a.cols, [&](auto tpr, auto ch) {
      constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
      hipLaunchKernelGGL((k_norm_grad<T, TPR, CH>), dim3((unsigned)parts), dim3(kThreads(TPR)), 0, s, a);
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
  return std::min<int64_t>(row_groups(rows, cols), 512);
}

hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  return dtype == MUON_BF16 ? forward<uint16_t>(a, s) : forward<float>(a, s);
}

hipError_t launch_norm_grad(const NormGradArgs& a, int dtype, hipStream_t s) {
  if (a.cols == 0) return hipSuccess;
  return dtype == MUON_BF16 ? backward<uint16_t>(a, s) : backward<float>(a, s);
}

}  // namespace muon
