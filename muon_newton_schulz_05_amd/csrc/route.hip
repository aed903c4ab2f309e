// route.hip -- tokens sorted by expert, moved there and back with weights, and
// the gradients of both moves.
//
// The sort is a stable counting sort.  Integer counts are exact in any
// order, so the histogram may use LDS atomics; a rank inside a wave comes from
// ballots over the bits of the expert index, which keeps the flat order.
// The moves are bound by memory.  They are cut by tokens, not by sorted rows:
// a token's row (or its gradient) is read once and meets its `top` rows
// from registers, and each sum over them runs in the order of the choices.
// 16384 tokens x 8 of 64 experts at h = 2048 in bf16: sort 17 - 21 us, dispatch 103 - 116,
// combine and dispatch's gradient 114 - 117 each, combine's gradient 234 - 250, back to
// back and in a trace from cold clocks (4.6 - 5.9 TB/s).
// Up to 4096 entries the sort is one launch (64 tokens x 6: 3.5 us).
#include "act.h"
#include "device_common.h"
#include "ops.h"

namespace muon {
namespace {

// Expert of flat entry i, or -1 where it is not routed.
__device__ __forceinline__ int expert_of(const RouteArgs& a, int64_t i) {
  if (i >= a.entries) return -1;
  const int64_t v = a.ids64 ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
  return v >= 0 && v < a.experts ? (int)v : -1;
}

// Lanes of the wave that hold the same value (0 <= v < 2^bits).
__device__ __forceinline__ uint64_t same_lanes(int v, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool on = (v >> b) & 1;
    const uint64_t w = __ballot(on);
    m &= on ? w : ~w;
  }
  return m;
}

// One wave places entries [first, last): run[e] is the next free place of
// expert e in this wave's share (LDS, this wave's own).
__device__ void place_entries(const RouteArgs& a, int64_t first, int64_t last, int* run, int bits) {
  const int lane = threadIdx.x & 63;
  for (int64_t i0 = first; i0 < last; i0 += 64) {
    const int64_t i = i0 + lane;
    const int e = i < last ? expert_of(a, i) : -1;
    const uint64_t same = same_lanes(e < 0 ? a.experts : e, bits);
    const int rank = __popcll(same & ((1ull << lane) - 1));
    const int base = e >= 0 ? run[e] : 0;
    wave_fence();
    if (e >= 0 && rank == 0) run[e] = base + __popcll(same);
    wave_fence();
    if (i < last) {
      a.position[i] = e >= 0 ? base + rank : -1;
      if (e >= 0) a.order[base + rank] = (int32_t)i;
    }
  }
}

__device__ __forceinline__ int id_bits(int experts) { return 32 - __builtin_clz(experts); }  // values 0 .. experts

// Exclusive prefix of v over the workgroup's threads (NT of them); total in *sum.
template <int NT>
__device__ int block_prefix(int v, int* sum) {
  __shared__ int waves[NT / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(incl, d, 64);
    if (lane >= d) incl += u;
  }
  if (lane == 63) waves[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < NT / 64; ++w) {
    if (w < wave) before += waves[w];
    all += waves[w];
  }
  *sum = all;
  return before + incl - v;
}

constexpr int kSmallWaves = 16;
constexpr int kSmallEntries = 4096;  // entries of the one-launch sort

// The whole sort in one workgroup: each wave counts its contiguous share, a
// prefix over experts and waves gives every wave its places.
__global__ __launch_bounds__(64 * kSmallWaves) void k_route_small(RouteArgs a) {
  __shared__ int run[kSmallWaves][kRouteMaxExperts];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t share = ((a.entries + kSmallWaves - 1) / kSmallWaves + 63) / 64 * 64;
  const int64_t first = min(a.entries, wave * share), last = min(a.entries, first + share);
  for (int i = tid; i < kSmallWaves * a.experts; i += 64 * kSmallWaves) run[i / a.experts][i % a.experts] = 0;
  __syncthreads();
  for (int64_t i = first + lane; i < last; i += 64) {
    const int e = expert_of(a, i);
    if (e >= 0) atomicAdd(&run[wave][e], 1);
  }
  __syncthreads();
  int total = 0;
  if (tid < a.experts)
    for (int w = 0; w < kSmallWaves; ++w) total += run[w][tid];
  int all;
  int base = block_prefix<64 * kSmallWaves>(total, &all);
  if (tid < a.experts) {
    a.offsets[tid] = base;
    for (int w = 0; w < kSmallWaves; ++w) {
      const int c = run[w][tid];
      run[w][tid] = base;
      base += c;
    }
  }
  if (tid == 0) a.offsets[a.experts] = all;
  __syncthreads();
  place_entries(a, first, last, run[wave], id_bits(a.experts));
  for (int64_t p = all + tid; p < a.entries; p += 64 * kSmallWaves) a.order[p] = -1;
}

// Counts of one block of kRouteBlock entries.
__global__ __launch_bounds__(256) void k_route_count(RouteArgs a) {
  __shared__ int cnt[kRouteMaxExperts];
  for (int i = threadIdx.x; i < a.experts; i += 256) cnt[i] = 0;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * kRouteBlock;
#pragma unroll
  for (int u = 0; u < kRouteBlock / 256; ++u) {
    const int e = expert_of(a, i0 + u * 256 + threadIdx.x);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.experts; i += 256) a.hist[(int64_t)blockIdx.x * a.experts + i] = cnt[i];
}

// Turns the blocks' counts into places: hist[b][e] = offsets[e] + counts of e
// in the blocks before b.  One workgroup; a thread takes one expert and one of
// `parts` stretches of blocks.
__global__ __launch_bounds__(1024) void k_route_scan(RouteArgs a, int blocks) {
  __shared__ int sums[1024];
  __shared__ int starts[kRouteMaxExperts];
  const int tid = threadIdx.x, parts = 1024 / a.experts;
  const int e = tid % a.experts, part = tid / a.experts;
  const int per = (blocks + parts - 1) / parts;
  const int b0 = min(part * per, blocks), b1 = part < parts ? min(b0 + per, blocks) : b0;
  int s = 0;
  for (int b = b0; b < b1; ++b) s += a.hist[(int64_t)b * a.experts + e];
  if (part < parts) sums[part * a.experts + e] = s;
  __syncthreads();
  int total = 0;
  if (tid < a.experts)
    for (int p = 0; p < parts; ++p) total += sums[p * a.experts + tid];
  int all;
  const int base = block_prefix<1024>(total, &all);
  if (tid < a.experts) {
    starts[tid] = base;
    a.offsets[tid] = base;
  }
  if (tid == 0) a.offsets[a.experts] = all;
  __syncthreads();
  if (part >= parts) return;
  int at = starts[e];
  for (int p = 0; p < part; ++p) at += sums[p * a.experts + e];
  for (int b = b0; b < b1; ++b) {
    int32_t* h = a.hist + (int64_t)b * a.experts + e;
    const int c = *h;
    *h = at;
    at += c;
  }
}

// Places one block's entries: four waves, 512 consecutive entries each.
__global__ __launch_bounds__(256) void k_route_place(RouteArgs a) {
  __shared__ int run[4][kRouteMaxExperts];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t i0 = (int64_t)blockIdx.x * kRouteBlock;
  const int64_t first = min(a.entries, i0 + wave * (kRouteBlock / 4));
  const int64_t last = min(a.entries, first + kRouteBlock / 4);
  for (int i = tid; i < a.experts; i += 256)
    for (int w = 0; w < 4; ++w) run[w][i] = 0;
  __syncthreads();
  for (int64_t i = first + lane; i < last; i += 64) {
    const int e = expert_of(a, i);
    if (e >= 0) atomicAdd(&run[wave][e], 1);
  }
  __syncthreads();
  for (int i = tid; i < a.experts; i += 256) {
    int base = a.hist[(int64_t)blockIdx.x * a.experts + i];
    for (int w = 0; w < 4; ++w) {
      const int c = run[w][i];
      run[w][i] = base;
      base += c;
    }
  }
  __syncthreads();
  place_entries(a, first, last, run[wave], id_bits(a.experts));
  const int all = a.offsets[a.experts];
  for (int64_t p = i0 + tid; p < min(a.entries, i0 + kRouteBlock); p += 256)
    if (p >= all) a.order[p] = -1;
}

// ------------------------------------------------------------------ moves

constexpr int kCols = 512;  // columns of one wave's piece, 8 a lane

struct Piece {
  int64_t token, col;
  int n;  // this lane's columns inside the row (8 where FULL: h is a multiple of 8)
};
template <bool FULL>
__device__ __forceinline__ bool my_piece(const MoveArgs& a, Piece& p) {
  const int64_t per = (a.h + kCols - 1) / kCols, u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  p.token = u / per;
  p.col = (u - p.token * per) * kCols + (threadIdx.x & 63) * 8;
  p.n = FULL ? 8 : (int)min((int64_t)8, a.h - p.col);
  return p.token < a.tokens && p.col < a.h;
}
__device__ __forceinline__ int routed_rows(const MoveArgs& a) {
  return (int)min(max((int64_t)a.offsets[a.experts], (int64_t)0), a.tokens * a.top);
}
// A position read from memory, as a row of a [tokens top] tensor or -1.
__device__ __forceinline__ int64_t row_at(const MoveArgs& a, int64_t t, int j) {
  const int32_t p = a.position[t * a.top + j];
  return p >= 0 && p < a.tokens * a.top ? p : -1;
}

template <typename T, bool FULL, bool NT>
__global__ __launch_bounds__(256) void k_dispatch(MoveArgs a) {
  Piece p;
  if (!my_piece<FULL>(a, p)) return;
  float v[8];
  load8(static_cast<const T*>(a.x) + p.token * a.ldx + p.col, p.n, v);
  const int all = routed_rows(a);
  T* out = static_cast<T*>(a.out);
  for (int j = 0; j < a.top; ++j) {
    const int64_t r = row_at(a, p.token, j);
    if (r >= 0) store8<T, NT>(out + r * a.h + p.col, p.n, v);
  }
  const float zero[8] = {};
  for (int j = 0; j < a.top; ++j) {
    const int64_t r = p.token * a.top + j;
    if (r >= all) store8(out + r * a.h + p.col, p.n, zero);
  }
}

// out[t] = sum_j w[t][j] x[position[t][j]] (+ res); w null: all ones.  U rows are
// in flight at once.
template <typename T, int U, bool FULL, bool NT>
__global__ __launch_bounds__(256) void k_gather_sum(MoveArgs a) {
  Piece p;
  if (!my_piece<FULL>(a, p)) return;
  float sum[8] = {};
  for (int j0 = 0; j0 < a.top; j0 += U) {
    float v[U][8], w[U];
    int64_t r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r[u] = j0 + u < a.top ? row_at(a, p.token, j0 + u) : -1;
      w[u] = a.w && j0 + u < a.top ? a.w[p.token * a.top + j0 + u] : 1.f;
    }
    // Unguarded, so that the loads are in flight together: a row that is not
    // there is read from row 0 and not used.
#pragma unroll
    for (int u = 0; u < U; ++u)
      load8<T, NT>(static_cast<const T*>(a.x) + max(r[u], (int64_t)0) * a.ldx + p.col, p.n, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += r[u] >= 0 ? w[u] * v[u][i] : 0.f;
  }
  if (a.res) {
    float v[8];
    load8(static_cast<const T*>(a.res) + p.token * a.ldr + p.col, p.n, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += v[i];
  }
  store8(static_cast<T*>(a.out) + p.token * a.h + p.col, p.n, sum);
}

// One wave a token: dys[position[t][j]] = w[t][j] dy[t] and
// dw[t][j] = <dy[t], ys[position[t][j]]>, both from one reading of dy; rows of
// dys past the routed ones are zero.
template <typename T, int U, bool FULL, bool NT>
__global__ __launch_bounds__(256) void k_combine_grad(MoveArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (t >= a.tokens) return;
  const int all = routed_rows(a);
  T* out = static_cast<T*>(a.out);
  for (int j0 = 0; j0 < a.top; j0 += U) {
    int64_t r[U];
    float w[U], dot[U] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r[u] = j0 + u < a.top ? row_at(a, t, j0 + u) : -1;
      w[u] = j0 + u < a.top ? a.w[t * a.top + j0 + u] : 0.f;
    }
    for (int64_t c = lane * 8; c < a.h; c += kCols) {
      const int n = FULL ? 8 : (int)min((int64_t)8, a.h - c);
      float d[8], v[U][8];
      load8(static_cast<const T*>(a.g) + t * a.ldg + c, n, d);
      if (a.dw) {
#pragma unroll
        for (int u = 0; u < U; ++u) load8<T, NT>(static_cast<const T*>(a.x) + max(r[u], (int64_t)0) * a.ldx + c, n, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[u] += r[u] >= 0 ? d[i] * v[u][i] : 0.f;
      }
      if (out) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (r[u] >= 0) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = w[u] * d[i];
            store8<T, NT>(out + r[u] * a.h + c, n, o);
          }
      }
    }
    if (a.dw) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float s = wave_sum(dot[u]);
        if (lane == 0 && j0 + u < a.top) a.dw[t * a.top + j0 + u] = s;
      }
    }
  }
  if (!out) return;
  const float zero[8] = {};
  for (int j = 0; j < a.top; ++j) {
    const int64_t r = t * a.top + j;
    if (r < all) continue;
    for (int64_t c = lane * 8; c < a.h; c += kCols) store8(out + r * a.h + c, FULL ? 8 : (int)min((int64_t)8, a.h - c), zero);
  }
}

template <typename F>
hipError_t launch_units(int64_t units, F&& f) {
  const int64_t blocks = (units + 3) / 4;
  if (blocks <= 0) return hipSuccess;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  f((unsigned)blocks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.entries <= kSmallEntries) {
    hipLaunchKernelGGL(k_route_small, dim3(1), dim3(64 * kSmallWaves), 0, s, a);
    return hipGetLastError();
  }
  const int64_t blocks = (a.entries + kRouteBlock - 1) / kRouteBlock;
  hipLaunchKernelGGL(k_route_count, dim3((unsigned)blocks), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_route_scan, dim3(1), dim3(1024), 0, s, a, (int)blocks);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(k_route_place, dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

namespace {

// Sorted rows past the memory-side cache's 256 MB are streamed (non-temporal):
// kept in it, their write-back takes the next kernel's bandwidth.  16384 tokens
// x 8 at h = 2048, bf16 (512 MiB of sorted rows): dispatch, combine and both
// gradients 611 us against 647.  Smaller tensors stay for their reader.
template <typename T>
bool streams(const MoveArgs& a) {
  return a.tokens * a.top * a.h * (int64_t)sizeof(T) > (int64_t(256) << 20);
}

template <typename T, bool FULL>
void move_rows(const MoveArgs& a, unsigned blocks, hipStream_t s) {
  if (streams<T>(a)) hipLaunchKernelGGL((k_dispatch<T, FULL, true>), dim3(blocks), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_dispatch<T, FULL, false>), dim3(blocks), dim3(256), 0, s, a);
}
// Four rows in flight, eight where there are more than four choices (16384
// tokens x 8: combine's gradient 5% faster; with three choices four are faster, 28
// us against 34, the others being read for nothing).
template <typename T, int U, bool FULL>
void gather(const MoveArgs& a, unsigned blocks, hipStream_t s) {
  if (streams<T>(a)) hipLaunchKernelGGL((k_gather_sum<T, U, FULL, true>), dim3(blocks), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_gather_sum<T, U, FULL, false>), dim3(blocks), dim3(256), 0, s, a);
}
template <typename T, int U, bool FULL>
void combine_grad(const MoveArgs& a, unsigned blocks, hipStream_t s) {
  if (streams<T>(a)) hipLaunchKernelGGL((k_combine_grad<T, U, FULL, true>), dim3(blocks), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_combine_grad<T, U, FULL, false>), dim3(blocks), dim3(256), 0, s, a);
}
template <typename T>
void pick_gather(const MoveArgs& a, unsigned b, hipStream_t s) {
  const bool wide = a.top > 4, full = a.h % 8 == 0;
  if (wide) full ? gather<T, 8, true>(a, b, s) : gather<T, 8, false>(a, b, s);
  else full ? gather<T, 4, true>(a, b, s) : gather<T, 4, false>(a, b, s);
}
template <typename T>
void pick_combine_grad(const MoveArgs& a, unsigned b, hipStream_t s) {
  const bool wide = a.top > 4, full = a.h % 8 == 0;
  if (wide) full ? combine_grad<T, 8, true>(a, b, s) : combine_grad<T, 8, false>(a, b, s);
  else full ? combine_grad<T, 4, true>(a, b, s) : combine_grad<T, 4, false>(a, b, s);
}
int64_t pieces(const MoveArgs& a) { return a.tokens * ((a.h + kCols - 1) / kCols); }

}  // namespace

hipError_t launch_dispatch(const MoveArgs& a, int dtype, hipStream_t s) {
  return launch_units(pieces(a), [&](unsigned b) {
    const bool full = a.h % 8 == 0;
    if (dtype == MUON_BF16) full ? move_rows<uint16_t, true>(a, b, s) : move_rows<uint16_t, false>(a, b, s);
    else full ? move_rows<float, true>(a, b, s) : move_rows<float, false>(a, b, s);
  });
}

hipError_t launch_gather_sum(const MoveArgs& a, int dtype, hipStream_t s) {
  return launch_units(pieces(a), [&](unsigned b) {
    if (dtype == MUON_BF16) pick_gather<uint16_t>(a, b, s);
    else pick_gather<float>(a, b, s);
  });
}

hipError_t launch_combine_grad(const MoveArgs& a, int dtype, hipStream_t s) {
  return launch_units(a.tokens, [&](unsigned b) {
    if (dtype == MUON_BF16) pick_combine_grad<uint16_t>(a, b, s);
    else pick_combine_grad<float>(a, b, s);
  });
}

}  // namespace muon
