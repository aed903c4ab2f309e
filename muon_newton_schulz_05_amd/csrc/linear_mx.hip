// linear_mx.hip -- products of rows and weights held in four bits (mx.h), with the epilogue of the linear layers.
//
// The matrix instruction takes 16 rows by 128 values of both operands, 32 consecutive values and their scale in each
// lane, and adds their products in float32.  It multiplies four times what bf16's does in the same time from the same
// bytes, so what surrounds it counts four times as much.
//
//  - Tiles: four waves share BM x BN, each a quarter of it.  Slices of 128 values go from memory straight into LDS, NS
//    stages deep, one barrier a slice.  Two or more workgroups share a compute unit, so that one multiplies while
//    another waits at its barrier, or writes its result.  A slice's 64-byte row has its 16-byte piece c at slot
//    c ^ (-(row / 4) mod 4): the sixteen lanes that LDS serves at once (0 to 3, 12 to 15 and 20 to 27, say: pieces of two
//    lane groups) touch distinct banks.  What is
//    out of range lies past a buffer descriptor's end and loads as zero.
//  - Few rows: nothing is shared, so the weight goes from memory to registers as the instruction takes it.  Each of
//    eight waves takes every eighth chunk of 512 values for all rows, and they add up in order in LDS.
//
// What bounds it.  A loop of nothing but these instructions on random operands reaches 6.6 - 6.8 PFLOP/s under the card's
// power limit (9.4 - 9.7 on zeros).  Times of the product alone, medians of several sessions: 16384^3 1750 - 1855 us (4.7 - 5.0
// PFLOP/s), the matrix cores 72% busy at 1.68 GHz, so that what moves operands takes its part of the power; 8192 x 16384 x 4096
// 230 - 255 (4.3 - 4.8).  8192 x 4096 x 16384 with gelu, bias and residual 358 - 380, with the bias alone 283 - 312: with 32
// slices a tile, starts and epilogues are 20 - 35% of the time, and only
// partly behind another workgroup's products (y written and the residual read are 512 MiB).  Stores that pass the caches by took 6 - 16% off, and more than that
// on top of the kernel that reads y next.  1 x 4096 x 16384, the whole call: 9.4 us, the weight's 36 MB at 3.8 TB/s, start and end included.
#include "gemm.h"
#include "mx_device.h"

namespace muon {
namespace {

constexpr uint32_t kRsrcFlags = 0x00020000;

// Rows' products: C += A B^T of 16 x 16, byte S of sa and sb the scales.
template <int S>
__device__ __forceinline__ f32x4_t multiply4(u32x4_t a, u32x4_t b, f32x4_t c, uint32_t sa, uint32_t sb) {
  typedef int i32x8_t __attribute__((ext_vector_type(8)));
  const i32x8_t a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};  // four bits read the first half
  const i32x8_t b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  constexpr int kE2m1 = 4;
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, kE2m1, kE2m1, S, (int)sa, S, (int)sb);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t descriptor(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, kRsrcFlags);
}
// Load U of 1 KiB of those that lie one behind the other in memory and in LDS (an instruction's offset counts for both).
template <int U>
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t rs, uint32_t off, char* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (void LDS_PTR*)dst, 16, off, 0, U * 1024, 0);
}

// What all lanes share, in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}

// f of 0 .. N - 1, as constants.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void counted(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    counted<N, I + 1>(f);
  }
}

// The workgroup's place: its rows [row0, end) of group e, its column tile, its slices [s0, s0 + steps).
struct Place {
  int64_t row0, end;
  int e, tn, split, s0, steps;
  // False where there is nothing to do (uniform, ahead of any barrier).
  __device__ __forceinline__ bool find(const GemmArgs& g, int bm) {
    int tm;
    split = 0;
    e = 0;
    s0 = 0;
    end = g.m;
    int s1 = (int)g.k;
    if (g.offsets) {
      const GroupBlocks gb(g.offsets, g.groups, g.m, bm);
      const int total = min(gb.total, g.tiles_m);
      if ((int)blockIdx.x >= total * g.tiles_n) return false;
      stripe(xcd_place(blockIdx.x, total * g.tiles_n), total, g.tiles_n, tm, tn);
      int lo, hi;
      gb.find(g.offsets, g.groups, g.m, bm, tm, e, lo, hi);
      e = uniform(e);
      row0 = uniform(lo);
      end = uniform(hi);
      if (e == g.groups) s1 = 0;  // rows past the last group: zeros
    } else {
      const int tiles = g.tiles_m * g.tiles_n;
      split = blockIdx.x / tiles;
      stripe(xcd_place(blockIdx.x - split * tiles, tiles), g.tiles_m, g.tiles_n, tm, tn);
      row0 = (int64_t)tm * bm;
      s0 = split * (int)g.k_per;
      s1 = min(s1, s0 + (int)g.k_per);
    }
    steps = max(0, s1 - s0);
    return true;
  }
};

// The activation of N pieces of eight, chosen once for all of them.
template <int ACT, int N>
__device__ __forceinline__ void act_all(float (&v)[N][8]) {
#pragma unroll
  for (int p = 0; p < N; ++p)
#pragma unroll
    for (int u = 0; u < 8; ++u) v[p][u] = act_f(v[p][u], ACT);
}
template <int N>
__device__ __forceinline__ void activate(float (&v)[N][8], int act) {
  switch (act) {
    case MUON_ACT_RELU: return act_all<MUON_ACT_RELU>(v);
    case MUON_ACT_SILU: return act_all<MUON_ACT_SILU>(v);
    case MUON_ACT_GELU: return act_all<MUON_ACT_GELU>(v);
    case MUON_ACT_GELU_TANH: return act_all<MUON_ACT_GELU_TANH>(v);
    default: return;
  }
}
template <typename O>
__device__ __forceinline__ void bias8(const GemmArgs& g, const Place& at, int col, int n, float (&bias)[8]) {
  if (g.bias && !g.part && n > 0 && !(g.offsets && at.e == g.groups))
    load8(static_cast<const O*>(g.bias) + at.e * g.sbias + col, n, bias);
}

template <typename O, int BM, int BN, int WGM, int WGN, int NS>
__global__ __launch_bounds__(64 * WGM * WGN, 2) void k_mx_tile(MxProduct a) {
  constexpr int NW = WGM * WGN, WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16, SB = kMxSliceBytes;
  constexpr int LA = BM * SB / 1024 / NW, LB = BN * SB / 1024 / NW, L = LA + LB;  // a wave's loads of a slice
  // and of a chunk's scales, 64 rows each (those past the tiles' rows write zeros)
  constexpr int SL = ((BM + BN) / 64 + NW - 1) / NW;
  constexpr int STAGE = (BM + BN) * SB, STRIDE = WN * 4 + 16;
  constexpr int LOOP = NS * STAGE + SL * NW * 1024, EPI = NW * 32 * STRIDE;
  static_assert(NS == 3 || NS == 4, "the waits below");
  __shared__ __attribute__((aligned(1024))) char lds[LOOP > EPI ? LOOP : EPI];
  const GemmArgs& g = a.g;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WGM, wn = wave / WGM;
  Place at;
  if (!at.find(g, BM)) return;
  const int64_t row0 = at.row0, col0 = (int64_t)at.tn * BN;
  const int rows_a = uniform((int)min((int64_t)BM, at.end - row0)), rows_b = uniform((int)min((int64_t)BN, g.n - col0));
  const int steps = uniform(at.steps);
  const uint8_t* A = static_cast<const uint8_t*>(g.a) + (at.s0 * g.m + row0) * SB;
  const uint8_t* B = static_cast<const uint8_t*>(g.b) + (steps ? at.e : 0) * g.sb + (at.s0 * g.n + col0) * SB;
  const uint8_t* SA = a.sca + (at.s0 / 4 * g.m + row0) * kMxChunkBytes;
  const uint8_t* SC = a.scb + (steps ? at.e : 0) * (mx_chunks(a.kx) * g.n * kMxChunkBytes) + (at.s0 / 4 * g.n + col0) * kMxChunkBytes;

  char* const scales = lds + NS * STAGE;
  // A load of 1 KiB is 16 rows of a slice: lane l fills slot l mod 4 of row l / 4.
  const uint32_t from = (lane >> 2) * SB + (((lane & 3) ^ (-(lane >> 4) & 3)) << 4);
  const uint8_t* const A_wave = A + wave * LA * 1024;
  const uint8_t* const B_wave = B + wave * LB * 1024;
  const int bytes_a = max(0, rows_a * SB - wave * LA * 1024), bytes_b = max(0, rows_b * SB - wave * LB * 1024);
  // Load U of slice h: A's, then B's.
  auto issue = [&](int h, char* st, auto which) __attribute__((always_inline)) {
    constexpr int U = decltype(which)::value;
    const bool in = h < steps;
    if constexpr (U < LA) to_lds<U>(descriptor(A_wave + (int64_t)h * g.m * SB, in ? bytes_a : 0), from, st + wave * LA * 1024);
    else to_lds<U - LA>(descriptor(B_wave + (int64_t)h * g.n * SB, in ? bytes_b : 0), from, st + BM * SB + wave * LB * 1024);
  };
  auto issue_all = [&](int h, char* st) __attribute__((always_inline)) { counted<L>([&](auto u) { issue(h, st, u); }); };
  // This wave's loads of scales: where the first chunk's are, the step to the next one's, and their bytes.
  const uint8_t* scale_from[SL];
  int64_t scale_step[SL];
  int scale_bytes[SL];
#pragma unroll
  for (int u = 0; u < SL; ++u) {
    const int r = (wave * SL + u) * 64;  // of the tile's rows of A, then B
    const bool of_a = r < BM;
    const int left = r >= BM + BN ? 0 : of_a ? rows_a - r : rows_b - (r - BM);
    scale_from[u] = uniform(of_a ? SA + (int64_t)r * kMxChunkBytes : SC + (int64_t)(r - BM) * kMxChunkBytes);
    scale_step[u] = (of_a ? g.m : g.n) * kMxChunkBytes;
    scale_bytes[u] = uniform(max(0, min(left, 64)) * kMxChunkBytes);
  }
  auto issue_scales = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < SL; ++u)
      to_lds<0>(descriptor(scale_from[u] + chunk * scale_step[u], 4 * chunk < steps ? scale_bytes[u] : 0), 16 * lane,
                scales + (wave * SL + u) * 1024);
  };

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{};
  // Fragments: A's of one slice, each replaced by the next slice's once it has been multiplied, and B's of two.
  u32x4_t af[FM] = {}, bf[2][FN] = {};
  uint32_t sa[FM] = {}, sb[FN] = {};
  const int i16 = lane & 15, g4 = lane >> 4;
  const char* const frag_at = lds + i16 * SB + ((g4 ^ (-(i16 >> 2) & 3)) << 4);
  const char* const scale_at = scales + i16 * kMxChunkBytes + g4 * 4;
  auto read_scales = [&] __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = *reinterpret_cast<const uint32_t*>(scale_at + (BM + wn * WN + 16 * j) * kMxChunkBytes);
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = *reinterpret_cast<const uint32_t*>(scale_at + (wm * WM + 16 * i) * kMxChunkBytes);
  };
  // Multiplies slice S of its chunk (products of B by A: a block's register u in a lane is row lane mod 16 and column 4
  // (lane / 16) + u) and, with MORE, reads the next slice from st in its place and lets slice h's loads to `fill` out, one
  // behind each block's products: together they would hold up the wave.  The order is kept as written: left to
  // itself the compiler holds fragments of three slices, and spills.
  auto multiply = [&](auto slice, auto more, const char* st, int h, char* fill) __attribute__((always_inline)) {
    constexpr int S = decltype(slice)::value, Q = S & 1;
    constexpr bool MORE = decltype(more)::value;
    counted<FM>([&](auto row) __attribute__((always_inline)) {
      constexpr int i = decltype(row)::value;
      if constexpr (MORE && i < FN) bf[Q ^ 1][i] = *reinterpret_cast<const u32x4_t*>(st + (BM + wn * WN + 16 * i) * SB);
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = multiply4<S>(bf[Q][j], af[i], acc[i][j], sb[j], sa[i]);
      if constexpr (MORE) {
        af[i] = *reinterpret_cast<const u32x4_t*>(st + (wm * WM + 16 * i) * SB);
        static_assert(L <= FM, "loads of a slice");
        if constexpr (i < L) issue(h, fill, row);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  const bool idle = wm * WM >= rows_a || wn * WN >= rows_b;  // nothing of C: such a wave only loads
  int stage = 0;
  // Slice h, the P-th of its chunk: wait for it (what was issued after it stays in flight), let the slice NS - 1 ahead
  // take the stage that all have read, read this one's fragments and multiply those of the slice before.  A chunk's scales
  // are read at its second slice, ahead of its first products, and the next chunk's are loaded at its third.
  auto step = [&](int h, auto place, auto idle_tag) __attribute__((always_inline)) {
    constexpr int P = decltype(place)::value;
    constexpr bool LATER = NS == 3 ? P == 3 : P == 3 || P == 0;  // scales were issued after this slice
    wait_loads<(NS - 2) * L + (LATER ? SL : 0)>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if constexpr (P == 2) issue_scales((h >> 2) + 1);
    char* const fill = lds + (stage == 0 ? NS - 1 : stage - 1) * STAGE;
    if constexpr (decltype(idle_tag)::value) {
      issue_all(h + NS - 1, fill);
    } else {
      if constexpr (P == 1) read_scales();
      __builtin_amdgcn_sched_barrier(0);
      multiply(std::integral_constant<int, (P + 3) & 3>{}, std::true_type{}, frag_at + stage * STAGE, h + NS - 1, fill);
    }
    stage = stage == NS - 1 ? 0 : stage + 1;
  };
  // Whole chunks: what lies past the last slice is zero.
  auto run = [&](auto idle_tag) __attribute__((always_inline)) {
    for (int h = 0; h < steps; h += 4) {
      step(h, std::integral_constant<int, 0>{}, idle_tag);
      step(h + 1, std::integral_constant<int, 1>{}, idle_tag);
      step(h + 2, std::integral_constant<int, 2>{}, idle_tag);
      step(h + 3, std::integral_constant<int, 3>{}, idle_tag);
    }
    if constexpr (!decltype(idle_tag)::value) multiply(std::integral_constant<int, 3>{}, std::false_type{}, nullptr, 0, nullptr);
  };
  if (steps > 0) {
    // As the steps ahead of the first would have: scales two steps ahead of it, with the slice of that step.
#pragma unroll
    for (int p = 0; p < NS - 1; ++p) {
      if (p == NS - 3) issue_scales(0);
      issue_all(p, lds + p * STAGE);
    }
    if (idle) run(std::true_type{});
    else run(std::false_type{});
    wait_loads<0>();
    __syncthreads();  // every wave is done with the stages
  }

  // 32 rows at a time through this wave's own staging, so that a row of C leaves as whole 16-byte pieces.  Where n is a
  // multiple of 8 every piece is whole, and the residual of the next rows is on its way while these are finished (its
  // loads one by one, each waited for, had taken a third of the kernel's time).
  constexpr int LPR = WN / 8, RPP = 64 / LPR, PS = 32 / RPP;
  char* stg = lds + wave * 32 * STRIDE;
  const int col = (int)col0 + wn * WN + 8 * (lane % LPR);
  const int n_in = (int)min((int64_t)8, g.n - col);
  float bias[8] = {};
  bias8<O>(g, at, col, n_in, bias);
  auto strips = [&](auto full_tag, auto res_tag) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(full_tag)::value, RES = decltype(res_tag)::value;
    constexpr int RV = sizeof(O) / 2;  // 16-byte registers of eight residuals
    u32x4_t res[RES ? PS : 1][RV];
    const O* const from = static_cast<const O*>(g.res) + (n_in > 0 ? col : 0);
    auto fetch = [&](int i) __attribute__((always_inline)) {
#pragma unroll
      for (int p = 0; p < (RES ? PS : 0); ++p) {
        const int64_t row = min(row0 + wm * WM + 32 * i + p * RPP + lane / LPR, at.end - 1);
#pragma unroll
        for (int q = 0; q < RV; ++q) res[p][q] = load16(from + row * g.ldr + q * 4);
      }
    };
    fetch(0);
#pragma unroll
    for (int i = 0; i < WM / 32; ++i) {
#pragma unroll
      for (int ii = 0; ii < 2; ++ii)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          *reinterpret_cast<f32x4_t*>(stg + (16 * ii + i16) * STRIDE + (16 * j + 4 * g4) * 4) = acc[2 * i + ii][j];
      wave_fence();
      float v[PS][8];
#pragma unroll
      for (int p = 0; p < PS; ++p) {
        const f32x4_t* src = reinterpret_cast<const f32x4_t*>(stg + (p * RPP + lane / LPR) * STRIDE + (lane % LPR) * 32);
        const f32x4_t x = src[0], y = src[1];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[p][u] = u < 4 ? x[u & 3] : y[u & 3];
      }
      if (!g.part) {
#pragma unroll
        for (int p = 0; p < PS; ++p)
#pragma unroll
          for (int u = 0; u < 8; ++u) v[p][u] += bias[u];
        activate(v, g.act);
      }
      if constexpr (RES) {
#pragma unroll
        for (int p = 0; p < PS; ++p)
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            if constexpr (sizeof(O) == 2) v[p][u] += u & 1 ? bf16_hi(res[p][0][u / 2]) : bf16_lo(res[p][0][u / 2]);
            else v[p][u] += __uint_as_float(res[p][u / 4][u & 3]);
          }
        if (i + 1 < WM / 32) fetch(i + 1);
      }
#pragma unroll
      for (int p = 0; p < PS; ++p) {
        const int64_t row = row0 + wm * WM + 32 * i + p * RPP + lane / LPR;
        if (row < at.end && n_in > 0) {
          const int n = FULL ? 8 : n_in;
          if (g.part) {
            store8(g.part + ((int64_t)at.split * g.m + row) * g.n + col, n, v[p]);
          } else {
            if (!FULL && g.res) {
              float r[8];
              load8(static_cast<const O*>(g.res) + row * g.ldr + col, n, r);
#pragma unroll
              for (int u = 0; u < 8; ++u) v[p][u] += r[u];
            }
            store8(static_cast<O*>(g.c) + row * g.ldc + col, n, v[p]);
          }
        }
      }
      wave_fence();
    }
  };
  if ((g.n & 7) != 0) strips(std::false_type{}, std::false_type{});
  else if (g.res && !g.part) strips(std::true_type{}, std::true_type{});
  else strips(std::true_type{}, std::false_type{});
}

// Up to 16 FM rows of a group by 16 FN columns, in rounds of WK chunks, one a wave.  A wave's part of the weight goes
// to its registers at once; further rounds are hidden by other workgroups.  OWN: the workgroup takes its rows of x to four
// bits itself, in LDS, while the weight is on its way; otherwise they come in four bits, like the weight.
template <typename O, int FM, int FN, int WK, bool OWN>
__global__ __launch_bounds__(64 * WK) void k_mx_rows(MxProduct a) {
  constexpr int BM = 16 * FM, BN = 16 * FN, STRIDE = BN + 4, NT = 64 * WK;
  constexpr int XB = OWN ? WK * 4 * BM * kMxSliceBytes : 0, XS = OWN ? WK * BM * kMxChunkBytes : 0, SUMS = WK * BM * STRIDE * 4;
  __shared__ __attribute__((aligned(16))) char lds[XB + XS > SUMS ? XB + XS : SUMS];
  const GemmArgs& g = a.g;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int i16 = lane & 15, g4 = lane >> 4;
  Place at;
  if (!at.find(g, BM)) return;
  const int64_t col0 = (int64_t)at.tn * BN;
  const int rows_a = uniform((int)min((int64_t)BM, at.end - at.row0)), rows_b = uniform((int)min((int64_t)BN, g.n - col0));
  const int steps = uniform(at.steps), chunks = (steps + 3) / 4;
  const uint8_t* B = static_cast<const uint8_t*>(g.b) + (chunks ? at.e : 0) * g.sb + col0 * kMxSliceBytes;
  const uint8_t* SC = a.scb + (chunks ? at.e : 0) * (mx_chunks(a.kx) * g.n * kMxChunkBytes) + col0 * kMxChunkBytes;

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{};
  const int value_at = (i16 << 6) + (g4 << 4), scale_at = (i16 << 4) + (g4 << 2);  // of a lane, in 16 rows
  for (int c0 = 0; c0 < chunks; c0 += WK) {
    const int c = c0 + wave;  // zeros past the last chunk
    u32x4_t bf[4][FN], af[OWN ? 1 : 4][FM];
    uint32_t sb[FN], sa[FM];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int h = 4 * c + s;
      const __amdgpu_buffer_rsrc_t rb = descriptor(B + (int64_t)h * g.n * kMxSliceBytes, h < steps ? rows_b * kMxSliceBytes : 0);
#pragma unroll
      for (int j = 0; j < FN; ++j) bf[s][j] = __builtin_amdgcn_raw_buffer_load_b128(rb, value_at + j * 1024, 0, 0);
      if constexpr (!OWN) {
        const __amdgpu_buffer_rsrc_t ra = descriptor(static_cast<const uint8_t*>(g.a) + ((int64_t)h * g.m + at.row0) * kMxSliceBytes,
                                                     h < steps ? rows_a * kMxSliceBytes : 0);
#pragma unroll
        for (int i = 0; i < FM; ++i) af[s][i] = __builtin_amdgcn_raw_buffer_load_b128(ra, value_at + i * 1024, 0, 0);
      }
    }
    const __amdgpu_buffer_rsrc_t rs = descriptor(SC + (int64_t)c * g.n * kMxChunkBytes, c < chunks ? rows_b * kMxChunkBytes : 0);
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = __builtin_amdgcn_raw_buffer_load_b32(rs, scale_at + j * 256, 0, 0);
    if constexpr (!OWN) {
      const __amdgpu_buffer_rsrc_t ra = descriptor(a.sca + ((int64_t)c * g.m + at.row0) * kMxChunkBytes,
                                                   c < chunks ? rows_a * kMxChunkBytes : 0);
#pragma unroll
      for (int i = 0; i < FM; ++i) sa[i] = __builtin_amdgcn_raw_buffer_load_b32(ra, scale_at + i * 256, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);  // all of them are on their way before the first is waited for
    if constexpr (OWN) {
      // A thread takes eight values of a row at a time, four lanes a block; what LDS holds past the last row never gets
      // into a row of C.
      const int pieces = min(WK, chunks - c0) * 64;
      for (int u = tid; u < rows_a * pieces; u += NT) {
        const int r = u / pieces, p = u - r * pieces;
        const int64_t k = (int64_t)c0 * kMxChunk + p * 8;
        float v[8];
        load8(static_cast<const O*>(a.x) + (at.row0 + r) * a.ldx + k, (int)max((int64_t)0, min((int64_t)8, a.kx - k)), v);
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) m = max(m, magnitude(v[q]));
        m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));
        m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));
        const int scale = scale_of(m);
        *reinterpret_cast<uint32_t*>(lds + ((p >> 4) * BM + r) * kMxSliceBytes + (p & 15) * 4) = pack8(v, scale);
        if ((p & 3) == 0)
          lds[XB + ((p >> 6) * BM + r) * kMxChunkBytes + 4 * ((p >> 2) & 3) + ((p >> 4) & 3)] = (char)scale;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < FM; ++i)
        sa[i] = *reinterpret_cast<const uint32_t*>(lds + XB + (wave * BM + 16 * i) * kMxChunkBytes + scale_at);
    }
    if (c < chunks) {
      counted<4>([&](auto tag) __attribute__((always_inline)) {
        constexpr int S = decltype(tag)::value;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          u32x4_t av;
          if constexpr (OWN) av = *reinterpret_cast<const u32x4_t*>(lds + ((4 * wave + S) * BM + 16 * i) * kMxSliceBytes + value_at);
          else av = af[S][i];
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = multiply4<S>(bf[S][j], av, acc[i][j], sb[j], sa[i]);
        }
      });
    }
    if constexpr (OWN) __syncthreads();
  }
  float* const sums = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      *reinterpret_cast<f32x4_t*>(sums + (wave * BM + 16 * i + i16) * STRIDE + 16 * j + 4 * g4) = acc[i][j];
  __syncthreads();
  for (int u = tid; u < BM * BN / 8; u += NT) {
    const int lr = u / (BN / 8), c8 = u % (BN / 8) * 8, col = (int)col0 + c8;
    const int n = (int)min((int64_t)8, g.n - col);
    if (lr >= rows_a || n <= 0) continue;
    float v[8] = {}, bias[8] = {};
#pragma unroll
    for (int w = 0; w < WK; ++w)
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += sums[(w * BM + lr) * STRIDE + c8 + q];
    bias8<O>(g, at, col, n, bias);
    finish8<O>(g, v, bias, 0, at.row0 + lr, col, n);
  }
}

// Eight waves where the contraction has a chunk for each, else four.
template <typename O, int FM, int FN, bool OWN>
void launch_waves(const MxProduct& a, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.g.tiles_m * a.g.tiles_n));
  if (a.g.k > 16) hipLaunchKernelGGL((k_mx_rows<O, FM, FN, 8, OWN>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((k_mx_rows<O, FM, FN, 4, OWN>), grid, dim3(256), 0, s, a);
}
template <typename O, int FM, bool OWN>
void launch_rows(const MxProduct& a, int cols, hipStream_t s) {
  if (cols == 64) launch_waves<O, FM, 4, OWN>(a, s);
  else if (cols == 32) launch_waves<O, FM, 2, OWN>(a, s);
  else launch_waves<O, FM, 1, OWN>(a, s);
}

template <typename O>
hipError_t launch(const MxProduct& a, int tile, int cols, hipStream_t s) {
  const int64_t blocks = (int64_t)a.g.tiles_m * a.g.tiles_n * a.g.splits;
  if (blocks <= 0) return hipSuccess;
  const dim3 grid((unsigned)blocks);
  if (tile == kMx256x128) hipLaunchKernelGGL((k_mx_tile<O, 256, 128, 2, 2, 3>), grid, dim3(256), 0, s, a);
  else if (tile == kMx128) hipLaunchKernelGGL((k_mx_tile<O, 128, 128, 2, 2, 4>), grid, dim3(256), 0, s, a);
  else if (tile == kMx64) hipLaunchKernelGGL((k_mx_tile<O, 64, 64, 2, 2, 4>), grid, dim3(256), 0, s, a);
  else if (tile == kMxRows32) launch_rows<O, 2, false>(a, cols, s);
  else if (tile == kMxRows16) launch_rows<O, 1, false>(a, cols, s);
  else launch_rows<O, 1, true>(a, cols, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_product(const MxProduct& a, int dtype, int tile, int cols, hipStream_t s) {
  return dtype == MUON_BF16 ? launch<uint16_t>(a, tile, cols, s) : launch<float>(a, tile, cols, s);
}

}  // namespace muon
