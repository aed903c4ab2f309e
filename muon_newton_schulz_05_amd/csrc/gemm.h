// gemm.h -- the tiled matrix product behind the linear and expert layers:
// C[i][j] = sum_k A[i][k] B[j][k], with either operand contiguous along k or
// along its rows, over groups of rows or of the contraction, and bias,
// activation and residual in the epilogue.
//
// A workgroup owns a BM x BN tile of C; each of its waves owns a block of it,
// as 16 x 16 matrix-core products.  Operand k-slices of KB = 128 bytes a row
// go from memory straight into LDS, NS stages deep, with one barrier a slice.
// What is out of range (rows past the group, the contraction's tail) is
// given an offset past the buffer descriptor's end, for which the load writes
// zeros to LDS.
//
//  - An operand contiguous along k sits in LDS as rows of KB bytes; the
//    16-byte chunk c of row r at slot c ^ (r / 2 mod 8), so that 16 lanes
//    reading one chunk of 16 rows touch 16 distinct 16-byte bank groups.
//  - An operand contiguous along its rows sits as k-rows.  bf16: fragments
//    are read by ds_read_b64_tr_b16, which hands lane i of 16 the column i of
//    a 4 x 16 block (four k of one row of the operand); the eight 32-byte
//    pieces that 32 lanes read at once are kept in distinct banks by an XOR of
//    the chunk with their k.  float32: 16 lanes read 16 consecutive values of
//    each of four k, no transposition.
//
// What bounds it.  bf16, 256 x 256 tiles, 8192^3: 1270 - 1420 TFLOP/s by card and
// layout (one run of the three: forward 1268, dx 1383, dW 1409); the matrix cores are
// busy 70 - 73% of the cycles, at about 1.9 GHz under the card's power limit (the best
// library kernel measured: 1574, 87% at 1.74 GHz).  The rest is waiting at the slices' barriers.  Four waves of
// 128 x 128 read a third less from LDS and were 7 - 12% slower; half slices, four
// or five deep, were equal for operands along their rows and 8% slower for
// operands along k, whose loads then take half lines.  With few slices a tile
// (experts: 12 to 32) the tile's start and its epilogue, about 12 us, show: one
// workgroup holds a unit's LDS, so nothing runs beside them.
#pragma once
#include <type_traits>

#include "act.h"
#include "device_common.h"
#include "ops.h"

namespace muon {
namespace {

#define LDS_PTR __attribute__((address_space(3)))

constexpr uint32_t kNoLoad = 0x80000000u;     // an offset past every descriptor's end
constexpr uint32_t kRecords = 0x7fffffffu;

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// LB bytes a lane from base + off (zeros past the descriptor's end) to LDS, lane l
// at byte LB l.
template <int LB>
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, char* dst) {
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, kRecords, 0x00020000);
  if constexpr (LB == 16) __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (void LDS_PTR*)dst, 16, off, 0, 0, 0);
  else __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (void LDS_PTR*)dst, 4, off, 0, 0, 0);
}
// Wait until at most N of this wave's loads are in flight and its LDS reads are
// done.  (The builtin, not inline asm: the compiler then knows that no LDS
// read is pending and adds no wait of its own behind it.)
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));  // vmcnt N, lgkmcnt 0, expcnt untouched
  asm volatile("" ::: "memory");
}
// Scheduling of one substep: RD fragment reads spread evenly over MM matrix-core
// products and VM loads to LDS over the first SV of them, each ahead of its
// product.
template <int RD, int VM, int SV, int MM, int Q = 0>
__device__ __forceinline__ void interleave() {
  if constexpr (Q < MM) {
    constexpr int vm = Q < SV ? ((Q + 1) * VM + SV - 1) / SV - (Q * VM + SV - 1) / SV : 0;
    constexpr int rd = ((Q + 1) * RD + MM - 1) / MM - (Q * RD + MM - 1) / MM;
    if constexpr (vm > 0) __builtin_amdgcn_sched_group_barrier(0x010, vm, 0);
    if constexpr (rd > 0) __builtin_amdgcn_sched_group_barrier(0x100, rd, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    interleave<RD, VM, SV, MM, Q + 1>();
  }
}

// Products of 16 x 16 blocks.  Against 32 x 32 x 16 the deeper contraction moves
// fewer accumulator registers a product (8 of 32 against 16 of 40 registers
// read and written a 32768 flops), which the card's power limit returns as clock.
template <typename T> struct Mma;
template <> struct Mma<uint16_t> {
  static constexpr int N = 1;
  typedef bf16x8_t Frag;  // eight k of one row: k = 32 s + 8 (lane / 16) + 0..7
  static __device__ __forceinline__ f32x4_t mul(Frag a, Frag b, f32x4_t c, int) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Mma<float> {
  static constexpr int N = 4;
  typedef f32x4_t Frag;   // four k of one row: k = 16 s + 4 (lane / 16) + 0..3
  static __device__ __forceinline__ f32x4_t mul(Frag a, Frag b, f32x4_t c, int q) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a[q], b[q], c, 0, 0, 0);
  }
};

constexpr int KB = 128;  // bytes of a k-slice's row

// One operand's tile: R rows x one k-slice, loaded by NW waves (PD: slices held in
// registers ahead of LDS where loads are not direct).
template <typename T, int R, bool TR, int NW, int LOADS, int PD>
struct Panel {
  static constexpr bool DIRECT = LOADS != kStaged;
  static constexpr int LB = LOADS == kDirect4 ? 4 : 16;  // bytes a lane
  static constexpr int EPC = 16 / sizeof(T);          // elements of a 16-byte chunk
  static constexpr int BK = KB / sizeof(T);           // k of a slice
  static constexpr int RB = TR ? R * (int)sizeof(T) : KB;  // bytes of an LDS row
  static constexpr int CPR = RB / 16;                 // its chunks
  static constexpr int BYTES = R * KB;
  static constexpr int LI = BYTES / (64 * LB) / NW;   // loads a wave and slice
  static constexpr int READS = !TR ? 1 : sizeof(T) == 2 ? 2 : 4;  // LDS reads of a fragment
  static_assert(BYTES % (64 * LB * NW) == 0, "whole loads");
  typedef typename Mma<T>::Frag Frag;

  static __device__ __forceinline__ int swz(int row) {
    if (!TR) return (row >> 1) & 7;
    if (sizeof(T) == 4) return (((row >> 2) & 3) << 2) & (CPR - 1);
    const int v = (row & 3) | (((row >> 3) & 1) << 2);  // eight k-rows read at once, 32 bytes of each
    return CPR >= 16 ? v << 1 : CPR == 8 ? (v >> 1) << 1 : (v >> 2) << 1;
  }

  const char* base;     // first element of this tile at k = 0 of the group
  int64_t ld;           // bytes from one row (k-row when TR) to the next
  uint32_t off[LI];     // this lane's offsets; kNoLoad outside the tile's rows
  int left[LI];         // not DIRECT: elements of the chunk inside the rows (TR) or 1 / 0
  u32x4_t reg[DIRECT ? 1 : PD][DIRECT ? 1 : LI];

  // Byte of the tile that load u fills in this lane; its 16-byte slot's row and
  // chunk, and the element inside the chunk.
  static __device__ __forceinline__ int place(int u, int wave, int lane) { return ((wave + NW * u) * 64 + lane) * LB; }
  static __device__ __forceinline__ int lrow(int b) { return b / RB; }
  static __device__ __forceinline__ int chunk(int b) { return (b % RB / 16) ^ swz(b / RB); }
  static __device__ __forceinline__ int element(int b) { return LB == 16 ? 0 : b % 16 / (int)sizeof(T); }

  // rows: rows of the operand inside the tile (at most R).
  __device__ __forceinline__ void init(const char* p, int64_t ld_bytes, int rows, int wave, int lane) {
    base = p;
    ld = ld_bytes;
#pragma unroll
    for (int u = 0; u < LI; ++u) {
      const int s = place(u, wave, lane), r = lrow(s), c = chunk(s);
      if constexpr (DIRECT) {
        const bool ok = TR ? c * EPC + element(s) < rows : r < rows;
        off[u] = ok ? (uint32_t)(r * (int)ld_bytes + c * 16 + element(s) * (int)sizeof(T)) : kNoLoad;
      } else {
        left[u] = TR ? min(EPC, rows - c * EPC) : (r < rows ? 1 : 0);
      }
    }
  }
  __device__ __forceinline__ const char* at(int kt) const { return base + (TR ? (int64_t)kt * BK * ld : (int64_t)kt * KB); }

  // DIRECT: slice kt into LDS; k_left: elements of the contraction from this
  // slice on (none left: zeros).  Branchless, so that the loads and the
  // products around them are scheduled as one block.
  __device__ __forceinline__ void issue(int kt, int k_left, char* st, int wave, int lane) {
    const char* p = at(kt);
    // A lane's first k.  In an operand contiguous along k the swizzle repeats every
    // 16 rows: with 16-byte pieces one value serves every load, with 4-byte
    // pieces every other one.
    static_assert(TR ? NW * 64 * LB % RB == 0 : (LB == 4 ? 2 : 1) * NW * 64 * LB / KB % 16 == 0, "rows of a lane");
    const int s0 = place(0, wave, lane), s1 = place(1, wave, lane);
    const int k0 = TR ? lrow(s0) : chunk(s0) * EPC + element(s0), k1 = LB == 4 ? chunk(s1) * EPC + element(s1) : k0;
#pragma unroll
    for (int u = 0; u < LI; ++u) {
      const int kk = TR ? k0 + u * (NW * 64 * LB / RB) : u & 1 ? k1 : k0;
      load_to_lds<LB>(p, kk < k_left ? off[u] : kNoLoad, st + (wave + NW * u) * 64 * LB);
    }
  }
  // Otherwise: slice kt into registers (any alignment; a chunk that is only
  // partly inside is taken element by element), then from there to LDS.
  __device__ __forceinline__ void fetch(int kt, int k_left, int q, int wave, int lane) {
#pragma unroll
    for (int u = 0; u < LI; ++u) {
      const int s = place(u, wave, lane), r = lrow(s), c = chunk(s);
      const int n = TR ? (r < k_left ? left[u] : 0) : (left[u] ? min(EPC, k_left - c * EPC) : 0);
      const char* p = at(kt) + (int64_t)r * ld + c * 16;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (n >= EPC) {
        __builtin_memcpy(&v, p, 16);
      } else {
        const T* el = reinterpret_cast<const T*>(p);
#pragma unroll
        for (int i = 0; i < EPC; ++i)
          if (i < n) {
            if constexpr (sizeof(T) == 4) v[i] = __float_as_uint(el[i]);
            else v[i / 2] |= (uint32_t)el[i] << (16 * (i & 1));
          }
      }
      reg[q][u] = v;
    }
  }
  __device__ __forceinline__ void put(char* st, int q, int wave, int lane) const {
#pragma unroll
    for (int u = 0; u < LI; ++u) *reinterpret_cast<u32x4_t*>(st + (wave + NW * u) * 1024 + lane * 16) = reg[q][u];
  }

  // The fragment of substep s (32 bf16 or 16 float32 of k) for rows
  // r0 .. r0 + 15 of the tile (r0 a multiple of 16).
  static __device__ __forceinline__ Frag frag(const char* st, int r0, int s, int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (!TR) {
      const int r = r0 + i;
      return *reinterpret_cast<const Frag*>(st + r * KB + (((4 * s + g) ^ swz(r)) << 4));
    } else if constexpr (sizeof(T) == 2) {
      const int k = 32 * s + 8 * g + (i >> 2);
      const int c = (r0 >> 3) + ((i & 3) >> 1);
      const char* p = st + k * RB + ((c ^ swz(k)) << 4) + (i & 1) * 8;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((s16x4_t LDS_PTR*)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((s16x4_t LDS_PTR*)(p + 4 * RB));
      typedef short s16x8_t __attribute__((ext_vector_type(8)));
      const s16x8_t v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(Frag, v);
    } else {
      const int c = (r0 + i) >> 2;
      Frag v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = 16 * s + 4 * g + j;
        v[j] = *reinterpret_cast<const float*>(st + k * RB + ((c ^ swz(k)) << 4) + (i & 3) * 4);
      }
      return v;
    }
  }
};

// z = v + bias (stored where asked), y = act(z) + res, eight columns of one row.
// y comes from the float32 z.  What is kept of z for the gradient has the layer's type: in
// bf16 half the bytes of float32, which a large layer would write and read once
// more, for a slope taken at most half a step of z away.
template <typename T>
__device__ __forceinline__ void finish8(const GemmArgs& g, float (&v)[8], const float (&bias)[8], int64_t e, int64_t row,
                                        int col, int n) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += bias[i];
  const int64_t at = e * g.sc + row * g.ldc + col;
  if (g.z) store8(static_cast<T*>(g.z) + at, n, v);
  if (g.act != MUON_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_f(v[i], g.act);
  }
  if (g.res) {
    float r[8];
    load8(static_cast<const T*>(g.res) + row * g.ldr + col, n, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  store8(static_cast<T*>(g.c) + at, n, v);
}

// Workgroups go to the 8 XCDs round robin: block b of n takes the place in
// which each XCD walks one contiguous stretch.
__device__ __forceinline__ int xcd_place(int b, int n) {
  const int x = b & 7, q = n >> 3, r = n & 7;
  return x * q + min(x, r) + (b >> 3);
}
// Tile t of a tiles_m x tiles_n grid, walked down stripes of 8 row tiles:
// the 32 tiles an XCD runs at once share 8 row and 4 column panels in its L2 (dx of
// [8192,4096]x[4096,16384] 801 us; with stripes of 4 829, of 2 946, of 16 910).
__device__ __forceinline__ void stripe(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int per = 8 * tiles_n, s = t / per, w = min(8, tiles_m - 8 * s), u = t - s * per;
  tn = u / w;
  tm = 8 * s + u - tn * w;
}

// WGM x WGN waves share a tile; WGK such sets of waves take every WGK-th k-slice
// each, with stages of their own, and add up in the epilogue in set order.
template <typename T, int BM, int BN, int WGM, int WGN, int WGK, int NS, bool TA, bool TB, int LOADS>
__global__ __launch_bounds__(64 * WGM * WGN * WGK) void k_gemm(GemmArgs g) {
  constexpr int NW = WGM * WGN, WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  constexpr bool DIRECT = LOADS != kStaged;
  constexpr int PD = DIRECT ? 1 : 4;
  typedef Panel<T, BM, TA, NW, LOADS, PD> PA;
  typedef Panel<T, BN, TB, NW, LOADS, PD> PB;
  typedef typename Mma<T>::Frag Frag;
  constexpr int BK = PA::BK, SUB = KB / 64, STAGE = PA::BYTES + PB::BYTES;
  constexpr int STRIDE = WN * 4 + 16;  // bytes of a staged epilogue row: 16 rows at one column fall on distinct 16-byte bank groups
  constexpr int LDS = WGK * (NS * STAGE > NW * 32 * STRIDE ? NS * STAGE : NW * 32 * STRIDE);
  __shared__ __attribute__((aligned(1024))) char lds[LDS];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = wave_all % NW, set = wave_all / NW;
  static_assert(WGK == 1 || (DIRECT && BM == 32), "sets of waves: direct loads, one strip of rows");
  static_assert(DIRECT || (NS == 2 && BM * BN <= 64 * 64), "staged loads: two stages, registers for four slices");
  // Waves w and w + 4 share a SIMD.  With 2 x 4 of them, each SIMD gets one wave
  // of the tile's upper and one of its lower half, and one of its left and one of
  // its right half, so that a tile with half of its rows or columns outside
  // C leaves every SIMD half its work (64 experts' [2048, 1408], whose last column
  // tile is half empty: forward 439 us against 460).
  const int wm = NW == 8 && WGM == 2 ? (wave & 1) ^ (wave >> 2) : wave / WGN;
  const int wn = NW == 8 && WGM == 2 ? (wave >> 1) & 3 : wave % WGN;

  // ---- which tile
  constexpr bool GK = TA && TB;  // groups divide the contraction
  const int tiles = g.tiles_m * g.tiles_n;
  int b = blockIdx.x, split = 0, e = 0, tm, tn;
  int64_t row0, end = g.m, k0 = 0, k1 = g.k;
  if (!GK && g.offsets) {
    // The grid is an upper bound: what the groups really fill is counted here, so
    // that every XCD gets its share of it.
    const GroupBlocks gb(g.offsets, g.groups, g.m, BM);
    const int total = min(gb.total, g.tiles_m);  // the bound itself, where offsets do not ascend
    if (b >= total * g.tiles_n) return;          // uniform, before any barrier
    stripe(xcd_place(b, total * g.tiles_n), total, g.tiles_n, tm, tn);
    int lo, hi;
    gb.find(g.offsets, g.groups, g.m, BM, tm, e, lo, hi);
    row0 = lo;
    end = hi;
    if (e == g.groups) k1 = 0;  // rows past the last group: zeros
  } else {
    // Splits, then groups, then tiles.
    const int e_split = b / tiles;
    b -= e_split * tiles;
    split = e_split / g.groups;
    e = e_split - split * g.groups;
    stripe(xcd_place(b, tiles), g.tiles_m, g.tiles_n, tm, tn);
    int64_t per = g.k_per;
    if (GK && g.offsets) {
      int lo, hi;
      group_range(g.offsets, g.groups, g.k, e, lo, hi);
      k0 = lo;
      k1 = hi;
      per = ((hi - lo + g.splits - 1) / g.splits + 63) / 64 * 64;
    }
    if (g.splits > 1) {
      k0 += split * per;
      k1 = min(k0 + per, k1);
    }
    row0 = (int64_t)tm * BM;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  const int rows_a = (int)min((int64_t)BM, end - row0), rows_b = (int)min((int64_t)BN, g.n - (int64_t)tn * BN);
  const int64_t kk = max((int64_t)0, k1 - k0);
  const int nk = (int)((kk + BK - 1) / BK);
  PA pa;
  PB pb;
  {
    const int64_t ra = row0, cb = (int64_t)tn * BN;
    const T* A = static_cast<const T*>(g.a) + (TA ? k0 * g.lda + ra : ra * g.lda + k0);
    const T* B = static_cast<const T*>(g.b) + (GK || k1 == 0 ? 0 : e * g.sb) + (TB ? k0 * g.ldb + cb : cb * g.ldb + k0);
    pa.init(reinterpret_cast<const char*>(A), g.lda * (int64_t)sizeof(T), rows_a, wave, lane);
    pb.init(reinterpret_cast<const char*>(B), g.ldb * (int64_t)sizeof(T), rows_b, wave, lane);
  }

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{};

  // float32: the accumulators are emptied into a second set every 512 of the
  // contraction, so that rounding grows with 512 + K / 512 additions, not with K
  // (a dW over 12000 rows is 4e-7 off its float64 value).
  constexpr bool TWO = sizeof(T) == 4;
  f32x4_t total[TWO ? FM : 1][TWO ? FN : 1] = {};
  auto empty = [&] __attribute__((always_inline)) {
    if constexpr (TWO) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          total[i][j] += acc[i][j];
          acc[i][j] = f32x4_t{};
        }
    }
  };

  // A wave whose rows or columns all lie outside C multiplies nothing.
  const bool idle = wm * WM >= rows_a || wn * WN >= rows_b;

  // Fragments of two substeps: one being read while the other is multiplied.
  Frag af[2][FM] = {}, bf[2][FN] = {};
  auto read = [&](const char* st, int s) __attribute__((always_inline)) {
    af[s & 1][0] = PA::frag(st, wm * WM, s, lane);
#pragma unroll
    for (int j = 0; j < FN; ++j) bf[s & 1][j] = PB::frag(st + PA::BYTES, wn * WN + 16 * j, s, lane);
#pragma unroll
    for (int i = 1; i < FM; ++i) af[s & 1][i] = PA::frag(st, wm * WM + 16 * i, s, lane);
  };
  auto multiply = [&](int s) __attribute__((always_inline)) {
    // A block's steps (four of float32) are apart by all the others: a product
    // that waits for the one before it in its accumulator would idle the unit.
#pragma unroll
    for (int q = 0; q < Mma<T>::N; ++q)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = Mma<T>::mul(bf[s & 1][j], af[s & 1][i], acc[i][j], q);
  };

  if constexpr (DIRECT) {
    constexpr int L = PA::LI + PB::LI;
    char* stages = lds + set * NS * STAGE;
    const int its = (nk + WGK - 1) / WGK;  // slices of a set (those past the end are zeros)
    auto issue = [&](int it, char* fill) __attribute__((always_inline)) {
      const int kt = it * WGK + set;
      const int k_left = (int)max((int64_t)0, min((int64_t)BK, kk - (int64_t)kt * BK));
      pa.issue(kt, k_left, fill, wave, lane);
      pb.issue(kt, k_left, fill + PA::BYTES, wave, lane);
    };
    if (nk > 0) {
#pragma unroll
      for (int p = 0; p < NS - 1; ++p) issue(p, stages + p * STAGE);
    }
    auto run = [&](auto idle_tag) __attribute__((always_inline)) {
      constexpr bool IDLE = decltype(idle_tag)::value;
      int stage = 0;
      for (int kt = 0; kt < its; ++kt) {
        // Slices kt + 1 .. kt + NS - 2 stay in flight; the barrier then says that
        // slice kt is whole and that slice kt - 1 has been read by all.
        static_assert((NS - 2) * L < 64, "waits");
        wait_loads<(NS - 2) * L>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        // The stage being filled and the one being read are never the same:
        // __restrict says so, or the compiler would wait for the loads in
        // flight ahead of every transposing read.
        auto step = [&](char* __restrict fill, const char* __restrict st) __attribute__((always_inline)) {
          issue(kt + NS - 1, fill);
          if constexpr (IDLE) return;
          // A slice's last substep is multiplied behind the next barrier, so the
          // matrix cores have work while the first fragments are read.  (Ahead of
          // the first slice these are products of zeros.)
          constexpr int RD = PA::READS * FM + PB::READS * FN, MM = FM * FN * Mma<T>::N;
#pragma unroll
          for (int s = 0; s < SUB; ++s) {
            read(st, s);
            multiply(s + 1);  // of the other parity: substep s - 1
            // The loads go out over the first half of the substep's products: at 8192^3
            // on one card 1416 / 1419 / 1411 TFLOP/s (forward, dx, dW) against 1388 /
            // 1392 / 1345 over all of them and 1407 / 1371 / 1406 over the first quarter.
            if (s == 0) interleave<RD, L, MM / 2, MM>();
            else interleave<RD, 0, 1, MM>();
          }
        };
        if (TWO && (kt & 15) == 15) empty();
        step(stages + (stage == 0 ? NS - 1 : stage - 1) * STAGE, stages + stage * STAGE);
        stage = stage == NS - 1 ? 0 : stage + 1;
      }
      if (!IDLE && nk > 0) multiply(SUB - 1);
    };
    if (NW == 8 && idle) run(std::true_type{});
    else run(std::false_type{});
    wait_loads<0>();
  } else {
    auto fetch = [&](int kt, int q) __attribute__((always_inline)) {
      const int k_left = (int)min((int64_t)BK, kk - (int64_t)kt * BK);
      pa.fetch(kt, k_left, q, wave, lane);
      pb.fetch(kt, k_left, q, wave, lane);
    };
#pragma unroll
    for (int q = 0; q < PD; ++q)
      if (q < nk) fetch(q, q);
    for (int k0t = 0; k0t < nk; k0t += PD) {
#pragma unroll
      for (int q = 0; q < PD; ++q) {
        const int kt = k0t + q;
        if (kt >= nk) break;
        char* st = lds + (q & 1) * STAGE;  // last read at slice kt - 2, a barrier ago
        pa.put(st, q, wave, lane);
        pb.put(st + PA::BYTES, q, wave, lane);
        if (kt + PD < nk) fetch(kt + PD, q);
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt 0: this wave's part is in LDS; loads stay in flight
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (TWO && (kt & 15) == 15) empty();
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
          read(st, s);
          multiply(s);
        }
      }
    }
  }
  if constexpr (TWO) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] += total[i][j];
  }
  __syncthreads();  // every wave is done with the operand stages

  // ---- epilogue: 32 rows at a time through this wave's own staging, so that
  // a row of C leaves as whole 16-byte pieces.  The products are of B by A, so a
  // block's register u in a lane is row lane mod 16 and column 4 (lane / 16) + u:
  // four columns of a row, one 16-byte write.
  constexpr int LPR = WN / 8, RPP = 64 / LPR;
  char* stg = lds + wave_all * 32 * STRIDE;
  const int col = tn * BN + wn * WN + 8 * (lane % LPR);
  const int n_in = (int)min((int64_t)8, g.n - col);
  float bias[8] = {};
  if (g.bias && n_in > 0 && !g.part && !(!GK && e == g.groups && g.offsets))
    load8(static_cast<const T*>(g.bias) + (GK ? 0 : e * g.sbias) + col, n_in, bias);
  // Where n is a multiple of 8 every piece is whole: no branch between the loads and
  // stores of a strip.
  auto strips = [&](auto full_tag) __attribute__((always_inline)) {
    const int n = decltype(full_tag)::value ? 8 : n_in;
#pragma unroll
    for (int i = 0; i < WM / 32; ++i) {
#pragma unroll
      for (int ii = 0; ii < 2; ++ii)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          *reinterpret_cast<f32x4_t*>(stg + (16 * ii + (lane & 15)) * STRIDE + (16 * j + 4 * (lane >> 4)) * 4) =
              acc[2 * i + ii][j];
      if constexpr (WGK > 1) __syncthreads();
      else wave_fence();
      // One wave reads its strip back; with several sets, each set takes its share
      // of the 32 rows and adds the sets' values in order.
      constexpr int ROWS = 32 / WGK;
#pragma unroll
      for (int p = 0; p < (ROWS + RPP - 1) / RPP; ++p) {
        const int pr = p * RPP + lane / LPR, lr = set * ROWS + pr;
        float v[8] = {};
#pragma unroll
        for (int q = 0; q < WGK; ++q) {
          const char* from = WGK == 1 ? stg : lds + (q * NW + wave) * 32 * STRIDE;
          const f32x4_t* src = reinterpret_cast<const f32x4_t*>(from + min(lr, 31) * STRIDE + (lane % LPR) * 32);
          const f32x4_t x = src[0], y = src[1];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            v[c] += x[c];
            v[4 + c] += y[c];
          }
        }
        const int64_t row = row0 + wm * WM + 32 * i + lr;
        if (pr < ROWS && row < end && n_in > 0) {
          if (g.part) store8(g.part + (((int64_t)split * (GK ? g.groups : 1) + (GK ? e : 0)) * g.m + row) * g.n + col, n, v);
          else finish8<T>(g, v, bias, GK ? e : 0, row, col, n);
        }
      }
      if constexpr (WGK == 1) wave_fence();
    }
  };
  if ((g.n & 7) == 0) strips(std::true_type{});
  else strips(std::false_type{});
}

// Joins a split contraction: the partials of an entry are added in split
// order, then the epilogue runs as in the kernel above.  The groups' results
// lie one behind the other, as rows of one matrix.  Of a pair of rows, what the
// second holds corrects the first's last digits.  Where the first is not finite (an
// infinite operand, say) there is nothing to correct, and the second, whose
// infinities need not have the first's sign, would turn it into NaN.
template <typename T>
__global__ __launch_bounds__(256) void k_gemm_join(GemmArgs g) {
  const int64_t per = (g.n + 7) / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x, rows = g.m * g.groups;
  if (i >= per * rows) return;
  const int64_t row = i / per;
  const int col = (int)(i - row * per) * 8, n = (int)min((int64_t)8, g.n - col);
  float v[8] = {}, rest[8] = {}, bias[8] = {};
  for (int s = 0; s < g.splits; ++s) {
    float p[8];
    const bool second = g.pairs && (s & 1);
    const int64_t at = g.pairs ? 2 * ((s >> 1) * rows + row) + (s & 1) : s * rows + row;
    load8(g.part + at * g.n + col, n, p);
#pragma unroll
    for (int k = 0; k < 8; ++k) (second ? rest[k] : v[k]) += p[k];
  }
  if (g.pairs) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (fabsf(v[k]) < __builtin_huge_valf()) v[k] += rest[k];
  }
  if (g.bias) load8(static_cast<const T*>(g.bias) + col, n, bias);
  finish8<T>(g, v, bias, 0, row, col, n);
}

template <typename T, int BM, int BN, int WGM, int WGN, int WGK, int NS, int LOADS>
hipError_t launch_tile(const GemmArgs& g, bool ta, bool tb, hipStream_t s) {
  const int64_t tiles = (int64_t)g.tiles_m * g.tiles_n;
  const int64_t blocks = tiles * g.splits * (ta && tb && g.offsets ? g.groups : 1);
  if (blocks <= 0) return hipSuccess;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(64 * WGM * WGN * WGK);
  if (ta && tb) hipLaunchKernelGGL((k_gemm<T, BM, BN, WGM, WGN, WGK, NS, true, true, LOADS>), grid, block, 0, s, g);
  else if (tb) hipLaunchKernelGGL((k_gemm<T, BM, BN, WGM, WGN, WGK, NS, false, true, LOADS>), grid, block, 0, s, g);
  else if (!ta) hipLaunchKernelGGL((k_gemm<T, BM, BN, WGM, WGN, WGK, NS, false, false, LOADS>), grid, block, 0, s, g);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace
}  // namespace muon
