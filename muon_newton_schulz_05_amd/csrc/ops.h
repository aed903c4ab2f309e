// ops.h -- launchers of the layer operators' kernels (include/muon_ops.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/muon_ops.h"

namespace muon {

// One (grouped) matrix product C[i][j] = sum_k A[i][k] B[j][k].
//  ta / tb = 0: the operand's rows are contiguous along k (element (r, k) at
//  r ld + k); 1: contiguous along its rows (element at k ld + r).
// Rows grouped (offsets set, not ta && tb): rows offsets[e] .. offsets[e + 1]
// of A and C belong to expert e and meet B + e sb; rows past offsets[groups]
// give zero.  Contraction grouped (ta && tb): expert e's product runs over
// k = offsets[e] .. offsets[e + 1] and goes to C + e sc.
struct GemmArgs {
  const void* a;
  const void* b;
  int64_t lda, ldb, sb;
  int64_t m, n, k;
  const int32_t* offsets;  // null: one group
  int32_t groups;          // 1 without offsets
  // epilogue: z = C + bias; y = act(z) + res
  void* c;
  void* z;                 // null, or where z is stored (rows of ldc elements)
  const void* bias;        // null, or [groups][n]
  const void* res;         // null, or rows of ldr elements
  int64_t ldc, sc, ldr, sbias;
  int32_t act;
  // split contraction: part != null stores float32 partials [splits][groups][m][n]
  float* part;
  int32_t splits;
  int64_t k_per;           // contraction of one split (a multiple of 64); a grouped
                           // contraction's splits go by each group's length
  int32_t tiles_m, tiles_n;
  int32_t pairs;           // join: row r of the result is row 2r and, where that is finite, row 2r + 1
};

enum GemmTile { kTile128 = 0, kTile256, kTile256x128, kTile64, kTile32x64, kTileRows32, kTileRows32K };
int gemm_tile_m(int tile);
int gemm_tile_n(int tile);
// How operands reach LDS: through registers (any alignment), or directly by
// aligned pieces of 16 or of 4 bytes a lane.
enum GemmLoads { kStaged = 0, kDirect16, kDirect4 };
hipError_t launch_gemm(const GemmArgs& g, int dtype, bool ta, bool tb, int loads, int tile, hipStream_t s);
hipError_t launch_gemm_bf16(const GemmArgs& g, bool ta, bool tb, int loads, int tile, hipStream_t s);
hipError_t launch_gemm_f32(const GemmArgs& g, bool ta, bool tb, int loads, int tile, hipStream_t s);
// dst[g][r][0 .. ld) = src[g][r][0 .. cols) with zeros behind: a bf16 operand laid
// out for 16-byte loads.  ld is cols rounded up to 8; one group's dst follows another's.
// pairs: odd rows of dst take zeros where src is not finite.
struct AlignArgs {
  const void* src;
  void* dst;
  int64_t rows, cols, src_ld, src_step, ld;  // src_step: from one group to the next
  int32_t groups, pairs;
};
hipError_t launch_align(const AlignArgs& a, hipStream_t s);
hipError_t launch_gemm_join(const GemmArgs& g, int dtype, hipStream_t s);

// dz = dy act'(z) and the column sums of dz over each group's rows.
struct ActGradArgs {
  const void* dy;
  const void* z;           // null: act'(z) = 1
  void* dz;                // null: not stored
  void* db;                // null, or [groups][n]
  float* part;             // column sums of one row block, [blocks][n]
  int64_t rows, n, lddy, ldz, lddz;
  const int32_t* offsets;
  int32_t groups, act;
  int32_t block;           // rows of one block (launch_act_grad sets it)
  int32_t pairs;           // bf16: dz rounded in row 2r of dz, and what that lost in row 2r + 1
  int32_t* offsets2;       // pairs of grouped rows: where the offsets of dz's rows go
};
int64_t act_grad_blocks(int64_t rows, int64_t n, int32_t groups, bool grouped);
hipError_t launch_act_grad(const ActGradArgs& a, int dtype, hipStream_t s);

// Most row blocks that `rows` rows in up to `groups` groups (and the rows
// past the last one) can fill.
inline int64_t group_blocks(int64_t rows, int64_t groups, bool grouped, int64_t block) {
  if (!grouped) return (rows + block - 1) / block;
  const int64_t most = rows / block + groups + 1;
  return most < rows ? most : rows;
}

struct RouteArgs {
  const void* ids;
  int32_t ids64, experts, top;
  int64_t entries;
  int32_t* order;
  int32_t* position;
  int32_t* offsets;
  int32_t* hist;           // workspace [blocks][experts]
};
constexpr int kRouteBlock = 2048;   // entries of one block
constexpr int kRouteMaxExperts = 1024;
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

struct MoveArgs {
  const void* x;           // dispatch: x; dispatch gradient: dxs; combine: ys
  const void* g;           // combine gradient: dy
  const void* res;         // combine: residual or null
  void* out;               // xs, dx, y, or dys
  float* dw;               // combine gradient: dweights or null
  const float* w;          // weights [tokens][top]
  const int32_t* position;
  const int32_t* offsets;
  int32_t experts, top;
  int64_t tokens, h, ldx, ldg, ldr;
};
hipError_t launch_dispatch(const MoveArgs& a, int dtype, hipStream_t s);
hipError_t launch_gather_sum(const MoveArgs& a, int dtype, hipStream_t s);
hipError_t launch_combine_grad(const MoveArgs& a, int dtype, hipStream_t s);

struct DropoutArgs {
  const void* x;
  const void* res;
  void* y;
  int64_t n;
  uint64_t seed, offset;
  const uint64_t* state;   // null, or {seed, offset} on the device
  uint32_t drop;           // of 65536
};
hipError_t launch_dropout(const DropoutArgs& a, int dtype, hipStream_t s);

}  // namespace muon
