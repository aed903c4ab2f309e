// norm.h -- launchers of the norms (include/muon_block.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

struct NormArgs {
  const void* x;
  const void* res;   // null: s is x
  const void* w;     // null: ones
  const void* b;     // null: zeros
  void* y;
  void* s;           // x + res, where res is given
  float* stats;      // null, or [rows][2]: mean and 1 / sqrt(var + eps)
  int64_t rows, cols, ldx, ldr;
  float eps;
  int32_t layer;     // 0: the root-mean-square norm
};
struct NormGradArgs {
  const void* dy;
  const void* x;
  const void* res;   // null: s is x
  const void* w;
  const void* ds;    // null, or what reaches s by other ways
  const float* stats;
  void* dx;          // each null where not wanted
  void* dw;
  void* db;
  float* part;       // [norm_parts][2][cols], where dw or db is wanted
  int64_t rows, cols, ldg, ldx, ldr, ldd;
  int32_t layer;
};
int64_t norm_parts(int64_t rows, int64_t cols);  // rows of partial sums
hipError_t launch_norm(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_norm_grad(const NormGradArgs& a, int dtype, hipStream_t s);

}  // namespace muon
