// dropout.hip -- dropout from a counter-based generator.
//
// The generator is Philox4x32 with 10 rounds (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011): the 128-bit counter is
// (block, offset), the key is the seed.  Elements 8 b .. 8 b + 7 take the
// eight 16-bit lanes of block b, so the mask follows from the element's
// flat index alone and the gradient makes it again instead of storing it.
//
// Bound by memory: [16384, 4096] in bf16 takes 108 - 117 us forward with a residual and
// backward together, 5.7 - 6.2 TB/s.  One generator call serves eight elements
// (16 bits each, so probabilities go in steps of 2^-16); with 32 bits an element
// its 20 wide multiplications a call would take as long as the memory.
#include "act.h"
#include "device_common.h"
#include "ops.h"

namespace muon {
namespace {

__device__ __forceinline__ u32x4_t philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4_t{c0, c1, c2, c3};
}

template <typename T, bool FULL>
__global__ __launch_bounds__(256) void k_dropout(DropoutArgs a) {
  const int64_t blk = (int64_t)blockIdx.x * 256 + threadIdx.x, i0 = blk * 8;
  if (i0 >= a.n) return;
  const int n = FULL ? 8 : (int)min((int64_t)8, a.n - i0);
  const uint64_t seed = a.state ? a.state[0] : a.seed, offset = a.state ? a.state[1] : a.offset;
  float v[8], r[8] = {};
  load8(static_cast<const T*>(a.x) + i0, n, v);
  if (a.res) load8(static_cast<const T*>(a.res) + i0, n, r);
  const u32x4_t w = philox((uint64_t)blk, offset, seed);
  const float scale = 65536.f / (float)(65536u - a.drop);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
    // A dropped element is zero whatever it held, infinities and NaN too.
    v[i] = (u >= a.drop ? v[i] * scale : 0.f) + r[i];
  }
  store8(static_cast<T*>(a.y) + i0, n, v);
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, int dtype, hipStream_t s) {
  const int64_t blocks = ((a.n + 7) / 8 + 255) / 256;
  if (blocks <= 0) return hipSuccess;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  const bool full = a.n % 8 == 0;
  const dim3 grid((unsigned)blocks), block(256);
  if (dtype == MUON_BF16 && full) hipLaunchKernelGGL((k_dropout<uint16_t, true>), grid, block, 0, s, a);
  else if (dtype == MUON_BF16) hipLaunchKernelGGL((k_dropout<uint16_t, false>), grid, block, 0, s, a);
  else if (full) hipLaunchKernelGGL((k_dropout<float, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_dropout<float, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace muon
