// linear_bf16.hip -- the bfloat16 products of the layer operators.
#include "gemm.h"

namespace muon {

hipError_t launch_gemm_bf16(const GemmArgs& g, bool ta, bool tb, int loads, int tile, hipStream_t s) {
  if (loads == kDirect4) return launch_tile<uint16_t, 64, 64, 2, 2, 1, 4, kDirect4>(g, ta, tb, s);
  if (loads == kStaged) return launch_tile<uint16_t, 64, 64, 2, 2, 1, 2, kStaged>(g, ta, tb, s);
  switch (tile) {
    case kTile256: return launch_tile<uint16_t, 256, 256, 2, 4, 1, 2, kDirect16>(g, ta, tb, s);
    case kTile256x128: return launch_tile<uint16_t, 256, 128, 4, 2, 1, 3, kDirect16>(g, ta, tb, s);
    case kTile64: return launch_tile<uint16_t, 64, 64, 2, 2, 1, 4, kDirect16>(g, ta, tb, s);
    case kTileRows32: return launch_tile<uint16_t, 32, 128, 1, 4, 1, 4, kDirect16>(g, ta, tb, s);
    case kTileRows32K: return launch_tile<uint16_t, 32, 64, 1, 2, 4, 3, kDirect16>(g, ta, tb, s);
    default: return launch_tile<uint16_t, 128, 128, 2, 2, 1, 2, kDirect16>(g, ta, tb, s);
  }
}

}  // namespace muon
