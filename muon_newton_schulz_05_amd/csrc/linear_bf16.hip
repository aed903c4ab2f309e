// linear_bf16.hip -- the bfloat16 products of the layer operators.
#include "gemm.h"

namespace muon {

hipError_t launch_gemm_bf16(const GemmArgs& g, bool ta, bool tb, bool direct, int tile, hipStream_t s) {
  if (!direct) {
    if (tile == kTile64) return launch_tile<uint16_t, 64, 64, 2, 2, 2, false, 1>(g, ta, tb, s);
    return launch_tile<uint16_t, 128, 128, 2, 2, 2, false, 1>(g, ta, tb, s);
  }
  switch (tile) {
    case kTile256: return launch_tile<uint16_t, 256, 256, 2, 4, 2, true, 1>(g, ta, tb, s);
    case kTile256x128: return launch_tile<uint16_t, 256, 128, 4, 2, 3, true, 1>(g, ta, tb, s);
    case kTile64: return launch_tile<uint16_t, 64, 64, 2, 2, 2, true, 1>(g, ta, tb, s);
    case kTileRows32: return launch_tile<uint16_t, 32, 128, 1, 4, 4, true, 1>(g, ta, tb, s);
    default: return launch_tile<uint16_t, 128, 128, 2, 2, 2, true, 1>(g, ta, tb, s);
  }
}

}  // namespace muon
