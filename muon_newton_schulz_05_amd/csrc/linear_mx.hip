// linear_mx.hip -- the products of the layers held in four bits.
#include "gemm.h"
#include "mx.h"

namespace muon {

namespace {
// The bf16 tiles; 32 x 128 has a stage less, so that two workgroups still share a unit's LDS beside the scales.
template <typename O>
hipError_t launch(const GemmArgs& g, int tile, hipStream_t s) {
  switch (tile) {
    case kTile256: return launch_tile<Mx4<O>, 256, 256, 2, 4, 1, 2, kDirect16>(g, false, false, s);
    case kTile256x128: return launch_tile<Mx4<O>, 256, 128, 4, 2, 1, 3, kDirect16>(g, false, false, s);
    case kTile64: return launch_tile<Mx4<O>, 64, 64, 2, 2, 1, 4, kDirect16>(g, false, false, s);
    case kTileRows32: return launch_tile<Mx4<O>, 32, 128, 1, 4, 1, 3, kDirect16>(g, false, false, s);
    case kTileRows32K: return launch_tile<Mx4<O>, 32, 64, 1, 2, 4, 3, kDirect16>(g, false, false, s);
    default: return launch_tile<Mx4<O>, 128, 128, 2, 2, 1, 2, kDirect16>(g, false, false, s);
  }
}
}  // namespace

hipError_t launch_gemm_mx(const GemmArgs& g, int dtype, int tile, hipStream_t s) {
  return dtype == MUON_BF16 ? launch<uint16_t>(g, tile, s) : launch<float>(g, tile, s);
}

}  // namespace muon
