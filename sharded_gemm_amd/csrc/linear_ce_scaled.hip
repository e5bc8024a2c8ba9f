// Tiled bf16 kernels: the cross entropy's gradients, but for a weight's that lies k-contiguous.
// Bound by MFMA: dX of 8192 x 32768 -> 4096 1405 us (1.56 PFLOP/s).
#include "linear_tiles.h"

namespace tpshard {

hipError_t lin_tiles_scaled(const ScaledGemm& p, const TilePick& t, hipStream_t s) {
  return p.w_t ? dispatch_tiles<kModeScaled, false, true>(p, t, s) : dispatch_tiles<kModeScaled, false, false>(p, t, s);
}

}  // namespace tpshard
