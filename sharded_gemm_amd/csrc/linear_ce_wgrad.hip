// Tiled bf16 kernels: the cross entropy's weight gradient, whose second operand lies k-contiguous.
#include "linear_tiles.h"

namespace tpshard {

hipError_t lin_tiles_wgrad(const ScaledGemm& p, const TilePick& t, hipStream_t s) {
  return dispatch_tiles<kModeScaled, true, true>(p, t, s);
}

}  // namespace tpshard
