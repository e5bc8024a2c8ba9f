// Tiled bf16 kernels: the cross entropy's weight gradient, whose second operand lies k-contiguous
// (X transposed).  Only the first goes through the transposing LDS read, and a 256 x 256 tile has the
// registers for that: 32768 x 8192 -> 4096 1564 us (1.41 PFLOP/s), in 256 x 128 tiles 1735.
#include "linear_tiles.h"

namespace tpshard {

hipError_t lin_tiles_wgrad(const ScaledGemm& p, const TilePick& t, hipStream_t s) {
  return dispatch_tiles<kModeScaled, true, true>(p, t, s);
}

}  // namespace tpshard
