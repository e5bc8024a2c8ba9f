// Tiled bf16 kernels: a weight gradient whose second operand lies k-contiguous.
#include "linear_tiles.h"

namespace tpshard {

hipError_t lin_tiles_wgrad(const LinGemm& p, const TilePick& t, hipStream_t s) {
  return dispatch_tiles<kModeOne, true, true>(p, t, s);
}

}  // namespace tpshard
