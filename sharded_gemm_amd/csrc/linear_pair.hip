// Tiled bf16 kernels: weight gradients: one product, or the gated block's two in one launch.
#include "linear_tiles.h"

namespace tpshard {

hipError_t lin_tiles_pair(const LinGemm& p, const TilePick& t, hipStream_t s) {
  return dispatch_tiles<kModePair, true, false>(p, t, s);
}

}  // namespace tpshard
