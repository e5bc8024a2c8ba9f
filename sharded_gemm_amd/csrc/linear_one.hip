// Tiled bf16 kernels: the linear layer's product and its epilogue.
#include "linear_tiles.h"

namespace tpshard {

hipError_t lin_tiles_one(const LinGemm& p, const TilePick& t, hipStream_t s) {
  return p.w_t ? dispatch_tiles<kModeOne, false, true>(p, t, s) : dispatch_tiles<kModeOne, false, false>(p, t, s);
}

}  // namespace tpshard
