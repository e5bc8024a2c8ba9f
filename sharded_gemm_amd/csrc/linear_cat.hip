// Tiled bf16 kernels: the gated block's input gradient, one accumulator over both weights.
#include "linear_tiles.h"

namespace tpshard {

hipError_t lin_tiles_cat(const LinGemm& p, const TilePick& t, hipStream_t s) {
  return p.w_t ? dispatch_tiles<kModeCat, false, true>(p, t, s) : dispatch_tiles<kModeCat, false, false>(p, t, s);
}

}  // namespace tpshard
