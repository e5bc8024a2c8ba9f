// Tiled bf16 kernels: the gated block's two projections, activation and product.
#include "linear_tiles.h"

namespace tpshard {

hipError_t lin_tiles_dual(const LinGemm& p, const TilePick& t, hipStream_t s) {
  return p.w_t ? dispatch_tiles<kModeDual, false, true>(p, t, s) : dispatch_tiles<kModeDual, false, false>(p, t, s);
}

}  // namespace tpshard
