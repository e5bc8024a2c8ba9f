// Tiled bf16 kernels: logits reduced to each tile's row statistics.
#include "linear_tiles.h"

namespace tpshard {

hipError_t lin_tiles_stats(const CeGemm& p, const TilePick& t, hipStream_t s) {
  return p.w_t ? dispatch_tiles<kModeStats, false, true>(p, t, s) : dispatch_tiles<kModeStats, false, false>(p, t, s);
}

}  // namespace tpshard
