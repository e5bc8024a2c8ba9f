// Tiled bf16 kernels: logits computed again and turned into the loss's gradient at them.
// Bound by MFMA: 8192 x 4096 -> 32768 1620 to 1700 us (1.3 PFLOP/s; 512 MiB leave in it).
#include "linear_tiles.h"

namespace tpshard {

hipError_t lin_tiles_prob(const CeGemm& p, const TilePick& t, hipStream_t s) {
  return p.w_t ? dispatch_tiles<kModeProb, false, true>(p, t, s) : dispatch_tiles<kModeProb, false, false>(p, t, s);
}

}  // namespace tpshard
