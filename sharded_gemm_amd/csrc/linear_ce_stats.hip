// Tiled bf16 kernels: logits reduced to each tile's row statistics.
//
// Many rows: bound by MFMA, 8192 x 4096 -> 16384 770 us (1.43 PFLOP/s); where K is short by the
// epilogue too, 4096 x 768 -> 50000 304 (1.03).  Few: by the weight's bytes, 24 x 4096 -> 65536 100
// (5.4 TB/s), 1 x 768 -> 32000 10.
#include "linear_tiles.h"

namespace tpshard {

hipError_t lin_tiles_stats(const CeGemm& p, const TilePick& t, hipStream_t s) {
  return p.w_t ? dispatch_tiles<kModeStats, false, true>(p, t, s) : dispatch_tiles<kModeStats, false, false>(p, t, s);
}

}  // namespace tpshard
