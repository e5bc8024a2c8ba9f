// Tiled bf16 kernels: a product cut into slices of K, for the cross entropy's input gradient.
#include "linear_tiles.h"

namespace tpshard {
namespace {

template <bool WT>
hipError_t slices(const LinGemm& p, const TilePick& t, hipStream_t s) {
  switch (t.tile) {
    case kTile256: return launch_lin_pps<256, 256, kModeSlices, false, WT>(p, s, t.splits);
    case kTile128w: return launch_lin_pps<256, 128, kModeSlices, false, WT, WT ? 4 : 2>(p, s, t.splits);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t lin_tiles_slices(const LinGemm& p, const TilePick& t, hipStream_t s) {
  return p.w_t ? slices<true>(p, t, s) : slices<false>(p, t, s);
}

}  // namespace tpshard
