// Which kernel a product of the linear layer or the gated block runs on.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "linear.h"

namespace tpshard {

namespace {

bool aligned(const void *p, int64_t ld, int64_t es, int64_t elems) {
  return !p || (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(elems * es) == 0 && ld % elems == 0);
}

}  // namespace

bool lin_tiles_ok(const LinGemm& p) {
  if (p.f32 || p.K <= 0 || p.K % 32) return false;
  if (!aligned(p.a, p.lda, 2, 8) || !aligned(p.a2, p.lda, 2, 8) || !aligned(p.w, p.ldw, 2, 8) || !aligned(p.w2, p.ldw, 2, 8))
    return false;
  return (!p.a_t || p.M % 8 == 0) && (p.w_t || p.N % 8 == 0);
}

namespace {

constexpr int64_t kCUs = 256;

// The small tile: 64 rows by 64 columns (of each weight).
int64_t small_tiles(const LinGemm& p) { return lin_tiles_count(p, 64, p.mode == kModeDual ? 128 : 64); }

// The tile: waves of workgroups over the CUs times the tile's work over its
// relative throughput (measured in gemm.hip).  Problems too small to give every
// CU a 128 x 128 tile take small ones, several of which share a CU: with three
// stages in flight (2048 -> 4096 at 256 rows 12.7 us against 17.4 with two; gated
// 12288 -> 6144 160 against 173, and 199 with four), or two where a workgroup has
// at most 16 (1024^3 9.0 us against 10.3).  They split K until there is one for
// every CU, and on to two where each still has 24 stages to pay for the join
// (gated 4096 -> 2048 at 64 rows: 40 -> 17 us; at 8 stages each the second split
// cost 25 -> 31 us at 128 rows).
TilePick pick(const LinGemm& p) {
  const bool dual = p.mode == kModeDual, k64 = p.K % 64 == 0;
  if (lin_tiles_count(p, 128, 128) < kCUs) {
    TilePick t{k64 ? kTile64 : kTile64k32, 1};
    const int64_t tiles = small_tiles(p), stages = p.K / (k64 ? 64 : 32) * (p.mode == kModeCat ? 2 : 1);
    while (t.splits < 16 && stages >= 2 * t.splits * 8 &&
           (tiles * t.splits < kCUs || (tiles * t.splits < 2 * kCUs && stages >= 2 * t.splits * 24)))
      t.splits *= 2;
    if (k64 && stages <= 16 * t.splits) t.tile = kTile64short;
    return t;
  }
  auto cost = [&](int bm, int bn, double eff) {
    return static_cast<double>((lin_tiles_count(p, bm, bn) + kCUs - 1) / kCUs) * bm * bn / eff;
  };
  const int64_t a_span = (p.a_t ? p.K : p.M) * p.lda * 2, w_span = (p.w_t ? p.N : p.K) * p.ldw * 2;
  const bool pps = k64 && a_span < (int64_t{1} << 31) && w_span < (int64_t{1} << 31);
  const double c256 = !p.a_t && pps ? cost(256, 256, 1.0) : 1e300, c192 = !dual && pps ? cost(256, 192, 0.95) : 1e300;
  const double c128w = pps ? cost(256, 128, 0.85) : 1e300, c128 = cost(128, 128, 0.7);
  const double best = std::min(std::min(c256, c192), std::min(c128w, c128));
  return {c256 == best ? kTile256 : c192 == best ? kTile192 : c128w == best ? kTile128w : kTile128, 1};
}

int64_t ws_of(const LinGemm& p, const TilePick& t) {
  if (t.splits < 2) return 0;
  const int64_t tiles = small_tiles(p);
  return kTicketBytes + tiles * t.splits * 64 * (p.mode == kModeDual ? 128 : 64) * 4;
}

// Whether few rows run on their own kernel: always where the tiled ones cannot,
// and up to 32 rows (16 < M with a weight of under 100 MB: 2048 -> 4096 at 32 rows
// 8.8 us against 12.9, but 6144 -> 12288 56 against 43, each row group reading
// its activations again).
bool takes_rows(const LinGemm& p) {
  if (!lin_rows_ok(p)) return false;
  if (p.M <= 16 || !lin_tiles_ok(p)) return true;
  return p.M <= 32 && (p.mode == kModeDual ? 2 : 1) * p.N * p.K < 50'000'000;
}

hipError_t launch_tiles(LinGemm p, void *ws, int64_t ws_bytes, hipStream_t s) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  TilePick t = pick(p);
  if (!ws || ws_bytes < ws_of(p, t)) t.splits = 1;
  if (t.splits > 1) {
    p.tickets = static_cast<uint32_t *>(ws);
    p.join = reinterpret_cast<float *>(static_cast<char *>(ws) + kTicketBytes);
  }
  if (p.a_t) return lin_tiles_pair(p, t, s);
  switch (p.mode) {
    case kModeOne: return lin_tiles_one(p, t, s);
    case kModeDual: return lin_tiles_dual(p, t, s);
    case kModeCat: return lin_tiles_cat(p, t, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

// (Asked before the strides are known: enough for either kernel.)
int64_t lin_gemm_ws(const LinGemm& p) {
  if (p.M <= 0 || p.N <= 0) return 0;
  if (takes_rows(p)) return lin_rows_ws(p);
  return std::max(lin_tiles_ok(p) ? ws_of(p, pick(p)) : 0, lin_staged_ws(p));
}

hipError_t lin_gemm_launch(LinGemm p, hipStream_t s, void *ws, int64_t ws_bytes) {
  if (takes_rows(p)) return lin_rows_launch(p, ws, ws_bytes, s);
  if (lin_tiles_ok(p)) return launch_tiles(p, ws, ws_bytes, s);
  return lin_staged_launch(p, ws, ws_bytes, s);
}

}  // namespace tpshard
