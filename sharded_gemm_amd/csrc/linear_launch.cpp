// Which kernel a product of the linear layer or the gated block runs on, its tiles
// and its workspace.  Host code only: what a launch reads and writes can be checked
// without a GPU.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "linear.h"

namespace tpshard {

namespace {

bool aligned(const void *p, int64_t ld, int64_t es, int64_t elems) {
  return !p || (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(elems * es) == 0 && ld % elems == 0);
}

// Whether the tiled bf16 kernels take it.
bool tiles_ok(const LinGemm& p) {
  if (p.f32 || p.K <= 0 || p.K % 32) return false;
  if (!aligned(p.a, p.lda, 2, 8) || !aligned(p.a2, p.lda, 2, 8) || !aligned(p.w, p.ldw, 2, 8) || !aligned(p.w2, p.ldw, 2, 8))
    return false;
  return (!p.a_t || p.M % 8 == 0) && (p.w_t || p.N % 8 == 0);
}

constexpr int64_t kCUs = 256;

// ---- few rows ----------------------------------------------------------------
// Up to 16 rows (one operand's worth); with a k-contiguous weight up to 64, since
// there more rows cost accumulators only (an n-contiguous one keeps four columns
// a lane, and their accumulators spill).
bool rows_ok(const LinGemm& p) {
  return p.M <= (p.w_t ? 64 : 16) && !p.a_t && p.K > 0 && (p.mode == kModeOne || p.mode == kModeDual) && !p.acc_c;
}

RowsShape rows_shape(const LinGemm& p) {
  const int es = p.f32 ? 4 : 2, mats = p.mode == kModeDual ? 2 : 1;
  RowsShape s;
  s.g = p.w_t ? 1 : 8 / es;
  const int tc = 16 * s.g;
  s.tiles = (p.N + tc - 1) / tc;
  s.cells = mats * p.M * tc;
  const int64_t steps = (p.K * es + 63) / 64;
  s.waves = kRowsWaves;
  while (s.waves > 1 && (s.waves * 2 > steps || s.waves * s.cells * 4 > 64 * 1024)) s.waves /= 2;
  // Workgroups of a tile: until every CU has one (a wave keeping two steps),
  // then up to two each where a workgroup still reads 256 KiB, which pays for
  // the join.  MI355X, one token: gated 12288 -> 6144 (k-contiguous) 65 us with
  // 384 workgroups, 55 with 768; 6144 -> 12288 (n-contiguous) 36 with 384, 31
  // with 768; but gated 4096 -> 2048 (131 KiB each at 256) 10.4 with 256, 11.7
  // with 512.
  s.splits = 1;
  static_assert(kMaxTickets >= 512, "a ticket for every tile that is split");
  while (s.splits < 16 && s.splits * 2 * s.waves * 2 <= steps) {
    const int64_t wgs = s.tiles * s.splits, each = static_cast<int64_t>(mats) * tc * es * p.K / s.splits;
    if (wgs >= 512 || (wgs >= 256 && each < 256 * 1024)) break;
    s.splits *= 2;
  }
  return s;
}

int64_t ws_of(const RowsShape& h) { return h.splits > 1 ? kTicketBytes + h.tiles * h.splits * h.cells * 4 : 0; }

// ---- any layout and size -------------------------------------------------------
// The tile's edge and the workgroups that split its K, by estimated time.  With
// k workgroups to the busiest CU a stage takes max(alone, k * shared) us, and
// joining S > 1 splits 2 us and 7 ns a workgroup (their partials' trip to memory
// and back).  The constants are fitted to MI355X times, e.g. (bf16 / fp32)
// 2049 x 2047 x 2049: edge 128 60 / 281 us, edge 64 71 / 194; 100 x 4097 x 2049: 29 / 88
// unsplit, 16 / 36 with three splits; 515 x 1021 x 1531: 13 / 28 unsplit, 20 / 32
// with four.
StagedShape staged_shape(const LinGemm& p, bool may_split) {
  const int64_t stages = (p.K * (p.f32 ? 4 : 2) + kStagedRow - 1) / kStagedRow * (p.mode == kModeCat ? 2 : 1);
  StagedShape best{64, 1, 0};
  double least = 0.0;
  for (int edge = 128; edge >= 64; edge -= 64) {
    const double shared = p.f32 ? (edge == 128 ? 2.08 : 0.58) : (edge == 128 ? 0.87 : 0.38);
    const double alone = p.f32 ? (edge == 128 ? 2.35 : 0.72) : (edge == 128 ? 1.1 : 0.55);
    const int64_t tiles = lin_tiles_count(p, edge, edge);
    // Only 64 x 64 tiles are split, few enough for a ticket each, down to 4 stages.
    for (int s = 1; s <= 16 && (s == 1 || (may_split && edge == 64 && tiles <= kMaxTickets && 4 * s <= stages)); ++s) {
      const int64_t k = (tiles * s + kCUs - 1) / kCUs;
      const double t = static_cast<double>((stages + s - 1) / s) * std::max(alone, shared * static_cast<double>(k)) +
                       (s > 1 ? 2.0 + 0.007 * static_cast<double>(tiles * s) : 0.0);
      if (!best.tiles || t < least) {
        best = {edge, s, tiles};
        least = t;
      }
    }
  }
  return best;
}

int64_t ws_of(const StagedShape& h) { return h.splits > 1 ? kTicketBytes + h.tiles * h.splits * 64 * 64 * 4 : 0; }

// ---- tiled bf16 ----------------------------------------------------------------

// The small tile: 64 rows by 64 columns (of each weight).
int64_t small_tiles(const LinGemm& p) { return lin_tiles_count(p, 64, p.mode == kModeDual ? 128 : 64); }

// The tile: waves of workgroups over the CUs times the tile's work over its
// relative throughput (measured in gemm.hip).  Problems too small to give every
// CU a 128 x 128 tile take small ones, several of which share a CU: with three
// stages in flight (2048 -> 4096 at 256 rows 12.7 us against 17.4 with two; gated
// 12288 -> 6144 at 256 rows 160 against 173, and 199 with four), or two where a workgroup has
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

// Whether few rows run on their own kernel: always where the tiled ones cannot, up
// to 16 rows, and up to 32 with a weight of under 20 million elements (which it
// reads once, but every 16 columns' workgroup all activations), or of under 50
// million where the workspace does not let the tiled ones split K.  At 17 / 32
// rows, this kernel against the tiled ones (us), with the workspace: 4096 -> 2048
// 8.4 / 9.7 : 12.5 / 12.6, 4096 -> 4096 11.1 / 13.7 : 14.2 / 14.3, gated 4096 -> 2048 11.1 / 12.3 :
// 15.6 / 15.6, 2048 -> 8192 14.3 / 16.3 : 12.9 / 13.0; 4096 -> 6144 20.7 / 25.9 : 14.9 / 15.0, gated
// 4096 -> 4096 17.0 / 19.2 : 17.8 / 17.8, 6144 -> 8192 30.5 / 37.6 : 24.6 / 25.8.  Without: 4096 ->
// 6144 20.7 / 25.8 : 30.7 / 30.8, gated 4096 -> 4096 16.6 / 18.5 : 35.0 / 35.2, 6144 -> 6144
// 28.4 / 36.2 : 29.9 / 29.9; 6144 -> 8192 28.5 / 36.3 : 29.8 / 29.9, 8192 -> 8192 36.3 / 46.6 : 38.6 / 38.6.
bool takes_rows(const LinGemm& p, int64_t ws_bytes) {
  if (!rows_ok(p)) return false;
  if (p.M <= 16 || !tiles_ok(p)) return true;
  if (p.M > 32) return false;
  const int64_t most = ws_bytes >= ws_of(p, pick(p)) ? 20'000'000 : 50'000'000;
  return (p.mode == kModeDual ? 2 : 1) * p.N * p.K < most;
}

// Splits K only where the workspace holds the tickets and partials.
void take_ws(LinGemm *p, void *ws) {
  p->tickets = static_cast<uint32_t *>(ws);
  p->join = reinterpret_cast<float *>(static_cast<char *>(ws) + kTicketBytes);
}

hipError_t launch_rows(LinGemm p, void *ws, int64_t ws_bytes, hipStream_t s) {
  RowsShape h = rows_shape(p);
  if (ws_bytes < ws_of(h)) h.splits = 1;
  if (h.splits > 1) take_ws(&p, ws);
  return lin_rows_launch(p, h, s);
}

hipError_t launch_staged(LinGemm p, void *ws, int64_t ws_bytes, hipStream_t s) {
  StagedShape h = staged_shape(p, true);
  if (ws_bytes < ws_of(h)) h = staged_shape(p, false);
  if (h.splits > 1) take_ws(&p, ws);
  return lin_staged_launch(p, h, s);
}

hipError_t launch_tiles(LinGemm p, void *ws, int64_t ws_bytes, hipStream_t s) {
  TilePick t = pick(p);
  if (ws_bytes < ws_of(p, t)) t.splits = 1;
  if (t.splits > 1) take_ws(&p, ws);
  if (p.a_t) return lin_tiles_pair(p, t, s);
  switch (p.mode) {
    case kModeOne: return lin_tiles_one(p, t, s);
    case kModeDual: return lin_tiles_dual(p, t, s);
    case kModeCat: return lin_tiles_cat(p, t, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

// A launch holds fewer than 2^32 threads. Tiles: up to 2^22 of 64 x 64, 256
// threads each, twice where two products share a launch (2^31). Few rows: 16
// columns to a workgroup of up to 512 threads, so N below 2^26 (2^31).
bool lin_grid_ok(int64_t M, int64_t N) {
  return N < (int64_t{1} << 26) && ((M + 63) / 64) * ((N + 63) / 64) < (int64_t{1} << 22);
}

// Asked before strides and addresses are known, so for aligned ones.  What an
// unaligned call runs on instead asks for no more: the general kernel's need is
// counted, and the few-row kernel's (17 to 64 rows) stays below the others'.
int64_t lin_gemm_ws(const LinGemm& p) {
  if (p.M <= 0 || p.N <= 0) return 0;
  if (takes_rows(p, INT64_MAX)) return ws_of(rows_shape(p));
  return std::max(tiles_ok(p) ? ws_of(p, pick(p)) : 0, ws_of(staged_shape(p, true)));
}

hipError_t lin_gemm_launch(const LinGemm& p, hipStream_t s, void *ws, int64_t ws_bytes) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  if (!ws) ws_bytes = 0;
  if (takes_rows(p, ws_bytes)) return launch_rows(p, ws, ws_bytes, s);
  if (tiles_ok(p)) return launch_tiles(p, ws, ws_bytes, s);
  return launch_staged(p, ws, ws_bytes, s);
}

// The grid of the activation's gradient: 64 rows to a slab, fewer where that leaves
// under 1024 workgroups (1021 x 999, gated: 67 us in 32 workgroups), though not
// so few that the partial rows weigh more than an eighth of the input, nor so
// many slabs that they exceed the grid.
ActGrid act_grad_grid(int64_t M, int64_t N) {
  ActGrid g{64, 0, 64, 0};
  while (g.lanes > 1 && (g.lanes / 2) * kActCols >= N) g.lanes /= 2;
  g.tiles = (N + g.lanes * kActCols - 1) / (g.lanes * kActCols);
  const int64_t least = std::max<int64_t>(16, kActThreads / g.lanes);
  while (g.rows > least && g.tiles * ((M + g.rows - 1) / g.rows) < 1024) g.rows /= 2;
  g.rows = std::max(std::max(g.rows, least), (M + 1023) / 1024);
  g.slabs = (M + g.rows - 1) / g.rows;
  return g;
}

}  // namespace tpshard
