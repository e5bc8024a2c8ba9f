// Host stand-ins for the launchers of the vocabulary cross entropy and the AdamW step
// (and of the products they share with the linear layer): each checks that every byte
// range its kernels would touch lies inside one registered allocation, and that the
// launch is one the kernels are built for; it aborts otherwise.  Nothing runs on a GPU.
#include "loss_stub.h"

#include <cstdio>
#include <cstdlib>

#include "../../sharded_gemm_amd/csrc/adamw.h"
#include "../../sharded_gemm_amd/csrc/ce.h"

using namespace tpshard;

namespace {

struct Range {
  uintptr_t lo, hi;
};
std::vector<Range> g_allocs;
std::vector<std::string> g_seen;
bool g_quiet = false;

void check(bool ok, const char *what) {
  if (ok) return;
  std::fprintf(stderr, "launch check: %s\n", what);
  std::abort();
}

void need(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t es, const char *what, int64_t align = 0) {
  if (rows <= 0 || cols <= 0) return;
  check(p && ld >= cols, what);
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + static_cast<uintptr_t>(((rows - 1) * ld + cols) * es);
  check(lo % static_cast<uintptr_t>(align ? align : es) == 0, what);
  for (const Range& r : g_allocs)
    if (lo >= r.lo && hi <= r.hi) return;
  std::fprintf(stderr, "launch check: %s [%#lx, %#lx) outside every allocation\n", what, (unsigned long)lo, (unsigned long)hi);
  std::abort();
}
void vec(const void *p, int64_t n, int64_t es, const char *what, int64_t align = 0) { need(p, 1, n, n, es, what, align); }

void grid(int64_t x, int64_t y, int64_t threads) {
  check(x >= 1 && y >= 1 && x < (int64_t{1} << 31) && y < 65536 && x * y * threads < (int64_t{1} << 32), "grid");
}

void seen(const std::string& s) {
  if (!g_quiet) g_seen.push_back(s);
}
void seen_product(const char *type, const char *kernel, int n, const LinGemm& p, int splits) {
  static const char *names[] = {"one", "dual", "cat", "pair", "stats", "prob", "slices", "scaled"};
  if (g_quiet) return;
  const std::string s = std::string(type) + kernel + (n ? std::to_string(n) : "") + " " + names[p.mode] + (p.a_t ? " a^T" : " a") + (p.w_t ? " w^T" : " w");
  if (splits > 1) g_seen.push_back(s + " split");
  g_seen.push_back(s);
}

// A product's operands and what its epilogue touches; bm x bn: its tiles.
void product(const LinGemm& p, int64_t align, int64_t bm, int64_t bn) {
  const int64_t es = p.f32 ? 4 : 2;
  check(p.mode == kModeOne || p.mode == kModeStats || p.mode == kModeProb || p.mode == kModeSlices || p.mode == kModeScaled, "mode");
  check(p.M > 0 && p.N > 0 && p.K >= 0 && p.N < (int64_t{1} << 31), "sizes");
  need(p.a, p.a_t ? p.K : p.M, p.a_t ? p.M : p.K, p.lda, es, "A", align);
  need(p.w, p.w_t ? p.N : p.K, p.w_t ? p.K : p.N, p.ldw, es, "W", align);
  check(!p.aux && !p.aux2 && !p.bias && !p.res && !p.act, "a plain product");
  if (p.mode == kModeScaled) {
    check(!p.f32, "scaled: bf16");
    vec(static_cast<const ScaledGemm&>(p).alpha, 1, 4, "alpha");
  }
  if (p.mode == kModeOne || p.mode == kModeScaled) {
    check(!p.acc_c || p.c_f32, "only fp32 accumulates");
    check(!p.f32 || p.c_f32, "fp32 operands have an fp32 output");
    need(p.c, p.M, p.N, p.ldc, p.c_f32 ? 4 : 2, "C");
    return;
  }
  if (p.mode == kModeSlices) return;
  const CeGemm& q = static_cast<const CeGemm&>(p);
  vec(q.targets, q.M, 8, "targets");
  check(q.cols > 0 && q.cols <= q.N, "columns");
  if (p.mode == kModeStats) {
    const int64_t tiles = (q.N + bn - 1) / bn;
    check(q.slot0 >= 0, "slots");
    vec(q.part + 2 * q.slot0 * q.M, 2 * tiles * q.M, 4, "pairs", 8);
    vec(q.logit, q.M, 4, "logits of targets");
  } else {
    check(q.pad_rows >= q.M && q.pad_rows <= (q.M + bm - 1) / bm * bm, "zero rows lie in the tiles");
    check(q.c_f32 == q.f32, "P in the operands' type");
    need(q.c, q.pad_rows, q.N, q.ldc, es, "P", 16);
    vec(q.lse, q.M, 4, "lse");
    check(!q.scale == static_cast<bool>(q.f32), "the scale is bf16's");
    if (q.scale) vec(q.scale, 1, 4, "scale");
    if (q.g) vec(q.g, q.g_step ? q.M : 1, 4, "g");
    if (q.h) vec(q.h, q.h_step ? q.M : 1, 4, "h");
  }
}

void split(const LinGemm& p, int splits, int64_t tiles, int64_t floats) {
  check(splits >= 1 && splits <= 16, "splits");
  if (splits == 1) return;
  check(tiles <= kMaxTickets, "a ticket for every tile");
  check(reinterpret_cast<const char *>(p.join) == reinterpret_cast<const char *>(p.tickets) + kTicketBytes, "the partials follow the tickets");
  vec(p.tickets, kTicketBytes + tiles * splits * floats * 4, 1, "workspace", 8);
}

hipError_t tiles(const LinGemm& p, const TilePick& t) {
  static const char *names[] = {"tile256", "tile192", "tile128w", "tile128", "tile64", "tile64short", "tile64k32", "tile32"};
  static const int bm[] = {256, 256, 256, 128, 64, 64, 64, 32}, bn[] = {256, 192, 128, 128, 64, 64, 64, 64};
  check(t.tile >= 0 && t.tile < 8 && (t.tile != kTile32 || p.mode == kModeStats), "tile");
  product(p, 16, bm[t.tile], bn[t.tile]);
  check(!p.f32 && p.lda % 8 == 0 && p.ldw % 8 == 0, "tiled: strides");
  check(p.K > 0 && p.K % 32 == 0, "tiled: K");
  if (t.tile != kTile128 && t.tile != kTile64k32) check(p.K % 64 == 0, "tiled: K of a 64-wide stage");
  check(p.groups || ((!p.a_t || p.M % 8 == 0) && (p.w_t || p.N % 8 == 0)), "tiled: whole column groups");
  if (p.a_t) need(p.a, p.K, (p.M + 7) / 8 * 8, p.lda, 2, "A's groups", 16);
  if (!p.w_t) need(p.w, p.K, (p.N + 7) / 8 * 8, p.ldw, 2, "W's groups", 16);
  check(!(t.tile == kTile256 && p.a_t && !p.w_t), "tiled: no such instance");
  if (t.tile == kTile256 || t.tile == kTile192 || t.tile == kTile128w)
    check((p.a_t ? p.K : p.M) * p.lda * 2 < (int64_t{1} << 31) && (p.w_t ? p.N : p.K) * p.ldw * 2 < (int64_t{1} << 31),
          "tiled: 32-bit offsets");
  check(t.tile >= kTile64 || t.splits == 1, "tiled: only the small tiles are split");
  const int64_t n = lin_tiles_count(p, bm[t.tile], bn[t.tile]);
  grid(n, t.splits, 512);
  split(p, t.splits, n, bm[t.tile] * bn[t.tile]);
  seen_product("", names[t.tile], 0, p, t.splits);
  return hipSuccess;
}

}  // namespace

std::vector<std::string> loss_stub_take() {
  std::vector<std::string> r;
  r.swap(g_seen);
  return r;
}
void loss_stub_register(const void *p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  g_allocs.push_back({lo, lo + static_cast<uintptr_t>(bytes)});
}
void loss_stub_reset() { g_allocs.clear(); }
void loss_stub_quiet(bool on) { g_quiet = on; }

namespace tpshard {

hipError_t lin_rows_launch(const LinGemm& p, const RowsShape& h, hipStream_t) {
  product(p, 0, 64, 16 * h.g);
  const int tc = 16 * h.g, es = p.f32 ? 4 : 2;
  check(p.M <= (p.w_t ? 64 : 16) && p.K >= 1 && !p.a_t && !p.acc_c && p.mode == kModeOne, "few rows");
  check(h.g == (p.w_t ? 1 : 8 / es) && h.waves >= 1 && h.waves <= kRowsWaves, "few rows: shape");
  check(h.tiles == (p.N + tc - 1) / tc && h.cells == p.M * tc, "few rows: tiles");
  grid(h.tiles, h.splits, 64 * h.waves);
  split(p, h.splits, h.tiles, h.cells);
  seen_product(p.f32 ? "f32 " : "bf16 ", "rows", 0, p, h.splits);
  return hipSuccess;
}

hipError_t lin_staged_launch(const LinGemm& p, const StagedShape& h, hipStream_t) {
  check(h.edge == 64 || h.edge == 128, "general: edge");
  product(p, 0, h.edge, h.edge);
  check(h.edge == 64 || h.splits == 1, "general: only the small tile is split");
  check(h.tiles == lin_tiles_count(p, h.edge, h.edge), "general: tiles");
  check(p.a_t ? p.mode == kModeOne && (p.f32 || !p.w_t) : p.mode != kModeScaled || !p.f32, "general: no such instance");
  grid(h.tiles, h.splits, h.edge == 128 ? 512 : 256);
  split(p, h.splits, h.tiles, 64 * 64);
  seen_product(p.f32 ? "f32 " : "bf16 ", "general", h.edge, p, h.splits);
  return hipSuccess;
}

hipError_t lin_tiles_one(const LinGemm& p, const TilePick& t, hipStream_t) {
  check(!p.a_t && p.mode == kModeOne, "one");
  return tiles(p, t);
}
hipError_t lin_tiles_stats(const CeGemm& p, const TilePick& t, hipStream_t) {
  check(!p.a_t && p.mode == kModeStats, "stats");
  return tiles(p, t);
}
hipError_t lin_tiles_prob(const CeGemm& p, const TilePick& t, hipStream_t) {
  check(!p.a_t && p.mode == kModeProb, "prob");
  return tiles(p, t);
}
hipError_t lin_tiles_wgrad(const ScaledGemm& p, const TilePick& t, hipStream_t) {
  check(p.a_t && p.w_t && p.mode == kModeScaled, "weight gradient");
  return tiles(p, t);
}
hipError_t lin_tiles_scaled(const ScaledGemm& p, const TilePick& t, hipStream_t) {
  check(!p.a_t && p.mode == kModeScaled, "scaled");
  return tiles(p, t);
}
hipError_t lin_tiles_slices(const LinGemm& p, const TilePick& t, hipStream_t) {
  static const int bn[] = {256, 192, 128};
  check(p.mode == kModeSlices && !p.a_t && !p.f32 && p.c_f32 && !p.acc_c, "slices");
  check(t.tile == kTile256 || t.tile == kTile128w, "slices: tile");
  product(p, 16, 256, bn[t.tile]);
  check(p.K % 64 == 0 && t.splits > 1 && t.splits <= p.K / 64, "slices: stages");
  check(p.lda % 8 == 0 && p.ldw % 8 == 0 && (p.w_t || p.groups || p.N % 8 == 0), "slices: operands");
  if (!p.w_t) need(p.w, p.K, (p.N + 7) / 8 * 8, p.ldw, 2, "W's groups", 16);
  check(p.M * p.lda * 2 < (int64_t{1} << 31) && (p.w_t ? p.N : p.K) * p.ldw * 2 < (int64_t{1} << 31), "slices: 32-bit offsets");
  need(p.c, t.splits * p.M, p.N, p.ldc, 4, "partial sums");
  grid(lin_tiles_count(p, 256, bn[t.tile]), t.splits, 512);
  static const char *names[] = {"tile256", "tile192", "tile128w"};
  seen_product("", names[t.tile], 0, p, 1);
  return hipSuccess;
}
hipError_t lin_tiles_dual(const LinGemm&, const TilePick&, hipStream_t) { std::abort(); }
hipError_t lin_tiles_cat(const LinGemm&, const TilePick&, hipStream_t) { std::abort(); }
hipError_t lin_tiles_pair(const LinGemm&, const TilePick&, hipStream_t) { std::abort(); }

hipError_t zero_tickets_launch(uint32_t *tickets, hipStream_t) {
  vec(tickets, kMaxTickets, 4, "tickets");
  return hipSuccess;
}

hipError_t ce_logits_launch(const CeLogits& p, hipStream_t) {
  const int64_t slots = (p.n + kCeStatCols - 1) / kCeStatCols;
  check(p.M >= 1 && p.M <= 64 && p.ld % 4 == 0, "logits: rows");
  grid(slots, p.M, 256);
  need(p.z, p.M, p.n, p.ld, 4, "logits", 16);
  vec(p.targets, p.M, 8, "targets");
  vec(p.part, 2 * slots * p.M, 4, "pairs", 8);
  vec(p.logit, p.M, 4, "logits of targets");
  seen("logits");
  return hipSuccess;
}
namespace {
void joined(const CeJoin& p) {
  check(p.slots >= 1, "slots");
  vec(p.part, 2 * p.slots * p.M, 4, "pairs", 8);
  vec(p.logit, p.M, 4, "logits of targets");
  vec(p.targets, p.M, 8, "targets");
  if (p.stats) vec(p.stats, 3 * p.M, 4, "stats");
  if (p.loss) vec(p.loss, p.M, 4, "loss");
  if (p.lse) vec(p.lse, p.M, 4, "lse");
}
}  // namespace
hipError_t ce_join_launch(const CeJoin& p, hipStream_t) {
  grid(p.M < 1024 ? p.M : (p.M + 15) / 16, 1, 256);
  joined(p);
  seen("join");
  return hipSuccess;
}
hipError_t ce_pieces_launch(const float *stats, int64_t pieces, int64_t M, const int64_t *targets, int64_t, float *loss,
                            float *lse, hipStream_t) {
  vec(stats, 3 * pieces * M, 4, "stats");
  vec(targets, M, 8, "targets");
  if (loss) vec(loss, M, 4, "loss");
  if (lse) vec(lse, M, 4, "lse");
  seen("pieces");
  return hipSuccess;
}
namespace {
void scaled(const CeScale& p) {
  vec(p.tickets, kMaxTickets, 4, "tickets");
  if (!p.scale) return;
  vec(p.scale, 1, 4, "scale");
  vec(p.targets, p.M, 8, "targets");
  if (p.g) vec(p.g, p.g_step ? p.M : p.M > 0, 4, "g");
  if (p.h) vec(p.h, p.h_step ? p.M : p.M > 0, 4, "h");
}
}  // namespace
hipError_t ce_scale_launch(const CeScale& p, hipStream_t) {
  scaled(p);
  seen("scale");
  return hipSuccess;
}
static int64_t padded(const CePads& pads) {
  int64_t blocks = 0;
  for (int i = 0; i < pads.num; ++i) {
    const CePad& p = pads.pad[i];
    check(p.cols % 8 == 0 && p.rows >= p.m && p.cols >= p.n && p.m > 0 && p.n > 0, "pad: sizes");
    need(p.from, p.m, p.n, p.ld, 2, "padded from");
    vec(p.to, p.rows * p.cols, 2, "padded copy", 16);
    blocks += (p.rows * (p.cols / 8) + 255) / 256;
  }
  if (pads.num) seen("pad");
  return blocks;
}
hipError_t ce_transpose_launch(const CeTranspose& p, const CePads& pads, hipStream_t) {
  check(p.rows % 64 == 0 && p.rows >= p.M && p.M > 0, "transpose: rows");
  grid((p.K + 63) / 64 * (p.rows / 64) + padded(pads), 1, 256);
  need(p.X, p.M, p.K, p.X_ld, p.f32 ? 4 : 2, "X");
  vec(p.xt, p.K * p.rows, p.f32 ? 4 : 2, "X^T", 16);
  vec(p.targets, p.M, 8, "targets");
  scaled(p.scale);
  seen("transpose");
  return hipSuccess;
}
hipError_t ce_pad_launch(const CePads& p, hipStream_t) {
  check(p.num > 0, "no copies");
  grid(padded(p), 1, 256);
  return hipSuccess;
}
hipError_t ce_sum_launch(const CeSum& p, hipStream_t) {
  grid((p.M * ((p.K + 3) / 4) + 255) / 256, 1, 256);
  check(p.slices >= 1, "sum: slices");
  vec(p.part, p.slices * p.M * p.K, 4, "partial sums");
  if (p.alpha) vec(p.alpha, 1, 4, "alpha");
  if (p.base) need(p.base, p.M, p.K, p.base_ld, 4, "sum so far");
  need(p.out, p.M, p.K, p.out_ld, p.out_f32 ? 4 : 2, "dX");
  seen("sum");
  return hipSuccess;
}

hipError_t adamw_launch(const AdamTensor *ts, int64_t num, bool codes, const AdamArgs& a, hipStream_t) {
  const int64_t chunk = adam_chunk(ts, num);
  int64_t at = 0;
  do {
    AdamTable t;
    next_adam(ts, num, &at, &t, chunk, chunk == kAdamChunk);
    check(t.num <= kMaxAdam, "tensors of a launch");
    for (int i = 0; i < t.num; ++i) {
      const AdamTensor& x = t.t[i];
      const int64_t scales = (x.n + kAdamBlock - 1) / kAdamBlock;
      const int64_t n = (t.first[i + 1] - t.first[i]) * chunk;
      check(chunk == kAdamChunk ? n <= x.n && n + chunk > x.n : n - chunk < x.n && n >= x.n, "chunks");
      vec(x.param, x.n, x.param_f32 ? 4 : 2, "param");
      vec(x.grad, x.n, x.grad_f32 ? 4 : 2, "grad");
      vec(x.m, x.n, codes ? 1 : 4, "m");
      vec(x.v, x.n, codes ? 1 : 4, "v");
      if (codes) vec(x.ms, scales, 4, "m_scale");
      if (codes) vec(x.vs, scales, 4, "v_scale");
      if (x.copy) vec(x.copy, x.n, 2, "copy");
    }
  } while (at < num);
  if (a.parts) vec(a.parts, a.ranks * kGradParts, 8, "parts");
  if (a.norm_out) vec(a.norm_out, 1, 4, "norm");
  if (a.step) vec(a.step, 1, 8, "step");
  if (a.lr_dev) vec(a.lr_dev, 1, 4, "lr");
  seen(codes ? "adamw 8" : "adamw 32");
  return hipSuccess;
}
hipError_t adamw_values_launch(const AdamValues *ts, int64_t num, hipStream_t) {
  for (int64_t i = 0; i < num; ++i) {
    const AdamValues& x = ts[i];
    vec(x.m, x.n, 1, "m");
    vec(x.v, x.n, 1, "v");
    vec(x.ms, (x.n + kAdamBlock - 1) / kAdamBlock, 4, "m_scale");
    vec(x.vs, (x.n + kAdamBlock - 1) / kAdamBlock, 4, "v_scale");
    vec(x.m_out, x.n, x.f32 ? 4 : 2, "m_out");
    vec(x.v_out, x.n, x.f32 ? 4 : 2, "v_out");
  }
  seen("adamw values");
  return hipSuccess;
}

}  // namespace tpshard
