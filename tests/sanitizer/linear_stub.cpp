// Host stand-ins for the launchers of the linear layer, the gated block and
// gradient clipping: each checks that every byte range its kernels would touch
// (operands, outputs, tickets and partials in the workspace) lies inside one
// registered allocation, and that the launch is one the kernels are built for;
// it aborts otherwise.  Nothing runs on a GPU.
#include "linear_stub.h"

#include <cstdio>
#include <cstdlib>

#include "../../sharded_gemm_amd/csrc/grad_table.h"
#include "../../sharded_gemm_amd/csrc/linear.h"

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

// rows x cols at row stride ld lie inside one allocation, aligned to `align` bytes.
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

void grid(int64_t x, int64_t y, int64_t threads) {
  check(x >= 1 && y >= 1 && x < (int64_t{1} << 31) && y < 65536 && x * y * threads < (int64_t{1} << 32), "grid");
}

const char *mode_name(int mode) {
  static const char *names[] = {"one", "dual", "cat", "pair"};
  check(mode >= 0 && mode < 4, "mode");
  return names[mode];
}

// The operands and outputs of a product.
void product(const tpshard::LinGemm& p, int64_t align) {
  using namespace tpshard;
  const int64_t es = p.f32 ? 4 : 2, ces = p.c_f32 ? 4 : 2;
  check(!p.f32 || p.c_f32, "fp32 operands have an fp32 output");
  const bool two_w = p.mode != kModeOne, two_a = p.mode == kModeCat || p.mode == kModePair;
  for (int i = 0; i < 1 + two_a; ++i)
    need(i ? p.a2 : p.a, p.a_t ? p.K : p.M, p.a_t ? p.M : p.K, p.lda, es, "A", align);
  for (int i = 0; i < 1 + two_w; ++i)
    need(i ? p.w2 : p.w, p.w_t ? p.N : p.K, p.w_t ? p.K : p.N, p.ldw, es, "W", align);
  need(p.c, p.M, p.N, p.ldc, ces, "C");
  if (p.mode == kModePair) need(p.c2, p.M, p.N, p.ldc, ces, "C2");
  check(!p.acc_c || p.c_f32, "only fp32 accumulates");
  if (p.bias) need(p.bias, 1, p.N, p.N, 4, "bias");
  if (p.res) need(p.res, p.M, p.N, p.ldres, es, "residual");
  if (p.aux) need(p.aux, p.M, p.N, p.ldaux, es, "aux");
  if (p.aux2) need(p.aux2, p.M, p.N, p.ldaux, es, "aux2");
  check(p.mode == kModeOne || (!p.bias && !p.res), "bias and residual are kModeOne's");
}

// Tickets and partials of a split launch.
void split(const tpshard::LinGemm& p, int splits, int64_t tiles, int64_t floats) {
  using namespace tpshard;
  check(splits >= 1 && splits <= 16, "splits");
  if (splits == 1) return;
  check(tiles <= kMaxTickets, "a ticket for every tile");
  check(reinterpret_cast<const char *>(p.join) == reinterpret_cast<const char *>(p.tickets) + kTicketBytes, "the partials follow the tickets");
  need(p.tickets, 1, kTicketBytes + tiles * splits * floats * 4, kTicketBytes + tiles * splits * floats * 4, 1, "workspace", 8);
}

void seen(const char *type, const char *kernel, int n, const tpshard::LinGemm& p, int splits) {
  if (g_quiet) return;
  std::string s = std::string(type) + kernel + (n ? std::to_string(n) : "") + " " + mode_name(p.mode) + (p.a_t ? " a^T" : " a") + (p.w_t ? " w^T" : " w");
  if (splits > 1) g_seen.push_back(s + " split");
  g_seen.push_back(s);
}

}  // namespace

std::vector<std::string> lin_stub_take() {
  std::vector<std::string> r;
  r.swap(g_seen);
  return r;
}
void lin_stub_register(const void *p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  g_allocs.push_back({lo, lo + static_cast<uintptr_t>(bytes)});
}
void lin_stub_reset() { g_allocs.clear(); }
void lin_stub_quiet(bool on) { g_quiet = on; }

namespace tpshard {

hipError_t lin_rows_launch(const LinGemm& p, const RowsShape& h, hipStream_t) {
  product(p, 0);
  const int tc = 16 * h.g, es = p.f32 ? 4 : 2;
  check(p.M >= 1 && p.M <= (p.w_t ? 64 : 16) && p.K >= 1 && !p.a_t && !p.acc_c, "few rows");
  check(p.mode == kModeOne || p.mode == kModeDual, "few rows: mode");
  check(h.g == (p.w_t ? 1 : 8 / es), "few rows: columns");
  check(h.waves >= 1 && h.waves <= kRowsWaves, "few rows: waves");
  check(h.tiles == (p.N + tc - 1) / tc && h.cells == (p.mode == kModeDual ? 2 : 1) * p.M * tc, "few rows: tiles");
  check(h.waves * h.cells * 4 + 16 <= 160 * 1024, "few rows: LDS");
  grid(h.tiles, h.splits, 64 * h.waves);
  split(p, h.splits, h.tiles, h.cells);
  const int mt = p.M <= 16 ? 1 : p.M <= 32 ? 2 : 4;
  seen(p.f32 ? "f32 " : "bf16 ", "rows", 16 * mt, p, h.splits);
  return hipSuccess;
}

hipError_t lin_staged_launch(const LinGemm& p, const StagedShape& h, hipStream_t) {
  product(p, 0);
  check(h.edge == 64 || h.edge == 128, "general: edge");
  check(h.edge == 64 || h.splits == 1, "general: only the small tile is split");
  check(h.tiles == lin_tiles_count(p, h.edge, h.edge), "general: tiles");
  check(p.a_t ? (p.mode == kModeOne || p.mode == kModePair) && !p.w_t : p.mode != kModePair, "general: no such instance");
  grid(h.tiles, h.splits, h.edge == 128 ? 512 : 256);
  split(p, h.splits, h.tiles, 64 * 64);
  seen(p.f32 ? "f32 " : "bf16 ", "general", h.edge, p, h.splits);
  return hipSuccess;
}

namespace {
hipError_t tiles(const LinGemm& p, const TilePick& t, bool dual, bool cat) {
  static const char *names[] = {"tile256", "tile192", "tile128w", "tile128", "tile64", "tile64short", "tile64k32"};
  static const int bm[] = {256, 256, 256, 128, 64, 64, 64}, bn[] = {256, 192, 128, 128, 64, 64, 64};
  check(t.tile >= 0 && t.tile < 7, "tile");
  product(p, 16);
  check(!p.f32 && p.lda % 8 == 0 && p.ldw % 8 == 0, "tiled: strides");
  check(p.K > 0 && p.K % 32 == 0, "tiled: K");
  if (t.tile != kTile128 && t.tile != kTile64k32) check(p.K % 64 == 0, "tiled: K of a 64-wide stage");
  check((!p.a_t || p.M % 8 == 0) && (p.w_t || p.N % 8 == 0), "tiled: whole column groups");
  check((p.mode == kModeDual) == dual && (p.mode == kModeCat) == cat, "tiled: mode");
  check(!(t.tile == kTile256 && p.a_t) && !(t.tile == kTile192 && dual), "tiled: no such instance");
  if (t.tile == kTile256 || t.tile == kTile192 || t.tile == kTile128w)
    check((p.a_t ? p.K : p.M) * p.lda * 2 < (int64_t{1} << 31) && (p.w_t ? p.N : p.K) * p.ldw * 2 < (int64_t{1} << 31),
          "tiled: 32-bit offsets");
  const bool small = t.tile >= kTile64;
  check(small || t.splits == 1, "tiled: only the small tiles are split");
  const int n = small && dual ? 128 : bn[t.tile];
  grid(lin_tiles_count(p, bm[t.tile], n), t.splits, 512);
  check(lin_tiles_count(p, bm[t.tile], n) < (int64_t{1} << 31), "tiled: 32-bit tile numbers");
  split(p, t.splits, lin_tiles_count(p, bm[t.tile], n), 64 * n);
  seen("", names[t.tile], 0, p, t.splits);
  return hipSuccess;
}
}  // namespace

hipError_t lin_tiles_one(const LinGemm& p, const TilePick& t, hipStream_t) {
  check(!p.a_t, "one: A as it lies");
  return tiles(p, t, false, false);
}
hipError_t lin_tiles_dual(const LinGemm& p, const TilePick& t, hipStream_t) {
  check(!p.a_t, "dual: A as it lies");
  return tiles(p, t, true, false);
}
hipError_t lin_tiles_cat(const LinGemm& p, const TilePick& t, hipStream_t) {
  check(!p.a_t, "cat: A as it lies");
  return tiles(p, t, false, true);
}
hipError_t lin_tiles_pair(const LinGemm& p, const TilePick& t, hipStream_t) {
  check(p.a_t && !p.w_t && (p.mode == kModeOne || p.mode == kModePair), "pair: weight gradients");
  return tiles(p, t, false, false);
}

hipError_t zero_tickets_launch(uint32_t *tickets, hipStream_t) {
  need(tickets, 1, kMaxTickets, kMaxTickets, 4, "tickets");
  return hipSuccess;
}

hipError_t act_grad_launch(const ActGrad& p, hipStream_t) {
  const int64_t es = p.f32 ? 4 : 2;
  const ActGrid g = act_grad_grid(p.M, p.N);
  check(g.lanes >= 1 && g.lanes <= 64 && kActThreads % g.lanes == 0, "activation: lanes");
  check(g.tiles * g.lanes * kActCols >= p.N && g.slabs * g.rows >= p.M && (p.M == 0 || (g.slabs - 1) * g.rows < p.M), "activation: grid covers");
  need(p.d_out, p.M, p.N, p.ld_dout, es, "dOut");
  if (p.pre) need(p.pre, p.M, p.N, p.ld_pre, es, "pre");
  if (p.gated) need(p.up, p.M, p.N, p.ld_pre, es, "up");
  if (p.d_pre) need(p.d_pre, p.M, p.N, p.N, es, "dPre", 16);
  if (p.gated) need(p.d_up, p.M, p.N, p.N, es, "dUp", 16);
  if (p.colsum && p.M > 0) need(p.parts, g.slabs, p.N, p.N, 4, "partial rows");
  if (p.colsum) need(p.colsum, 1, p.N, p.N, 4, "dbias");
  if (p.tickets) need(p.tickets, 1, kMaxTickets, kMaxTickets, 4, "tickets");
  if (p.M > 0) {
    grid(g.tiles, g.slabs, kActThreads);
    const bool flat = p.gated && p.ld_dout == p.N && p.ld_pre == p.N;
    if (!g_quiet) g_seen.push_back(std::string(p.f32 ? "f32 " : "bf16 ") + (flat ? "gated gradient, flat" : p.gated ? "gated gradient, rows" : "activation gradient"));
  }
  if (p.colsum) grid((p.N + 63) / 64, 1, 1024);
  return hipSuccess;
}

namespace {
// Every tensor's chunks come once, in tables of at most kMaxTensors.
void tables(const GradTensor *ts, int64_t num, bool outs) {
  int64_t at = 0, k = 0;
  do {
    GradTable t;
    next_table(ts, num, &at, &t);
    check(t.num >= 0 && t.num <= kMaxTensors, "table size");
    for (int i = 0; i < t.num; ++i, ++k) {
      while (k < num && ts[k].n <= 0) ++k;
      check(k < num && t.g[i] == ts[k].g && t.n[i] == ts[k].n && (t.f32 >> i & 1) == static_cast<uint64_t>(ts[k].f32), "table order");
      check((t.first[i + 1] - t.first[i]) * kGradChunk >= t.n[i] && (t.first[i + 1] - t.first[i] - 1) * kGradChunk < t.n[i], "table chunks");
      need(t.g[i], 1, t.n[i], t.n[i], ts[k].f32 ? 4 : 2, "gradient");
      if (outs) need(t.out[i], 1, t.n[i], t.n[i], ts[k].f32 ? 4 : 2, "clipped gradient");
    }
  } while (at < num);
  while (k < num && ts[k].n <= 0) ++k;
  check(k == num, "every tensor has its table");
}
}  // namespace

hipError_t grad_sumsq_launch(const GradTensor *ts, int64_t num, double *parts, hipStream_t) {
  need(parts, 1, kGradParts, kGradParts, 8, "parts");
  tables(ts, num, false);
  return hipSuccess;
}
hipError_t grad_clip_launch(const GradTensor *ts, int64_t num, const double *parts, int64_t ranks, double, double,
                            float *norm_out, hipStream_t) {
  need(parts, ranks, kGradParts, kGradParts, 8, "parts");
  if (norm_out) need(norm_out, 1, 1, 1, 4, "norm");
  tables(ts, num, true);
  return hipSuccess;
}

}  // namespace tpshard
