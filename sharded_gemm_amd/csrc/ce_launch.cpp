// The vocabulary cross entropy: which kernels run, over which pieces of the
// vocabulary, and where in the workspace.  Host code only: what a launch reads and
// writes can be checked without a GPU.
#include "ce.h"

#include <algorithm>

#include "common.h"
#include "timing.h"

namespace tpshard {

namespace {

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t cut(int64_t n, int64_t by) { return (n + by - 1) / by; }
constexpr int64_t kAlign = 256;   // of the workspace's parts

LinGemm logits_product(const CeSizes& c, int mode, int64_t N) {
  LinGemm p;
  p.mode = mode;
  p.M = c.M;
  p.N = N;
  p.K = c.K;
  p.f32 = c.f32;
  p.w_t = c.linear;
  return p;
}

// The weight from column n on.
const void *weight_at(const CeSizes& c, const void *W, int64_t ld, int64_t n) {
  return static_cast<const char *>(W) + (c.linear ? n * ld : n) * (c.f32 ? 4 : 2);
}

// Whether X and W are copied into the workspace, K padded to whole stages and W's
// rows aligned, so that the tiled bf16 kernels take sizes that are no multiple of
// anything.  The copy moves four bytes for each element of W, so it pays from some
// number of tokens on; later where rows are aligned anyway and only K's last stage is
// not whole.  MI355X, general kernel : padded (us), 4095 -> 32001 forward at 256
// tokens 138 : 168, 512 251 : 191, 1024 445 : 292; backward at 65 tokens 372 : 414, 129 468 :
// 452, 512 893 : 701; aligned, 1000 -> 8000 forward at 512 25 : 33, backward 69 : 70, at 1024 100 : 96.
bool padded(const CeSizes& c, bool backward) {
  if (c.f32 || (c.K % 32 == 0 && (c.K % 64 == 0 || c.K < 256) && (c.linear || c.V % 8 == 0))) return false;
  return c.M >= (c.K % 8 == 0 && (c.linear || c.V % 8 == 0) ? 1024 : backward ? 128 : 512);
}
// Columns from n on of W, `cols` of them, as [columns][K] or [K][columns], padded.
CePad pad_weight(const CeSizes& c, const CeOperands& o, int64_t n, int64_t cols, int64_t cols_pad, int64_t K_pad, void *to) {
  CePad p;
  p.from = weight_at(c, o.W, o.W_ld, n);
  p.ld = o.W_ld;
  p.to = to;
  p.m = c.linear ? cols : c.K;
  p.n = c.linear ? c.K : cols;
  p.rows = c.linear ? cols_pad : K_pad;
  p.cols = c.linear ? K_pad : cols_pad;
  return p;
}
CePad pad_x(const CeSizes& c, const CeOperands& o, int64_t K_pad, void *to) {
  CePad p;
  p.from = o.X;
  p.ld = o.X_ld;
  p.to = to;
  p.m = p.rows = c.M;
  p.n = c.K;
  p.cols = K_pad;
  return p;
}
template <typename F>
hipError_t timed(hipStream_t s, int kind, double work, F&& f) {
  hipEvent_t t0 = timing_begin(s);
  const hipError_t e = f();
  if (e == hipSuccess) timing_end(t0, s, kind, work);
  return e;
}
double bytes_of(const CePads& p) {
  double n = 0;
  for (int i = 0; i < p.num; ++i) n += 4.0 * static_cast<double>(p.pad[i].rows) * static_cast<double>(p.pad[i].cols);
  return n;
}
hipError_t pad(const CePads& p, hipStream_t s) {
  return p.num ? timed(s, TP_KERNEL_REDUCE, bytes_of(p), [&] { return ce_pad_launch(p, s); }) : hipSuccess;
}

// ---- forward ---------------------------------------------------------------------
// A product whose epilogue reduces each tile: in one launch, unless the weight's bytes
// pass the 2^31 up to which the ping-pong kernels' offsets reach, or its tiles the
// grid; then in even pieces of whole tiles.
// Up to 64 rows run in 64-column tiles of 32 or 64 rows, three or more of which share a
// CU: bound by the weight's bytes, whether there is one row or 32.  (MI355X, 16 rows,
// us, against the few-row kernel and a pass over its logits: 768 -> 32000 13.8 : 23.7, 4096
// -> 131072 175.8 : 257; one row 13.0 : 21.0, 172.9 : 172.5, but 4096 -> 65536 103 : 92.  32 rows
// a tile and four stages: 64 rows and three took 14.7 and 112 at 4096 -> 65536.)
// fp32 has no such tiles; up to 16 rows of it take the few-row kernel, which leaves
// the logits (M of them a column, where a column of the weight has K), and a pass of
// its own reduces them, 2^18 columns at a time: one row of 1024 -> 40000 39 us, the
// general kernel 63.
constexpr int64_t kLogitCols = int64_t{1} << 18;
constexpr int64_t kTileCols = 768;   // a multiple of every tile's columns

struct Forward {
  bool rows = false, small = false, pad = false;   // the few-row kernel; tiles of 64 columns; padded copies
  int64_t piece = 0, slots = 0, K = 0;             // columns of a launch; pairs of a row at most; K as multiplied
  int64_t held = 0;                                // columns of W that there is room for a copy of, whatever M is
  int64_t part = 0, logit = 0, logits = 0, x = 0, w = 0, total = 0;   // offsets; total: bytes
};

Forward forward_plan(const CeSizes& c) {
  Forward f;
  if (c.M <= 0) return f;
  const LinGemm one = logits_product(c, kModeOne, std::min(c.V, kLogitCols)), st = logits_product(c, kModeStats, c.V);
  f.rows = c.f32 && lin_takes_rows(one) && c.M <= 16;
  f.small = c.M <= 64 || lin_tiles_count(st, 128, 128) < 256;
  f.pad = !f.rows && padded(c, false);
  f.K = f.pad ? up(c.K, 64) : c.K;
  int64_t joined = 0;
  if (f.rows) {
    f.piece = std::min(c.V, kLogitCols);
    f.slots = cut(c.V, kCeStatCols);
    joined = lin_gemm_ws(one);
    if (c.V % f.piece) joined = std::max(joined, lin_gemm_ws(logits_product(c, kModeOne, c.V % f.piece)));
  } else if (f.small) {
    f.piece = f.held = std::min(c.V, int64_t{1} << 24);   // (a launch's threads stay below 2^32)
    f.slots = cut(c.V, 64);
    LinGemm q = st;
    q.K = f.K;
    q.groups = f.pad;
    joined = lin_gemm_ws(q);
  } else {
    const int64_t span = std::max(kTileCols, ((int64_t{1} << 31) - 1) / (2 * c.K));
    const int64_t grid = ((int64_t{1} << 22) - 1) / cut(c.M, 64) * 64;
    int64_t most = int64_t{1} << 25;
    if (c.linear && !c.f32) most = std::min(most, span);
    if (f.pad) most = std::min(most, std::max(16 * kTileCols, (int64_t{1} << 27) / f.K));   // 256 MiB of W
    auto even = [&](int64_t cols) { return up(cut(c.V, cut(c.V, cols / kTileCols * kTileCols)), kTileCols); };
    f.piece = even(std::min(most, grid));
    f.held = even(most);
    f.slots = cut(c.V, c.f32 ? 64 : 128) + cut(c.V, f.piece);
  }
  f.part = up(std::max(joined, kTicketBytes), kAlign);
  f.logit = f.part + up(f.slots * c.M * 8, kAlign);
  f.logits = f.logit + up(c.M * 4, kAlign);
  f.x = f.logits + (f.rows ? up(c.M * up(f.piece, 4) * 4, kAlign) : 0);
  f.w = f.x + (f.pad && c.K != f.K ? up(c.M * f.K * 2, kAlign) : 0);
  f.total = f.w + (f.pad ? up(std::min(f.held, c.V), 64) * f.K * 2 : 0);
  return f;
}

// What every M up to this one needs, so that a workspace of a full batch serves a ragged one: few rows
// split K, have twice the pairs, or (fp32) keep logits, where many do not.  Between the places
// below a plan's bytes only grow: all rows that the few-row kernel takes; whole 64s
// of those on small tiles; the last rows without padded copies.
int64_t forward_bytes(const CeSizes& c) {
  int64_t need = forward_plan(c).total;
  auto with = [&](int64_t M) {
    if (M >= c.M) return false;
    CeSizes d = c;
    d.M = M;
    const Forward f = forward_plan(d);
    need = std::max(need, f.total);
    return f.small;
  };
  if (c.f32)
    for (int64_t M = 1; M <= 16; ++M) (void)with(M);
  for (int64_t M : {511, 1023}) (void)with(M);
  for (int64_t M = 64; with(M); M += 64) {
  }
  return need;
}

// Columns of a tile.
int64_t columns_of(const LinChoice& h) {
  if (!h.tiles) return h.staged.edge;
  switch (h.tile.tile) {
    case kTile256: return 256;
    case kTile192: return 192;
    case kTile128w:
    case kTile128: return 128;
  }
  return 64;
}

// ---- backward ----------------------------------------------------------------------
// For each piece of the vocabulary: the gradient at its logits, P [M, columns] in the
// operands' type, from the product computed again; dX += P W^T; dW = X^T P.
//
// P has zero rows up to a multiple of 64 tokens, and X^T is kept transposed with as
// many zero columns, those of ignored tokens among them: so the products over tokens
// run on the tiled kernels whatever M is, what lies in X at an ignored token (a
// padded batch's rest) does not reach dW, and only one of their operands goes
// through the transposing LDS read.
// The product over columns, dX's, takes whole stages of them on the tiled kernels, so
// the vocabulary's last V % 64 columns are a piece of their own, with a padded copy
// of their part of W; where X and W are padded anyway every piece is copied.
//
// Pieces: 2^28 elements of P (512 MiB in bf16, 1 GiB in fp32), but 8192 columns at least (so with more than
// 32768 tokens P grows with them), so that dX is not read and written again often: with 8192 x 4096
// tokens every further piece costs 268 MB.  A bf16 weight's
// part of a piece stays below the 2^31 bytes that the ping-pong kernels' offsets reach, where rows are
// columns of the vocabulary or copied ([K, V] spans all its bytes whatever the piece): in one
// piece 800 x 12288 -> 131072 ran on 128 x 128 tiles throughout.
// The tail comes first, so that the last piece's sum can be dX itself.
//
// dX has few tiles where M K is not large, and a long sum: it is cut into slices of
// columns, each a partial dX in fp32, that a pass of its own adds up (slices below).
struct Backward {
  int64_t rows = 0, piece = 0, whole = 0, K = 0;   // tokens of P; its columns; the vocabulary in pieces of them; K as multiplied
  bool pad = false, tail = false;                  // every piece of W is copied; the last V - whole columns are
  bool keeps = false;                              // dX is summed in the workspace
  int64_t scale = 0, xt = 0, p = 0, acc = 0, x = 0, w = 0, part = 0, total = 0;
};

LinGemm dx_product(const CeSizes& c, int64_t n, bool copied) {
  LinGemm p;
  p.mode = c.f32 ? kModeOne : kModeScaled;
  p.groups = copied;
  p.M = c.M;
  p.N = c.K;
  p.K = n;
  p.f32 = c.f32;
  p.w_t = !c.linear;
  return p;
}
// Whether the ping-pong kernels' 32-bit offsets reach all of both operands.
bool spans_ok(const LinGemm& p) {
  const int64_t a = (p.a_t ? p.K : p.M) * p.lda * 2, w = (p.w_t ? p.N : p.K) * p.ldw * 2;
  return a < (int64_t{1} << 31) && w < (int64_t{1} << 31);
}
LinGemm dw_product(const CeSizes& c, int64_t n, int64_t rows) {
  LinGemm p;
  p.mode = c.f32 ? kModeOne : kModeScaled;
  p.groups = !c.f32;   // P's rows go on to a multiple of 64
  p.M = c.linear ? n : c.K;
  p.N = c.linear ? c.K : n;
  p.K = rows;
  p.f32 = c.f32;
  p.a_t = p.w_t = c.linear;
  return p;
}

// f(first column, columns, columns as multiplied) of each piece, until one fails.
template <typename F>
hipError_t each_piece(const CeSizes& c, const Backward& b, F&& f) {
  if (b.tail) {
    const hipError_t e = f(b.whole, c.V - b.whole, int64_t{64});
    if (e != hipSuccess) return e;
  }
  for (int64_t n = 0; n < b.whole; n += b.piece) {
    const int64_t cols = std::min(b.whole - n, b.piece);
    const hipError_t e = f(n, cols, b.pad ? up(cols, 64) : cols);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The slices that dX's product over n columns is cut into, and its tile, where that takes
// at most 0.9 of the estimated time (us).  A stage of 64 columns takes a 256 x 256 tile
// 1.45, smaller ones by their area and rate; a tile's fill and drain 4; every partial is
// written and read at 4.5 TB/s.  Uncut, fewer than 256 tiles of 128 x 128 run as 64 x 64
// ones, whose operands come through the caches, at 0.29 a stage for each of a CU's.
// MI355X, the backward uncut : cut (us): 4096 x 768 x 50000 1369 : 995, 2048 x 2048 x 50000 1373 :
// 1140, 512 x 4096 x 65000 1293 : 892, 128 x 4096 x 65536 645 : 598, 300 x 8192 x 10000 383 : 338.
TilePick slices_of(const CeSizes& c, int64_t n) {
  TilePick best{kTile256, 1};
  if (c.f32 || n % 64 || c.M < 128) return best;
  struct Kind {
    int tile, cols;
    double stage;
  };
  constexpr Kind kinds[] = {{kTile256, 256, 1.45}, {kTile128w, 128, 0.85}};
  const int64_t stages = n / 64, small = cut(c.M, 64) * cut(c.K, 64);
  const double each = static_cast<double>(c.M) * static_cast<double>(c.K) * 8.0 / 4.5e6;
  double uncut = 1e300, least = 1e300;
  for (const Kind& k : kinds) {
    const int64_t tiles = cut(c.M, 256) * cut(c.K, k.cols);
    for (int s = 1; s <= 16 && s * 8 <= stages; ++s) {
      const double t = static_cast<double>(cut(tiles * s, 256)) * (static_cast<double>(cut(stages, s)) * k.stage + 4.0);
      if (s == 1) {
        uncut = std::min(uncut, t);
      } else if (t + static_cast<double>(s) * each + 4.0 < least) {
        least = t + static_cast<double>(s) * each + 4.0;
        best = {k.tile, s};
      }
    }
  }
  if (cut(c.M, 128) * cut(c.K, 128) < 256) uncut = static_cast<double>(stages) * std::max(0.5, 0.29 * static_cast<double>(cut(small, 256)));
  if (least > 0.9 * uncut) best.splits = 1;
  return best;
}

Backward backward_plan(const CeSizes& c, const CeBackward& b) {
  Backward q;
  q.rows = up(c.M, 64);
  q.pad = padded(c, true);
  q.tail = !q.pad && !c.f32 && c.K % 32 == 0 && c.V % 64 && c.V > 64;
  q.whole = q.tail ? c.V / 64 * 64 : c.V;
  q.K = q.pad ? up(c.K, 64) : c.K;
  const int64_t grid = ((int64_t{1} << 22) - 1) / std::max<int64_t>(1, std::max(cut(c.M, 64), cut(c.K, 64))) * 64;
  int64_t most = b.piece > 0 ? std::max<int64_t>(64, b.piece / 64 * 64)
                             : std::max<int64_t>(8192, (int64_t{1} << 28) / std::max<int64_t>(1, q.rows));
  if (!c.f32 && (c.linear || q.pad)) most = std::min(most, ((int64_t{1} << 30) - 1) / q.K);
  most = std::max<int64_t>(64, std::min(std::min(most, grid), int64_t{1} << 25) / 64 * 64);
  const int64_t pieces = cut(q.whole, most);
  q.piece = up(cut(q.whole, pieces), 64);
  q.keeps = b.dX && !c.f32 && !b.dx_f32 && (pieces > 1 || q.tail);
  const int64_t es = c.f32 ? 4 : 2;
  int64_t joined = kTicketBytes, slices = 0;
  if (c.M > 0)
    (void)each_piece(c, q, [&](int64_t, int64_t cols, int64_t wide) {
      LinGemm z = logits_product(c, kModeProb, wide);
      z.K = q.K;
      joined = std::max(joined, lin_gemm_ws(z));
      if (b.dX) {
        LinGemm p = dx_product(c, wide, cols != wide || q.pad);
        joined = std::max(joined, lin_gemm_ws(p));
        p.lda = q.piece;
        p.ldw = c.linear ? q.K : p.groups ? wide : c.V;   // at least
        if (spans_ok(p)) slices = std::max<int64_t>(slices, slices_of(c, wide).splits);
      }
      if (b.dW) joined = std::max(joined, lin_gemm_ws(dw_product(c, cols, q.rows)));
      return hipSuccess;
    });
  q.scale = up(joined, kAlign);
  q.xt = q.scale + kAlign;
  q.p = q.xt + (b.dW ? up(c.K * q.rows * es, kAlign) : 0);
  q.acc = q.p + up(q.rows * q.piece * es, kAlign);
  q.x = q.acc + (q.keeps ? up(c.M * c.K * 4, kAlign) : 0);
  q.w = q.x + (q.K != c.K ? up(c.M * q.K * 2, kAlign) : 0);
  q.part = q.w + up(q.pad ? q.piece * q.K * 2 : q.tail ? 64 * c.K * 2 : 0, kAlign);
  q.total = q.part + (slices > 1 ? slices * c.M * c.K * 4 : 0);
  return q;
}

}  // namespace

bool ce_sizes_ok(const CeSizes& c) {
  // A piece of kTileCols columns against all rows, and of all of K against them, within the grid.
  return c.M < (int64_t{1} << 31) && c.V < (int64_t{1} << 31) && c.K < (int64_t{1} << 24) &&
         cut(c.M, 64) * (kTileCols / 64) < (int64_t{1} << 22) && cut(c.M, 64) * cut(c.K, 64) < (int64_t{1} << 22);
}

int64_t ce_forward_ws(const CeSizes& c) { return forward_bytes(c); }

hipError_t ce_forward_launch(const CeSizes& c, const CeOperands& o, float *stats, float *loss, float *lse, void *ws,
                             hipStream_t s) {
  const Forward f = forward_plan(c);
  char *base = static_cast<char *>(ws);
  float *part = reinterpret_cast<float *>(base + f.part), *logit = reinterpret_cast<float *>(base + f.logit);
  int64_t slots = 0;
  hipError_t e;
  CeJoin j;
  j.part = part;
  j.logit = logit;
  j.targets = o.targets;
  j.M = c.M;
  j.V = c.V;
  j.begin = o.begin;
  j.ignore = o.ignore;
  j.stats = stats;
  j.loss = loss;
  j.lse = lse;
  CePads copies;
  if (f.w != f.x) copies.pad[copies.num++] = pad_x(c, o, f.K, base + f.x);
  for (int64_t n = 0; n < c.V; n += f.piece) {
    const int64_t cols = std::min(f.piece, c.V - n), cols_pad = up(cols, 64);
    CeGemm p;
    static_cast<LinGemm&>(p) = logits_product(c, f.rows ? kModeOne : kModeStats, cols);
    p.a = o.X;
    p.lda = o.X_ld;
    p.w = weight_at(c, o.W, o.W_ld, n);
    p.ldw = o.W_ld;
    if (f.pad) {
      copies.pad[copies.num++] = pad_weight(c, o, n, cols, cols_pad, f.K, base + f.w);
      if ((e = pad(copies, s)) != hipSuccess) return e;
      copies.num = 0;
      p.w = base + f.w;
      p.ldw = c.linear ? f.K : cols_pad;
      p.K = f.K;
      p.groups = 1;
      if (f.w != f.x) {
        p.a = base + f.x;
        p.lda = f.K;
      }
    }
    const double flops = 2.0 * static_cast<double>(c.M) * static_cast<double>(cols) * static_cast<double>(c.K);
    if (f.rows) {
      p.c = base + f.logits;
      p.ldc = up(f.piece, 4);
      p.c_f32 = 1;
      e = timed(s, TP_KERNEL_GEMM1, flops, [&] { return lin_gemm_launch(p, s, ws, f.part); });
      if (e != hipSuccess) return e;
      CeLogits q;
      q.z = reinterpret_cast<const float *>(base + f.logits);
      q.ld = p.ldc;
      q.M = c.M;
      q.n = p.N;
      q.targets = o.targets;
      q.begin = o.begin + n;
      q.part = part + 2 * slots * c.M;
      q.logit = logit;
      e = timed(s, TP_KERNEL_REDUCE, 4.0 * static_cast<double>(c.M) * static_cast<double>(p.N), [&] { return ce_logits_launch(q, s); });
      slots += cut(p.N, kCeStatCols);
    } else {
      p.targets = o.targets;
      p.begin = o.begin + n;
      p.cols = cols;
      p.part = part;
      p.slot0 = slots;
      p.logit = logit;
      LinChoice h = lin_choose(&p, ws, f.small ? f.part : 0);
      if (f.small && h.tiles && columns_of(h) > 64) h.tile = {p.K % 64 ? kTile64k32 : kTile64, 1};
      if (f.small && h.tiles && c.M <= 32 && p.K % 64 == 0) h.tile.tile = kTile32;
      if (!f.small) {   // what the workspace was measured for
        if (h.tiles && columns_of(h) < 128) h.tile = {kTile128, 1};
        if (!h.tiles && !c.f32) h.staged = {128, 1, lin_tiles_count(p, 128, 128)};
      }
      e = timed(s, TP_KERNEL_GEMM1, flops, [&] { return h.tiles ? lin_tiles_stats(p, h.tile, s) : lin_staged_launch(p, h.staged, s); });
      slots += cut(p.N, columns_of(h));
    }
    if (e != hipSuccess) return e;
  }
  j.slots = slots;
  return timed(s, TP_KERNEL_REDUCE, 8.0 * static_cast<double>(slots) * static_cast<double>(c.M), [&] { return ce_join_launch(j, s); });
}

int64_t ce_backward_ws(const CeSizes& c, const CeBackward& b) { return b.dX || b.dW ? backward_plan(c, b).total : 0; }

hipError_t ce_backward_launch(const CeSizes& c, const CeOperands& o, const CeBackward& b, void *ws, hipStream_t s) {
  if (!b.dX && !b.dW) return hipSuccess;
  const Backward q = backward_plan(c, b);
  char *base = static_cast<char *>(ws);
  const int64_t es = c.f32 ? 4 : 2, dw_es = b.dw_f32 ? 4 : 2;
  const double MK = static_cast<double>(c.M) * static_cast<double>(c.K);
  float *scale = reinterpret_cast<float *>(base + q.scale);
  CeScale g;
  g.targets = o.targets;
  g.M = c.M;
  g.ignore = o.ignore;
  g.g = b.g;
  g.g_step = b.g_step;
  g.h = b.h;
  g.h_step = b.h_step;
  g.scale = c.f32 ? nullptr : scale;
  g.tickets = reinterpret_cast<uint32_t *>(base);
  hipError_t e;
  CePads copies;   // with the first piece's part of W
  if (c.M > 0 && q.K != c.K) copies.pad[copies.num++] = pad_x(c, o, q.K, base + q.x);
  const int64_t n0 = q.tail ? q.whole : 0;
  if (c.M > 0 && (q.pad || q.tail)) {
    const int64_t cols = std::min(c.V - n0, q.piece);
    copies.pad[copies.num++] = pad_weight(c, o, n0, cols, up(cols, 64), q.K, base + q.w);
  }
  if (b.dW && c.M > 0) {
    CeTranspose t;
    t.X = o.X;
    t.xt = base + q.xt;
    t.M = c.M;
    t.K = c.K;
    t.X_ld = o.X_ld;
    t.rows = q.rows;
    t.targets = o.targets;
    t.ignore = o.ignore;
    t.f32 = c.f32;
    t.scale = g;
    e = timed(s, TP_KERNEL_REDUCE, 2.0 * static_cast<double>(es) * MK + bytes_of(copies), [&] { return ce_transpose_launch(t, copies, s); });
  } else if ((e = pad(copies, s)) == hipSuccess) {
    e = timed(s, TP_KERNEL_REDUCE, 12.0 * static_cast<double>(c.M), [&] { return ce_scale_launch(g, s); });
  }
  if (e != hipSuccess) return e;
  // A product of the gradients: in bf16 multiplied by the scale again.
  auto gradient = [&](const LinGemm& of, int kind, double flops) {
    return timed(s, kind, flops, [&] {
      if (of.mode == kModeOne && !(of.a_t && of.w_t)) return lin_gemm_launch(of, s, ws, q.scale);
      ScaledGemm p;
      static_cast<LinGemm&>(p) = of;
      p.alpha = scale;
      const LinChoice h = lin_choose(&p, ws, q.scale);
      if (!h.tiles) return lin_staged_launch(p, h.staged, s);
      return p.a_t ? lin_tiles_wgrad(p, h.tile, s) : lin_tiles_scaled(p, h.tile, s);
    });
  };
  e = each_piece(c, q, [&](int64_t n, int64_t cols, int64_t wide) {
    const double flops = 2.0 * MK * static_cast<double>(cols);
    const bool copied = q.pad || cols != wide;
    const void *W = weight_at(c, o.W, o.W_ld, n);
    int64_t W_ld = o.W_ld;
    hipError_t r = hipSuccess;
    if (c.M > 0 && copied) {
      CePads next;
      next.pad[next.num++] = pad_weight(c, o, n, cols, wide, q.K, base + q.w);
      if (n != n0 && (r = pad(next, s)) != hipSuccess) return r;
      W = base + q.w;
      W_ld = c.linear ? q.K : wide;
    }
    if (c.M > 0) {
      CeGemm p;
      static_cast<LinGemm&>(p) = logits_product(c, kModeProb, wide);
      p.a = q.K != c.K ? base + q.x : o.X;
      p.lda = q.K != c.K ? q.K : o.X_ld;
      p.K = q.K;
      p.w = W;
      p.ldw = W_ld;
      p.cols = cols;
      p.c = base + q.p;
      p.ldc = q.piece;
      p.c_f32 = c.f32;
      p.targets = o.targets;
      p.begin = o.begin + n;
      p.ignore = o.ignore;
      p.lse = b.lse;
      p.g = b.g;
      p.g_step = b.g_step;
      p.h = b.h;
      p.h_step = b.h_step;
      p.scale = g.scale;
      p.pad_rows = q.rows;
      const LinChoice h = lin_choose(&p, ws, q.scale);
      r = timed(s, TP_KERNEL_GEMM1, flops, [&] { return h.tiles ? lin_tiles_prob(p, h.tile, s) : lin_staged_launch(p, h.staged, s); });
      if (r != hipSuccess) return r;
    }
    if (b.dX && c.M > 0) {
      LinGemm p = dx_product(c, wide, copied);
      p.a = base + q.p;
      p.lda = q.piece;
      p.w = W;
      p.ldw = W_ld;
      const bool first = n == (q.tail ? q.whole : 0), last = n < q.whole && n + cols == q.whole;
      float *sum = q.keeps ? reinterpret_cast<float *>(base + q.acc) : static_cast<float *>(b.dX);   // of the pieces so far
      const int64_t sum_ld = q.keeps ? c.K : b.dX_ld;
      const TilePick t = slices_of(c, wide);
      const LinChoice h = lin_choose(&p, nullptr, 0);
      if (t.splits > 1 && h.tiles && spans_ok(p)) {
        p.mode = kModeSlices;
        p.c = base + q.part;
        p.ldc = c.K;
        p.c_f32 = 1;
        r = timed(s, TP_KERNEL_GEMM_DGRAD, flops, [&] { return lin_tiles_slices(p, t, s); });
        if (r != hipSuccess) return r;
        CeSum u;
        u.part = reinterpret_cast<const float *>(base + q.part);
        u.slices = t.splits;
        u.alpha = scale;
        u.base = first ? nullptr : sum;
        u.base_ld = sum_ld;
        u.out = last ? b.dX : sum;
        u.out_ld = last ? b.dX_ld : sum_ld;
        u.out_f32 = last ? c.f32 || b.dx_f32 : 1;
        u.M = c.M;
        u.K = c.K;
        r = timed(s, TP_KERNEL_REDUCE, 4.0 * MK * (t.splits + 1), [&] { return ce_sum_launch(u, s); });
      } else {
        p.c = sum;
        p.ldc = sum_ld;
        p.c_f32 = q.keeps || b.dx_f32 || c.f32;
        p.acc_c = !first;
        r = gradient(p, TP_KERNEL_GEMM_DGRAD, flops);
        if (r == hipSuccess && last && q.keeps) {
          CeSum u;
          u.part = sum;
          u.slices = 1;
          u.out = b.dX;
          u.out_ld = b.dX_ld;
          u.M = c.M;
          u.K = c.K;
          r = timed(s, TP_KERNEL_REDUCE, 6.0 * MK, [&] { return ce_sum_launch(u, s); });
        }
      }
      if (r != hipSuccess) return r;
    }
    if (b.dW) {
      LinGemm p = dw_product(c, cols, q.rows);
      const void *P = base + q.p, *xt = base + q.xt;
      p.a = c.linear ? P : xt;
      p.lda = c.linear ? q.piece : q.rows;
      p.w = c.linear ? xt : P;
      p.ldw = c.linear ? q.rows : q.piece;
      p.c = static_cast<char *>(b.dW) + (c.linear ? n * b.dW_ld : n) * dw_es;
      p.ldc = b.dW_ld;
      p.c_f32 = b.dw_f32;
      p.acc_c = b.accumulate;
      if (c.M == 0) {   // a sum of nothing, on the general kernel
        p.mode = kModeOne;
        p.w_t = 0;
      }
      r = gradient(p, TP_KERNEL_GEMM_WGRAD, flops);
    }
    return r;
  });
  return e;
}

}  // namespace tpshard
