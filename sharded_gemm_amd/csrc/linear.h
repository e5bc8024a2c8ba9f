// Launch interface of the linear layer, the gated block, their backward passes
// and the gradient norm (linear_api.cpp validates and schedules; the kernels
// trust what reaches them).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace tpshard {

// What a product's two weight operands mean.
enum {
  kModeOne = 0,   // c = epi(A W)
  kModeDual = 1,  // gated: G = A W, U = A W2, c = act(G) * U; aux, aux2 keep G, U
  kModeCat = 2,   // c = A W + A2 W2 (one accumulator over both)
  kModePair = 3,  // c = A W and c2 = A2 W2, two products of one shape in one launch
};

// A workspace's first bytes are tickets (zero before and after every launch), its
// rest a launch's partials.  The tickets' place does not depend on the launch, so
// calls of any shapes may follow one another on one workspace.  (K is only split
// where a launch has a ticket for every tile.)
constexpr int64_t kTicketBytes = 4096, kMaxTickets = kTicketBytes / 4;

// C[M,N] = epi(A[M,K] W[K,N]), strides in elements.  As in GemmArgs, a_t: A is
// stored [K][lda]; w_t: W is stored [N][ldw].  The second operands share the
// first ones' shape and stride.  Epilogue, on the fp32 accumulator (kModeOne):
//   pre = acc + bias[n];  aux <- pre;  c <- act(pre) + res
// aux, res in the operands' type; c in it too, or fp32 (c_f32).  acc_c: c is
// added to (fp32 c).  Every optional pointer may be null.
struct LinGemm {
  const void *a = nullptr, *a2 = nullptr;
  const void *w = nullptr, *w2 = nullptr;
  void *c = nullptr, *c2 = nullptr;
  int64_t M = 0, N = 0, K = 0;
  int64_t lda = 0, ldw = 0, ldc = 0;
  const float *bias = nullptr;
  const void *res = nullptr;
  int64_t ldres = 0;
  void *aux = nullptr, *aux2 = nullptr;
  int64_t ldaux = 0;
  int32_t a_t = 0, w_t = 0;
  int32_t mode = kModeOne;
  int32_t f32 = 0;      // operands are fp32 (else bf16)
  int32_t act = 0;      // TP_ACT_*
  int32_t c_f32 = 0;    // c holds fp32 (always with f32)
  int32_t acc_c = 0;
  // Several workgroups to a tile: their partials and arrival counts.
  float *join = nullptr;
  uint32_t *tickets = nullptr;
};

// Which kernel takes a product, and how (linear_launch.cpp).

// Whether the grids of the kernels below reach every tile of [M, N].
bool lin_grid_ok(int64_t M, int64_t N);

// Bytes of workspace that the product can use: zeros, left zeroed where they have
// to be.
int64_t lin_gemm_ws(const LinGemm& p);
// Enqueues the product; ws may be null.
hipError_t lin_gemm_launch(const LinGemm& p, hipStream_t s, void *ws = nullptr, int64_t ws_bytes = 0);

// Tiles of a launch of bm x bn: kModeDual counts both weights' columns, kModePair both products.
inline int64_t lin_tiles_count(const LinGemm& p, int bm, int bn) {
  const int bno = p.mode == kModeDual ? bn / 2 : bn;
  return (p.M + bm - 1) / bm * ((p.N + bno - 1) / bno) * (p.mode == kModePair ? 2 : 1);
}

// The general kernel: any layout, alignment and size.
constexpr int kStagedRow = 128;   // bytes of K in a stage
struct StagedShape {
  int edge, splits;               // of a tile; workgroups that split a tile's K
  int64_t tiles;
};
hipError_t lin_staged_launch(const LinGemm& p, const StagedShape& h, hipStream_t s);

// The tiled bf16 kernels: 16-byte aligned operands and rows, K a multiple of 32, a
// row-contiguous operand of whole 8-column groups.
enum Tile { kTile256, kTile192, kTile128w, kTile128, kTile64, kTile64short, kTile64k32 };
struct TilePick {
  int tile;     // Tile
  int splits;   // workgroups that split a tile's K
};
hipError_t lin_tiles_one(const LinGemm& p, const TilePick& t, hipStream_t s);
hipError_t lin_tiles_dual(const LinGemm& p, const TilePick& t, hipStream_t s);
hipError_t lin_tiles_cat(const LinGemm& p, const TilePick& t, hipStream_t s);
hipError_t lin_tiles_pair(const LinGemm& p, const TilePick& t, hipStream_t s);

// The kernel for few rows.
constexpr int kRowsWaves = 8;   // of a workgroup, at most (measured against 4 and 16 with one token)
struct RowsShape {
  int g, waves, splits;         // columns of a tile (16 g), waves of a workgroup, workgroups of a tile
  int64_t tiles, cells;         // cells: floats of a workgroup's partial
};
hipError_t lin_rows_launch(const LinGemm& p, const RowsShape& h, hipStream_t s);

// ---- gradients at the activation -----------------------------------------
// kLinear: d_pre = d_out * act'(pre) (pre NULL: d_pre = d_out, not written) and,
// with colsum, the column sums of the unrounded d_pre.
// kGated : d_up = d_out * act(gate), d_gate = d_out * up * act'(gate).
struct ActGrad {
  const void *d_out = nullptr, *pre = nullptr, *up = nullptr;
  void *d_pre = nullptr, *d_up = nullptr;   // contiguous [M, N]
  int64_t M = 0, N = 0, ld_dout = 0, ld_pre = 0;
  float *parts = nullptr;                   // [slabs][N], or null
  float *colsum = nullptr;                  // [N]
  int32_t f32 = 0, act = 0, gated = 0, accumulate = 0;
  uint32_t *tickets = nullptr;              // kMaxTickets to set to zero, or null
};
// The launch: lanes of a row, tiles of columns, rows of a slab, and slabs (rows of `parts`).
struct ActGrid {
  int lanes;
  int64_t tiles, rows, slabs;
};
constexpr int kActThreads = 256, kActCols = 8;   // of a workgroup; columns of a lane
ActGrid act_grad_grid(int64_t M, int64_t N);
hipError_t act_grad_launch(const ActGrad& p, hipStream_t s);
hipError_t zero_tickets_launch(uint32_t *tickets, hipStream_t s);

// ---- gradient norm and clipping --------------------------------------------
constexpr int kGradParts = 1024;   // partial sums of squares of one call

struct GradTensor {
  const void *g;
  void *out;
  int64_t n;
  int32_t f32;
};
hipError_t grad_sumsq_launch(const GradTensor *ts, int64_t num, double *parts, hipStream_t s);
// parts: `ranks` blocks of kGradParts.
hipError_t grad_clip_launch(const GradTensor *ts, int64_t num, const double *parts, int64_t ranks, double max_norm,
                            double eps, float *norm_out, hipStream_t s);

}  // namespace tpshard
