// Launch interface of the vocabulary cross entropy (ce_api.cpp validates, ce_launch.cpp
// chooses kernels, pieces and workspaces; the kernels trust what reaches them).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "linear.h"

namespace tpshard {

// ---- products on the vocabulary (ce_launch.cpp) ---------------------------------

// X [M, K] against W's V columns, in W's layout.
struct CeSizes {
  int64_t M, V, K;
  int32_t f32, linear;   // linear: W is [V, K]
};
struct CeOperands {
  const void *X, *W;
  int64_t X_ld, W_ld;
  const int64_t *targets;
  int64_t begin, ignore;
};

// Whether the kernels' indexes and grids reach all of it.
bool ce_sizes_ok(const CeSizes& c);

// Workspace of the forward: tickets (zero before and after every call), row
// statistics, target logits and, for few rows, the logits of the rows.
int64_t ce_forward_ws(const CeSizes& c);
// stats, loss and lse as in tp_linear_ce_args.
hipError_t ce_forward_launch(const CeSizes& c, const CeOperands& o, float *stats, float *loss, float *lse, void *ws,
                             hipStream_t s);

struct CeBackward {
  const float *lse = nullptr, *g = nullptr, *h = nullptr;
  int64_t g_step = 0, h_step = 0;
  void *dX = nullptr, *dW = nullptr;
  int64_t dX_ld = 0, dW_ld = 0;
  int32_t dx_f32 = 0, dw_f32 = 0, accumulate = 0;
  int64_t piece = 0;   // columns of a piece at most; 0: chosen
};
int64_t ce_backward_ws(const CeSizes& c, const CeBackward& b);
hipError_t ce_backward_launch(const CeSizes& c, const CeOperands& o, const CeBackward& b, void *ws, hipStream_t s);

// ---- the other kernels (ce.hip) --------------------------------------------------

// Logits z [M, n] of ids `begin` on: a pair for every kCeStatCols of them, and the targets' logits.
constexpr int kCeStatCols = 2048;
struct CeLogits {
  const float *z = nullptr;
  int64_t M = 0, n = 0, ld = 0;
  const int64_t *targets = nullptr;
  int64_t begin = 0;
  float *part = nullptr, *logit = nullptr;
};
hipError_t ce_logits_launch(const CeLogits& p, hipStream_t s);

// The pairs of every row joined over its slots; each output may be null.
struct CeJoin {
  const float *part = nullptr;    // [slots][M] pairs
  const float *logit = nullptr;   // [M]: those of targets in [begin, begin + V)
  const int64_t *targets = nullptr;
  int64_t M = 0, V = 0, slots = 0, begin = 0, ignore = 0;
  float *stats = nullptr, *loss = nullptr, *lse = nullptr;
};
hipError_t ce_join_launch(const CeJoin& p, hipStream_t s);

// Every piece's statistics joined: stats [pieces][3][M].
hipError_t ce_pieces_launch(const float *stats, int64_t pieces, int64_t M, const int64_t *targets, int64_t ignore,
                            float *loss, float *lse, hipStream_t s);

// Before the products: *scale (optional) <- what the gradient at the logits is divided by,
// the largest finite |g| (where it is at least 2^-64 of the largest |h|, else that) over tokens that are not
// ignored, 1 where there is none; tickets (kMaxTickets) <- 0.
struct CeScale {
  const int64_t *targets = nullptr;
  int64_t M = 0, ignore = 0, g_step = 0, h_step = 0;
  const float *g = nullptr, *h = nullptr;
  float *scale = nullptr;
  uint32_t *tickets = nullptr;
};
hipError_t ce_scale_launch(const CeScale& p, hipStream_t s);

// xt [K, rows] <- the transpose of X, zero for ignored targets and for m >= M; and ce_scale_launch's work beside it.
struct CeTranspose {
  const void *X = nullptr;
  void *xt = nullptr;
  int64_t M = 0, K = 0, X_ld = 0, rows = 0;
  const int64_t *targets = nullptr;
  int64_t ignore = 0;
  int32_t f32 = 0;
  CeScale scale;
};

// to [rows, cols] (bf16, contiguous, both multiples of 8) <- from [m, n] at stride ld, zero beyond.
struct CePad {
  const void *from = nullptr;
  void *to = nullptr;
  int64_t m = 0, n = 0, ld = 0, rows = 0, cols = 0;
};
// Up to two of them in one launch, which nothing orders; beside a transpose too (`pads` may be empty).
struct CePads {
  CePad pad[2];
  int32_t num = 0;
};
hipError_t ce_pad_launch(const CePads& p, hipStream_t s);
hipError_t ce_transpose_launch(const CeTranspose& p, const CePads& pads, hipStream_t s);

// out [M, K] <- base + *alpha (null: 1) times the sum over s < slices, in order, of part[s]; part [slices][M][K] fp32,
// base (optional) fp32, out bf16 or fp32 (then it may be base).
struct CeSum {
  const float *part = nullptr, *base = nullptr, *alpha = nullptr;
  void *out = nullptr;
  int64_t M = 0, K = 0, slices = 0, base_ld = 0, out_ld = 0;
  int32_t out_f32 = 0;
};
hipError_t ce_sum_launch(const CeSum& p, hipStream_t s);

}  // namespace tpshard
