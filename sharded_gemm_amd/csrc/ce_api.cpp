// C ABI of the vocabulary cross entropy: validation, then the launches.  A call checks
// every argument before it enqueues anything.
#include "args.h"
#include "ce.h"
#include "timing.h"

namespace tpshard {
namespace {

constexpr int64_t kMaxPieces = 64;

int check_sizes(int32_t dtype, int32_t layout, int64_t M, int64_t V, int64_t K, CeSizes *c) {
  if (!dtype_size(dtype)) return fail(TP_ERR_ARG, "unknown dtype %d", dtype);
  if (layout != TP_WEIGHTS_MATH && layout != TP_WEIGHTS_LINEAR)
    return fail(TP_ERR_ARG, "unknown weight_layout %d", layout);
  if (M < 0 || V < 1 || K < 1) return fail(TP_ERR_ARG, "need M >= 0, V >= 1 and K >= 1");
  *c = CeSizes{M, V, K, dtype == TP_F32, layout == TP_WEIGHTS_LINEAR};
  if (!ce_sizes_ok(*c)) return fail(TP_ERR_UNSUPPORTED, "sizes exceed the kernels' index range or grid");
  return TP_OK;
}

int check_begin(int64_t begin, int64_t V) {
  if (begin < 0 || begin > INT64_MAX - V) return fail(TP_ERR_ARG, "vocab_begin = %lld", (long long)begin);
  return TP_OK;
}

// A vector of n elements of es bytes.
int take_vec(Mat *m, const char *name, const void *p, int64_t n, int64_t es, bool needed) {
  *m = Mat{p, 1, n, n, es, name};
  if (!p) return needed ? fail(TP_ERR_ARG, "%s must be non-NULL", name) : TP_OK;
  if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(es)) return fail(TP_ERR_ARG, "%s is not aligned to its elements", name);
  return TP_OK;
}

int check_stride(int64_t stride, const char *name) {
  if (stride != 0 && stride != 1) return fail(TP_ERR_ARG, "%s must be 0 or 1", name);
  return TP_OK;
}

CeBackward asked(const tp_linear_ce_bwd_args *a) {
  CeBackward b;
  b.lse = a->lse;
  b.g = a->dloss;
  b.g_step = a->dloss_stride;
  b.h = a->dlse;
  b.h_step = a->dlse_stride;
  b.dX = a->dX;
  b.dW = a->dW;
  b.dx_f32 = a->dx_dtype == TP_F32;
  b.dw_f32 = a->dw_dtype == TP_F32;
  b.accumulate = a->accumulate;
  b.piece = a->piece;
  return b;
}

int check_backward(const tp_linear_ce_bwd_args *a, CeSizes *c) {
  int rc = check_sizes(a->dtype, a->weight_layout, a->M, a->V, a->K, c);
  if (rc == TP_OK) rc = check_out_dtype(a->dx_dtype, a->dtype, "dx_dtype");
  if (rc == TP_OK && a->piece < 0) rc = fail(TP_ERR_ARG, "piece = %lld", (long long)a->piece);
  return rc;
}

}  // namespace
}  // namespace tpshard

using namespace tpshard;

extern "C" {

int tp_linear_ce_ws(const tp_linear_ce_args *a, int64_t *bytes) {
  clear_error();
  if (!a || !bytes) return fail(TP_ERR_ARG, "args or bytes is NULL");
  CeSizes c;
  const int rc = check_sizes(a->dtype, a->weight_layout, a->M, a->V, a->K, &c);
  if (rc != TP_OK) return rc;
  *bytes = ce_forward_ws(c);
  return TP_OK;
}

int tp_linear_ce(const tp_linear_ce_args *a, tp_stream_t stream) {
  clear_error();
  if (!a) return fail(TP_ERR_ARG, "args is NULL");
  CeSizes c;
  int rc = check_sizes(a->dtype, a->weight_layout, a->M, a->V, a->K, &c);
  if (rc == TP_OK) rc = check_begin(a->vocab_begin, a->V);
  if (rc != TP_OK) return rc;
  const int64_t es = dtype_size(a->dtype);
  const bool any = a->M > 0;
  if (any && !a->stats && !a->loss && !a->lse) return fail(TP_ERR_ARG, "neither stats, loss nor lse is asked for");
  Mat x, w, t, st, lo, le;
  if ((rc = take(&x, "X", a->X, a->M, a->K, a->X_ld, es, any)) != TP_OK ||
      (rc = take(&w, "W", a->W, c.linear ? a->V : a->K, c.linear ? a->K : a->V, a->W_ld, es, any)) != TP_OK ||
      (rc = take_vec(&t, "targets", a->targets, a->M, 8, any)) != TP_OK ||
      (rc = take_vec(&st, "stats", a->stats, 3 * a->M, 4, false)) != TP_OK ||
      (rc = take_vec(&lo, "loss", a->loss, a->M, 4, false)) != TP_OK ||
      (rc = take_vec(&le, "lse", a->lse, a->M, 4, false)) != TP_OK)
    return rc;
  const int64_t need = ce_forward_ws(c);
  if ((rc = check_ws(a->ws, a->ws_bytes, need)) != TP_OK) return rc;
  const Mat wsm{need ? a->ws : nullptr, 1, need, need, 1, "ws"};
  if ((rc = disjoint({x, w, t}, {st, lo, le, wsm})) != TP_OK) return rc;
  if (!any) return TP_OK;
  const CeOperands o{x.p, w.p, x.ld, w.ld, a->targets, a->vocab_begin, a->ignore_index};
  const hipError_t e = ce_forward_launch(c, o, a->stats, a->loss, a->lse, a->ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TP_OK : hip_fail(e, "cross entropy launch");
}

int tp_ce_join(const float *stats, int64_t pieces, int64_t M, const int64_t *targets, int64_t ignore_index, float *loss,
               float *lse, tp_stream_t stream) {
  clear_error();
  if (pieces < 1 || pieces > kMaxPieces)
    return fail(TP_ERR_ARG, "pieces = %lld outside [1, %lld]", (long long)pieces, (long long)kMaxPieces);
  if (M < 0) return fail(TP_ERR_ARG, "need M >= 0");
  if (M >= kMaxDim) return fail(TP_ERR_UNSUPPORTED, "M = %lld exceeds the kernels' range", (long long)M);
  if (M > 0 && !loss && !lse) return fail(TP_ERR_ARG, "neither loss nor lse is asked for");
  Mat st, t, lo, le;
  int rc;
  if ((rc = take_vec(&st, "stats", stats, 3 * pieces * M, 4, M > 0)) != TP_OK ||
      (rc = take_vec(&t, "targets", targets, M, 8, M > 0)) != TP_OK ||
      (rc = take_vec(&lo, "loss", loss, M, 4, false)) != TP_OK || (rc = take_vec(&le, "lse", lse, M, 4, false)) != TP_OK ||
      (rc = disjoint({st, t}, {lo, le})) != TP_OK)
    return rc;
  if (M == 0) return TP_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipEvent_t t0 = timing_begin(s);
  const hipError_t e = ce_pieces_launch(stats, pieces, M, targets, ignore_index, loss, lse, s);
  if (e != hipSuccess) return hip_fail(e, "cross entropy join launch");
  timing_end(t0, s, TP_KERNEL_REDUCE, 12.0 * static_cast<double>(pieces) * static_cast<double>(M));
  return TP_OK;
}

int tp_linear_ce_backward_ws(const tp_linear_ce_bwd_args *a, int64_t *bytes) {
  clear_error();
  if (!a || !bytes) return fail(TP_ERR_ARG, "args or bytes is NULL");
  CeSizes c;
  const int rc = check_backward(a, &c);
  if (rc != TP_OK) return rc;
  *bytes = ce_backward_ws(c, asked(a));
  return TP_OK;
}

int tp_linear_ce_backward(const tp_linear_ce_bwd_args *a, tp_stream_t stream) {
  clear_error();
  if (!a) return fail(TP_ERR_ARG, "args is NULL");
  CeSizes c;
  int rc = check_backward(a, &c);
  if (rc == TP_OK) rc = check_out_dtype(a->dw_dtype, a->dtype, "dw_dtype");
  if (rc == TP_OK) rc = check_begin(a->vocab_begin, a->V);
  if (rc == TP_OK && a->dloss) rc = check_stride(a->dloss_stride, "dloss_stride");
  if (rc == TP_OK && a->dlse) rc = check_stride(a->dlse_stride, "dlse_stride");
  if (rc != TP_OK) return rc;
  if (a->accumulate != 0 && a->accumulate != 1) return fail(TP_ERR_ARG, "accumulate must be 0 or 1");
  if (a->accumulate && a->dW && a->dw_dtype != TP_F32) return fail(TP_ERR_ARG, "accumulate needs an fp32 dW");
  const int64_t es = dtype_size(a->dtype), wr = c.linear ? a->V : a->K, wc = c.linear ? a->K : a->V;
  const bool any = a->M > 0 && (a->dX || a->dW);
  Mat x, w, t, l, g, h, dx, dw;
  if ((rc = take(&x, "X", a->X, a->M, a->K, a->X_ld, es, any)) != TP_OK ||
      (rc = take(&w, "W", a->W, wr, wc, a->W_ld, es, any)) != TP_OK ||
      (rc = take_vec(&t, "targets", a->targets, a->M, 8, any)) != TP_OK ||
      (rc = take_vec(&l, "lse", a->lse, a->M, 4, any)) != TP_OK ||
      (rc = take_vec(&g, "dloss", a->dloss, a->dloss_stride ? a->M : 1, 4, false)) != TP_OK ||
      (rc = take_vec(&h, "dlse", a->dlse, a->dlse_stride ? a->M : 1, 4, false)) != TP_OK ||
      (rc = take(&dx, "dX", a->dX, a->M, a->K, a->dX_ld, dtype_size(a->dx_dtype), false)) != TP_OK ||
      (rc = take(&dw, "dW", a->dW, wr, wc, a->dW_ld, dtype_size(a->dw_dtype), false)) != TP_OK)
    return rc;
  CeBackward b = asked(a);
  const int64_t need = ce_backward_ws(c, b);
  if ((rc = check_ws(a->ws, a->ws_bytes, need)) != TP_OK) return rc;
  const Mat wsm{need ? a->ws : nullptr, 1, need, need, 1, "ws"};
  if ((rc = disjoint({x, w, t, l, g, h}, {dx, dw, wsm})) != TP_OK) return rc;
  b.dX_ld = dx.ld;
  b.dW_ld = dw.ld;
  const CeOperands o{x.p, w.p, x.ld, w.ld, a->targets, a->vocab_begin, a->ignore_index};
  const hipError_t e = ce_backward_launch(c, o, b, a->ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TP_OK : hip_fail(e, "cross entropy backward launch");
}

}  // extern "C"
