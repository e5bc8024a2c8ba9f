// C ABI of the linear layer, the gated block, their backward passes and the
// gradient norm: validation, then the launches.  As in api.cpp, a call checks
// every argument before it enqueues anything.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>
#include <new>
#include <vector>

#include "args.h"
#include "linear.h"
#include "timing.h"

namespace tpshard {
namespace {

constexpr int64_t kMaxRanks = 64;
constexpr int64_t kWsAlign = 256;
static_assert(kGradParts == TP_GRAD_PARTS, "the header's count");

int check_common(int32_t dtype, int32_t act, int32_t layout, int64_t M, int64_t N, int64_t K, const char *n_name) {
  if (!dtype_size(dtype)) return fail(TP_ERR_ARG, "unknown dtype %d", dtype);
  if (act < TP_ACT_NONE || act > TP_ACT_RELU) return fail(TP_ERR_ARG, "unknown act %d", act);
  if (layout != TP_WEIGHTS_MATH && layout != TP_WEIGHTS_LINEAR)
    return fail(TP_ERR_ARG, "unknown weight_layout %d", layout);
  if (M < 0 || N < 1 || K < 1) return fail(TP_ERR_ARG, "need M >= 0, %s >= 1 and K >= 1", n_name);
  if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim || !lin_grid_ok(M, N) || !lin_grid_ok(M, K) || !lin_grid_ok(K, N))
    return fail(TP_ERR_UNSUPPORTED, "sizes exceed the kernels' index range or grid");
  return TP_OK;
}

int launch(const LinGemm& p, hipStream_t s, int kind, double flops, const char *what, void *ws = nullptr,
           int64_t ws_bytes = 0) {
  hipEvent_t t0 = timing_begin(s);
  const hipError_t e = lin_gemm_launch(p, s, ws, ws_bytes);
  if (e != hipSuccess) return hip_fail(e, what);
  timing_end(t0, s, kind, flops);
  return TP_OK;
}

// The backward's products (pointers to the gradients at the activation apart).
// dX [M, K] = dPre [M, N] W^T; with two weights both, in one accumulator.
LinGemm dx_product(int64_t M, int64_t N, int64_t K, int32_t dtype, bool linear, bool gated) {
  LinGemm p;
  p.mode = gated ? kModeCat : kModeOne;
  p.w_t = !linear;
  p.M = M;
  p.N = K;
  p.K = N;
  p.f32 = dtype == TP_F32;
  return p;
}
// dW: math [K, N] = X^T dPre; linear [N, K] = dPre^T X.
LinGemm dw_product(int64_t M, int64_t N, int64_t K, int32_t dtype, bool linear, bool gated) {
  LinGemm p;
  p.mode = gated ? kModePair : kModeOne;
  p.a_t = 1;
  p.M = linear ? N : K;
  p.N = linear ? K : N;
  p.K = M;
  p.f32 = dtype == TP_F32;
  return p;
}

// Workspace of a backward: the gradients at the activation in the operands' type
// (where a product reads them) and the bias gradient's partial rows, which a call
// cannot do without, then what the products need to split K, used where it is
// there (and, without the rest, aligned).
struct BwdWs {
  int64_t d_pre = 0, d_up = 0, parts = 0, join = 0, total = 0;   // offsets; total: bytes
  bool keeps = false;                                            // d_pre is written
  int64_t used(const void *ws, int64_t bytes) const {
    return ws && bytes >= total && (reinterpret_cast<uintptr_t>(ws) & 15) == 0 ? total : join;
  }
};
BwdWs linear_ws(const tp_linear_bwd_args *a) {
  const bool linear = a->weight_layout == TP_WEIGHTS_LINEAR;
  BwdWs w;
  w.keeps = a->act != TP_ACT_NONE && (a->dX || a->dW) && a->M > 0;
  w.parts = w.keeps ? round_up(a->M * a->N * dtype_size(a->dtype), kWsAlign) : 0;
  w.join = w.parts + (a->dbias ? round_up(act_grad_grid(a->M, a->N).slabs * a->N * 4, kWsAlign) : 0);
  const int64_t x = a->dX ? lin_gemm_ws(dx_product(a->M, a->N, a->K, a->dtype, linear, false)) : 0;
  const int64_t y = a->dW ? lin_gemm_ws(dw_product(a->M, a->N, a->K, a->dtype, linear, false)) : 0;
  w.total = w.join + std::max(x, y);
  return w;
}
// (Enough for either weight layout and any of the gradients.)
BwdWs gated_ws(int64_t M, int64_t F, int64_t K, int32_t dtype) {
  BwdWs w;
  w.keeps = M > 0;
  w.d_up = round_up(M * F * dtype_size(dtype), kWsAlign);
  w.join = 2 * w.d_up;
  int64_t most = 0;
  for (const bool linear : {false, true})
    most = std::max(most, std::max(lin_gemm_ws(dx_product(M, F, K, dtype, linear, true)),
                                   lin_gemm_ws(dw_product(M, F, K, dtype, linear, true))));
  w.total = w.join + most;
  return w;
}

}  // namespace
}  // namespace tpshard

using namespace tpshard;

extern "C" {

int tp_linear_ws(const tp_linear_args *a, int64_t *bytes) {
  clear_error();
  if (!a || !bytes) return fail(TP_ERR_ARG, "args or bytes is NULL");
  const int rc = check_common(a->dtype, a->act, a->weight_layout, a->M, a->N, a->K, "N");
  if (rc != TP_OK) return rc;
  LinGemm p;
  p.M = a->M;
  p.N = a->N;
  p.K = a->K;
  p.w_t = a->weight_layout == TP_WEIGHTS_LINEAR;
  p.f32 = a->dtype == TP_F32;
  *bytes = lin_gemm_ws(p);
  return TP_OK;
}

int tp_gated_linear_ws(const tp_gated_args *a, int64_t *bytes) {
  clear_error();
  if (!a || !bytes) return fail(TP_ERR_ARG, "args or bytes is NULL");
  const int rc = check_common(a->dtype, a->act, a->weight_layout, a->M, a->F, a->K, "F");
  if (rc != TP_OK) return rc;
  LinGemm p;
  p.mode = kModeDual;
  p.M = a->M;
  p.N = a->F;
  p.K = a->K;
  p.w_t = a->weight_layout == TP_WEIGHTS_LINEAR;
  p.f32 = a->dtype == TP_F32;
  *bytes = lin_gemm_ws(p);
  return TP_OK;
}

int tp_linear(const tp_linear_args *a, tp_stream_t stream) {
  clear_error();
  if (!a) return fail(TP_ERR_ARG, "args is NULL");
  int rc = check_common(a->dtype, a->act, a->weight_layout, a->M, a->N, a->K, "N");
  if (rc == TP_OK) rc = check_out_dtype(a->out_dtype, a->dtype, "out_dtype");
  if (rc != TP_OK) return rc;
  const int64_t M = a->M, N = a->N, K = a->K, es = dtype_size(a->dtype), oes = dtype_size(a->out_dtype);
  const bool linear = a->weight_layout == TP_WEIGHTS_LINEAR, any = M > 0;
  Mat x, w, b, r, o, pre, wsm;
  if ((rc = take(&x, "X", a->X, M, K, a->X_ld, es, any)) != TP_OK ||
      (rc = take(&w, "W", a->W, linear ? N : K, linear ? K : N, a->W_ld, es, any)) != TP_OK ||
      (rc = take(&b, "bias", a->bias, 1, N, 0, 4, false)) != TP_OK ||
      (rc = take(&r, "residual", a->residual, M, N, a->residual_ld, es, false)) != TP_OK ||
      (rc = take(&o, "out", a->out, M, N, a->out_ld, oes, any)) != TP_OK ||
      (rc = take(&pre, "pre_out", a->pre_out, M, N, a->pre_ld, es, false)) != TP_OK ||
      (rc = take_ws(&wsm, a->ws, a->ws_bytes)) != TP_OK)
    return rc;
  // Each output element is written by the lane that read the residual's.
  const bool in_place = r.p && r.p == o.p && r.ld == o.ld && es == oes;
  if ((rc = disjoint({x, w, b, in_place ? Mat{} : r}, {o, pre, wsm})) != TP_OK) return rc;
  if (in_place && (rc = disjoint({r}, {pre})) != TP_OK) return rc;
  if (!any) return TP_OK;
  LinGemm p;
  p.a = x.p;
  p.lda = x.ld;
  p.w = w.p;
  p.ldw = w.ld;
  p.w_t = linear;
  p.c = a->out;
  p.ldc = o.ld;
  p.M = M;
  p.N = N;
  p.K = K;
  p.bias = a->bias;
  p.res = r.p;
  p.ldres = r.ld;
  p.aux = a->pre_out;
  p.ldaux = pre.ld;
  p.act = a->act;
  p.f32 = a->dtype == TP_F32;
  p.c_f32 = a->out_dtype == TP_F32;
  return launch(p, static_cast<hipStream_t>(stream), TP_KERNEL_GEMM1, 2.0 * M * N * K, "linear launch", a->ws,
                a->ws_bytes);
}

int tp_linear_backward_ws(const tp_linear_bwd_args *a, int64_t *bytes) {
  clear_error();
  if (!a || !bytes) return fail(TP_ERR_ARG, "args or bytes is NULL");
  const int rc = check_common(a->dtype, a->act, a->weight_layout, a->M, a->N, a->K, "N");
  if (rc != TP_OK) return rc;
  *bytes = linear_ws(a).total;
  return TP_OK;
}

int tp_linear_backward(const tp_linear_bwd_args *a, tp_stream_t stream) {
  clear_error();
  if (!a) return fail(TP_ERR_ARG, "args is NULL");
  int rc = check_common(a->dtype, a->act, a->weight_layout, a->M, a->N, a->K, "N");
  if (rc == TP_OK) rc = check_out_dtype(a->dx_dtype, a->dtype, "dx_dtype");
  if (rc == TP_OK) rc = check_out_dtype(a->dw_dtype, a->dtype, "dw_dtype");
  if (rc != TP_OK) return rc;
  if (a->accumulate != 0 && a->accumulate != 1) return fail(TP_ERR_ARG, "accumulate must be 0 or 1");
  if (a->accumulate && a->dW && a->dw_dtype != TP_F32) return fail(TP_ERR_ARG, "accumulate needs an fp32 dW");
  const int64_t M = a->M, N = a->N, K = a->K, es = dtype_size(a->dtype);
  const bool linear = a->weight_layout == TP_WEIGHTS_LINEAR, any = M > 0, acts = a->act != TP_ACT_NONE;
  const int64_t wr = linear ? N : K, wc = linear ? K : N;
  Mat x, w, d, pre, dx, dw, db;
  if ((rc = take(&x, "X", a->X, M, K, a->X_ld, es, any && a->dW)) != TP_OK ||
      (rc = take(&w, "W", a->W, wr, wc, a->W_ld, es, any && a->dX)) != TP_OK ||
      (rc = take(&d, "dOut", a->dOut, M, N, a->dOut_ld, es, any)) != TP_OK ||
      (rc = take(&pre, "pre", acts ? a->pre : nullptr, M, N, acts ? a->pre_ld : 0, es, any && acts)) != TP_OK ||
      (rc = take(&dx, "dX", a->dX, M, K, a->dX_ld, dtype_size(a->dx_dtype), false)) != TP_OK ||
      (rc = take(&dw, "dW", a->dW, wr, wc, a->dW_ld, dtype_size(a->dw_dtype), false)) != TP_OK ||
      (rc = take(&db, "dbias", a->dbias, 1, N, 0, 4, false)) != TP_OK)
    return rc;
  const BwdWs ws = linear_ws(a);
  if ((rc = check_ws(a->ws, a->ws_bytes, ws.join)) != TP_OK) return rc;
  const int64_t used = ws.used(a->ws, a->ws_bytes);
  const Mat wsm{used ? a->ws : nullptr, 1, used, used, 1, "ws"};
  if ((rc = disjoint({x, w, d, pre}, {dx, dw, db, wsm})) != TP_OK) return rc;

  hipStream_t s = static_cast<hipStream_t>(stream);
  char *base = static_cast<char *>(a->ws);
  uint32_t *tickets = used > ws.join ? reinterpret_cast<uint32_t *>(base + ws.join) : nullptr;
  const void *d_pre = d.p;
  int64_t ld_pre = d.ld;
  if (ws.keeps || a->dbias) {
    ActGrad g;
    g.d_out = d.p;
    g.ld_dout = d.ld;
    g.pre = acts ? pre.p : nullptr;
    g.ld_pre = pre.ld;
    g.d_pre = ws.keeps ? base : nullptr;
    g.M = M;
    g.N = N;
    g.parts = a->dbias && any ? reinterpret_cast<float *>(base + ws.parts) : nullptr;
    g.colsum = a->dbias;
    g.f32 = a->dtype == TP_F32;
    g.act = a->act;
    g.accumulate = a->accumulate;
    g.tickets = tickets;
    hipEvent_t t0 = timing_begin(s);
    const hipError_t e = act_grad_launch(g, s);
    if (e != hipSuccess) return hip_fail(e, "activation gradient launch");
    timing_end(t0, s, TP_KERNEL_REDUCE,
               static_cast<double>(es) * M * N * (1 + acts + ws.keeps) + (a->dbias ? 4.0 * N : 0.0));
    if (ws.keeps) {
      d_pre = base;
      ld_pre = N;
    }
  } else if (tickets) {
    const hipError_t e = zero_tickets_launch(tickets, s);
    if (e != hipSuccess) return hip_fail(e, "ticket launch");
  }
  const double flops = 2.0 * M * N * K;
  if (a->dX && any) {
    LinGemm p = dx_product(M, N, K, a->dtype, linear, false);
    p.a = d_pre;
    p.lda = ld_pre;
    p.w = w.p;
    p.ldw = w.ld;
    p.c = a->dX;
    p.ldc = dx.ld;
    p.c_f32 = a->dx_dtype == TP_F32;
    if ((rc = launch(p, s, TP_KERNEL_GEMM_DGRAD, flops, "dX launch", tickets, used - ws.join)) != TP_OK) return rc;
  }
  if (a->dW) {
    LinGemm p = dw_product(M, N, K, a->dtype, linear, false);
    p.a = linear ? d_pre : x.p;
    p.lda = linear ? ld_pre : x.ld;
    p.w = linear ? x.p : d_pre;
    p.ldw = linear ? x.ld : ld_pre;
    p.c = a->dW;
    p.ldc = dw.ld;
    p.c_f32 = a->dw_dtype == TP_F32;
    p.acc_c = a->accumulate;
    if ((rc = launch(p, s, TP_KERNEL_GEMM_WGRAD, flops, "dW launch", tickets, used - ws.join)) != TP_OK) return rc;
  }
  return TP_OK;
}

int tp_gated_linear(const tp_gated_args *a, tp_stream_t stream) {
  clear_error();
  if (!a) return fail(TP_ERR_ARG, "args is NULL");
  int rc = check_common(a->dtype, a->act, a->weight_layout, a->M, a->F, a->K, "F");
  if (rc != TP_OK) return rc;
  const int64_t M = a->M, F = a->F, K = a->K, es = dtype_size(a->dtype);
  const bool linear = a->weight_layout == TP_WEIGHTS_LINEAR, any = M > 0;
  const int64_t wr = linear ? F : K, wc = linear ? K : F;
  Mat x, wg, wu, o, g, u, wsm;
  if ((rc = take(&x, "X", a->X, M, K, a->X_ld, es, any)) != TP_OK ||
      (rc = take(&wg, "W_gate", a->W_gate, wr, wc, a->W_ld, es, any)) != TP_OK ||
      (rc = take(&wu, "W_up", a->W_up, wr, wc, a->W_ld, es, any)) != TP_OK ||
      (rc = take(&o, "out", a->out, M, F, a->out_ld, es, any)) != TP_OK ||
      (rc = take(&g, "gate_out", a->gate_out, M, F, a->keep_ld, es, false)) != TP_OK ||
      (rc = take(&u, "up_out", a->up_out, M, F, a->keep_ld, es, false)) != TP_OK ||
      (rc = take_ws(&wsm, a->ws, a->ws_bytes)) != TP_OK)
    return rc;
  if (!g.p != !u.p) return fail(TP_ERR_ARG, "gate_out and up_out: both or neither");
  if ((rc = disjoint({x, wg, wu}, {o, g, u, wsm})) != TP_OK) return rc;
  if (!any) return TP_OK;
  LinGemm p;
  p.mode = kModeDual;
  p.a = x.p;
  p.lda = x.ld;
  p.w = wg.p;
  p.w2 = wu.p;
  p.ldw = wg.ld;
  p.w_t = linear;
  p.c = a->out;
  p.ldc = o.ld;
  p.M = M;
  p.N = F;
  p.K = K;
  p.aux = a->gate_out;
  p.aux2 = a->up_out;
  p.ldaux = g.ld;
  p.act = a->act;
  p.f32 = p.c_f32 = a->dtype == TP_F32;
  return launch(p, static_cast<hipStream_t>(stream), TP_KERNEL_GEMM1, 4.0 * M * F * K, "gated linear launch",
                a->ws, a->ws_bytes);
}

int tp_gated_linear_backward_ws(const tp_gated_bwd_args *a, int64_t *bytes) {
  clear_error();
  if (!a || !bytes) return fail(TP_ERR_ARG, "args or bytes is NULL");
  const int rc = check_common(a->dtype, a->act, a->weight_layout, a->M, a->F, a->K, "F");
  if (rc != TP_OK) return rc;
  *bytes = gated_ws(a->M, a->F, a->K, a->dtype).total;
  return TP_OK;
}

int tp_gated_linear_backward(const tp_gated_bwd_args *a, tp_stream_t stream) {
  clear_error();
  if (!a) return fail(TP_ERR_ARG, "args is NULL");
  int rc = check_common(a->dtype, a->act, a->weight_layout, a->M, a->F, a->K, "F");
  if (rc == TP_OK) rc = check_out_dtype(a->dx_dtype, a->dtype, "dx_dtype");
  if (rc == TP_OK) rc = check_out_dtype(a->dw_dtype, a->dtype, "dw_dtype");
  if (rc != TP_OK) return rc;
  if (a->accumulate != 0 && a->accumulate != 1) return fail(TP_ERR_ARG, "accumulate must be 0 or 1");
  if (!a->dW_gate != !a->dW_up) return fail(TP_ERR_ARG, "dW_gate and dW_up: both or neither");
  if (a->accumulate && a->dW_gate && a->dw_dtype != TP_F32) return fail(TP_ERR_ARG, "accumulate needs fp32 dW_gate and dW_up");
  const int64_t M = a->M, F = a->F, K = a->K, es = dtype_size(a->dtype);
  const bool linear = a->weight_layout == TP_WEIGHTS_LINEAR, any = M > 0;
  const int64_t wr = linear ? F : K, wc = linear ? K : F, dwes = dtype_size(a->dw_dtype);
  Mat x, wg, wu, g, u, d, dx, dwg, dwu;
  if ((rc = take(&x, "X", a->X, M, K, a->X_ld, es, any && a->dW_gate)) != TP_OK ||
      (rc = take(&wg, "W_gate", a->W_gate, wr, wc, a->W_ld, es, any && a->dX)) != TP_OK ||
      (rc = take(&wu, "W_up", a->W_up, wr, wc, a->W_ld, es, any && a->dX)) != TP_OK ||
      (rc = take(&g, "gate", a->gate, M, F, a->keep_ld, es, any)) != TP_OK ||
      (rc = take(&u, "up", a->up, M, F, a->keep_ld, es, any)) != TP_OK ||
      (rc = take(&d, "dOut", a->dOut, M, F, a->dOut_ld, es, any)) != TP_OK ||
      (rc = take(&dx, "dX", a->dX, M, K, a->dX_ld, dtype_size(a->dx_dtype), false)) != TP_OK ||
      (rc = take(&dwg, "dW_gate", a->dW_gate, wr, wc, a->dW_ld, dwes, false)) != TP_OK ||
      (rc = take(&dwu, "dW_up", a->dW_up, wr, wc, a->dW_ld, dwes, false)) != TP_OK)
    return rc;
  const BwdWs ws = gated_ws(M, F, K, a->dtype);
  if ((rc = check_ws(a->ws, a->ws_bytes, ws.join)) != TP_OK) return rc;
  const int64_t used = ws.used(a->ws, a->ws_bytes);
  const Mat wsm{used ? a->ws : nullptr, 1, used, used, 1, "ws"};
  if ((rc = disjoint({x, wg, wu, g, u, d}, {dx, dwg, dwu, wsm})) != TP_OK) return rc;

  hipStream_t s = static_cast<hipStream_t>(stream);
  char *d_gate = static_cast<char *>(a->ws), *d_up = d_gate + ws.d_up;
  uint32_t *tickets = used > ws.join ? reinterpret_cast<uint32_t *>(d_gate + ws.join) : nullptr;
  if (any) {
    ActGrad q;
    q.d_out = d.p;
    q.ld_dout = d.ld;
    q.pre = g.p;
    q.up = u.p;
    q.ld_pre = g.ld;
    q.d_pre = d_gate;
    q.d_up = d_up;
    q.M = M;
    q.N = F;
    q.f32 = a->dtype == TP_F32;
    q.act = a->act;
    q.gated = 1;
    q.tickets = tickets;
    hipEvent_t t0 = timing_begin(s);
    const hipError_t e = act_grad_launch(q, s);
    if (e != hipSuccess) return hip_fail(e, "activation gradient launch");
    timing_end(t0, s, TP_KERNEL_REDUCE, 5.0 * es * M * F);
  } else if (tickets) {
    const hipError_t e = zero_tickets_launch(tickets, s);
    if (e != hipSuccess) return hip_fail(e, "ticket launch");
  }
  const double flops = 4.0 * M * F * K;
  if (a->dX && any) {
    LinGemm p = dx_product(M, F, K, a->dtype, linear, true);
    p.a = d_gate;
    p.a2 = d_up;
    p.lda = F;
    p.w = wg.p;
    p.w2 = wu.p;
    p.ldw = wg.ld;
    p.c = a->dX;
    p.ldc = dx.ld;
    p.c_f32 = a->dx_dtype == TP_F32;
    if ((rc = launch(p, s, TP_KERNEL_GEMM_DGRAD, flops, "dX launch", tickets, used - ws.join)) != TP_OK) return rc;
  }
  if (a->dW_gate) {
    LinGemm p = dw_product(M, F, K, a->dtype, linear, true);
    p.a = linear ? d_gate : x.p;
    p.a2 = linear ? d_up : x.p;
    p.lda = linear ? F : x.ld;
    p.w = linear ? x.p : d_gate;
    p.w2 = linear ? x.p : d_up;
    p.ldw = linear ? x.ld : F;
    p.c = a->dW_gate;
    p.c2 = a->dW_up;
    p.ldc = dwg.ld;
    p.c_f32 = a->dw_dtype == TP_F32;
    p.acc_c = a->accumulate;
    if ((rc = launch(p, s, TP_KERNEL_GEMM_WGRAD, flops, "dW launch", tickets, used - ws.join)) != TP_OK) return rc;
  }
  return TP_OK;
}

}  // extern "C"

namespace {

// Validated tensors of a norm or clipping call; `clip`: the outputs too.
int take_grads(const tp_grad_tensor *ts, int64_t num, bool clip, std::vector<GradTensor> *out) {
  if (num < 0 || (num > 0 && !ts)) return fail(TP_ERR_ARG, "need num >= 0 and a tensor array");
  for (int64_t i = 0; i < num; ++i) {
    const tp_grad_tensor& t = ts[i];
    const int64_t es = dtype_size(t.dtype);
    if (!es) return fail(TP_ERR_ARG, "tensor %lld: unknown dtype %d", (long long)i, t.dtype);
    if (t.n < 0 || t.n >= (int64_t{1} << 48)) return fail(TP_ERR_ARG, "tensor %lld: n = %lld", (long long)i, (long long)t.n);
    if (t.n == 0) continue;
    if (!t.grad || (clip && !t.out)) return fail(TP_ERR_ARG, "tensor %lld: a buffer is NULL", (long long)i);
    if ((reinterpret_cast<uintptr_t>(t.grad) | (clip ? reinterpret_cast<uintptr_t>(t.out) : 0)) % static_cast<uintptr_t>(es))
      return fail(TP_ERR_ARG, "tensor %lld is not aligned to its elements", (long long)i);
    out->push_back({t.grad, clip ? t.out : nullptr, t.n, t.dtype == TP_F32});
  }
  return TP_OK;
}

int no_memory() { return fail(TP_ERR_HIP, "out of host memory"); }

double grad_bytes(const std::vector<GradTensor>& ts) {
  double b = 0;
  for (const GradTensor& t : ts) b += static_cast<double>(t.n) * (t.f32 ? 4 : 2);
  return b;
}

}  // namespace

extern "C" {

int tp_grad_sumsq(const tp_grad_tensor *tensors, int64_t num, double *parts, tp_stream_t stream) try {
  clear_error();
  std::vector<GradTensor> ts;
  int rc = take_grads(tensors, num, false, &ts);
  if (rc != TP_OK) return rc;
  if (!parts || reinterpret_cast<uintptr_t>(parts) % 8) return fail(TP_ERR_ARG, "parts is NULL or not 8-byte aligned");
  for (const GradTensor& t : ts)
    if (overlaps(parts, kGradParts * 8, t.g, t.n * (t.f32 ? 4 : 2))) return fail(TP_ERR_ARG, "parts overlaps a gradient");
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipEvent_t t0 = timing_begin(s);
  const hipError_t e = grad_sumsq_launch(ts.data(), static_cast<int64_t>(ts.size()), parts, s);
  if (e != hipSuccess) return hip_fail(e, "sum of squares launch");
  timing_end(t0, s, TP_KERNEL_REDUCE, grad_bytes(ts));
  return TP_OK;
} catch (const std::bad_alloc&) {
  return no_memory();
}

int tp_grad_clip(const tp_grad_tensor *tensors, int64_t num, const double *parts, int64_t ranks, double max_norm,
                 double eps, float *norm_out, tp_stream_t stream) try {
  clear_error();
  std::vector<GradTensor> ts;
  const int rc = take_grads(tensors, num, true, &ts);
  if (rc != TP_OK) return rc;
  if (!parts || reinterpret_cast<uintptr_t>(parts) % 8) return fail(TP_ERR_ARG, "parts is NULL or not 8-byte aligned");
  if (ranks < 1 || ranks > kMaxRanks) return fail(TP_ERR_ARG, "ranks = %lld outside [1, %lld]", (long long)ranks, (long long)kMaxRanks);
  if (!(max_norm >= 0) || !(eps >= 0)) return fail(TP_ERR_ARG, "max_norm and eps must be >= 0");
  if (reinterpret_cast<uintptr_t>(norm_out) % 4) return fail(TP_ERR_ARG, "norm_out is not aligned");
  // Outputs are apart from one another and from everything read, but for a
  // tensor scaled in place.  Sorted by address, one pass sees every overlap.
  struct Span {
    const void *p;
    int64_t n;
    bool written;
  };
  std::vector<Span> spans = {{parts, ranks * kGradParts * 8, false}};
  if (norm_out) spans.push_back({norm_out, 4, true});
  for (const GradTensor& t : ts) {
    const int64_t bytes = t.n * (t.f32 ? 4 : 2);
    spans.push_back({t.out, bytes, true});
    if (t.out != t.g) spans.push_back({t.g, bytes, false});
  }
  std::sort(spans.begin(), spans.end(),
            [](const Span& x, const Span& y) { return reinterpret_cast<uintptr_t>(x.p) < reinterpret_cast<uintptr_t>(y.p); });
  uintptr_t end_any = 0, end_written = 0;
  for (const Span& x : spans) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(x.p), end = at + static_cast<uintptr_t>(x.n);
    if (at < (x.written ? end_any : end_written)) return fail(TP_ERR_ARG, "a clipped output or norm_out overlaps another buffer");
    end_any = std::max(end_any, end);
    if (x.written) end_written = std::max(end_written, end);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipEvent_t t0 = timing_begin(s);
  const hipError_t e = grad_clip_launch(ts.data(), static_cast<int64_t>(ts.size()), parts, ranks, max_norm, eps, norm_out, s);
  if (e != hipSuccess) return hip_fail(e, "clipping launch");
  timing_end(t0, s, TP_KERNEL_REDUCE, 2.0 * grad_bytes(ts));
  return TP_OK;
} catch (const std::bad_alloc&) {
  return no_memory();
}

}  // extern "C"
