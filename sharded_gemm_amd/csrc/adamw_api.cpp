// C ABI of the AdamW step: validation, then the launches.  A call checks every argument
// before it enqueues anything.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "adamw.h"
#include "args.h"
#include "linear.h"
#include "timing.h"

namespace tpshard {
namespace {

constexpr int64_t kMaxRanks = 64;
constexpr int64_t kMaxElements = int64_t{1} << 48;
static_assert(kAdamBlock == TP_ADAMW_BLOCK, "the header's count");

int no_memory() { return fail(TP_ERR_HIP, "out of host memory"); }

// Buffers that are read or written.  Those written are apart from all others.
struct Span {
  const void *p;
  int64_t n;
  bool written;
};
int apart(std::vector<Span> *spans) {
  std::sort(spans->begin(), spans->end(),
            [](const Span& x, const Span& y) { return reinterpret_cast<uintptr_t>(x.p) < reinterpret_cast<uintptr_t>(y.p); });
  uintptr_t end_any = 0, end_written = 0;
  for (const Span& x : *spans) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(x.p), end = at + static_cast<uintptr_t>(x.n);
    if (at < (x.written ? end_any : end_written)) return fail(TP_ERR_ARG, "a buffer that is written overlaps another");
    end_any = std::max(end_any, end);
    if (x.written) end_written = std::max(end_written, end);
  }
  return TP_OK;
}

// Adds a buffer of n bytes of tensor i, aligned to its elements.
int add(std::vector<Span> *spans, const void *p, int64_t n, int64_t es, bool written, const char *name, int64_t i) {
  if (!p) return fail(TP_ERR_ARG, "tensor %lld: %s is NULL", (long long)i, name);
  if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(es))
    return fail(TP_ERR_ARG, "tensor %lld: %s is not aligned to its elements", (long long)i, name);
  spans->push_back({p, n, written});
  return TP_OK;
}

int check_count(int64_t n, int64_t i) {
  if (n < 0 || n >= kMaxElements) return fail(TP_ERR_ARG, "tensor %lld: n = %lld", (long long)i, (long long)n);
  return TP_OK;
}

int check_args(const tp_adamw_args *a) {
  if (a->states != TP_ADAMW_F32 && a->states != TP_ADAMW_8BIT) return fail(TP_ERR_ARG, "unknown states %d", a->states);
  if (!(a->lr >= 0) || !(a->eps >= 0)) return fail(TP_ERR_ARG, "lr and eps must be >= 0");
  if (!(a->beta1 >= 0 && a->beta1 < 1) || !(a->beta2 >= 0 && a->beta2 < 1)) return fail(TP_ERR_ARG, "beta1 and beta2 must be in [0, 1)");
  if (!a->step_dev && a->step < 1) return fail(TP_ERR_ARG, "step = %lld: counted from 1", (long long)a->step);
  if (reinterpret_cast<uintptr_t>(a->step_dev) % 8 || reinterpret_cast<uintptr_t>(a->lr_dev) % 4)
    return fail(TP_ERR_ARG, "step_dev or lr_dev is not aligned");
  if (a->skip_nonfinite != 0 && a->skip_nonfinite != 1) return fail(TP_ERR_ARG, "skip_nonfinite must be 0 or 1");
  if (!a->parts) {
    if (a->norm_out || a->skip_nonfinite) return fail(TP_ERR_ARG, "norm_out and skip_nonfinite need parts");
    return TP_OK;
  }
  if (reinterpret_cast<uintptr_t>(a->parts) % 8 || reinterpret_cast<uintptr_t>(a->norm_out) % 4)
    return fail(TP_ERR_ARG, "parts or norm_out is not aligned");
  if (a->ranks < 1 || a->ranks > kMaxRanks)
    return fail(TP_ERR_ARG, "ranks = %lld outside [1, %lld]", (long long)a->ranks, (long long)kMaxRanks);
  if (!(a->max_norm >= 0) || !(a->clip_eps >= 0)) return fail(TP_ERR_ARG, "max_norm and clip_eps must be >= 0");
  return TP_OK;
}

}  // namespace
}  // namespace tpshard

using namespace tpshard;

extern "C" {

int tp_adamw_step(const tp_adamw_tensor *tensors, int64_t num, const tp_adamw_args *a, tp_stream_t stream) try {
  clear_error();
  if (!a) return fail(TP_ERR_ARG, "args is NULL");
  if (num < 0 || (num > 0 && !tensors)) return fail(TP_ERR_ARG, "need num >= 0 and a tensor array");
  int rc = check_args(a);
  if (rc != TP_OK) return rc;
  const bool codes = a->states == TP_ADAMW_8BIT;
  std::vector<AdamTensor> ts;
  std::vector<Span> spans;
  double bytes = 0;
  for (int64_t i = 0; i < num; ++i) {
    const tp_adamw_tensor& t = tensors[i];
    const int64_t pes = dtype_size(t.param_dtype), ges = dtype_size(t.grad_dtype), ses = codes ? 1 : 4;
    if (!pes || !ges) return fail(TP_ERR_ARG, "tensor %lld: unknown dtype", (long long)i);
    if (!(t.weight_decay >= 0)) return fail(TP_ERR_ARG, "tensor %lld: weight_decay must be >= 0", (long long)i);
    if ((rc = check_count(t.n, i)) != TP_OK) return rc;
    if (t.n == 0) continue;
    const int64_t scales = (t.n + kAdamBlock - 1) / kAdamBlock * 4;
    if ((rc = add(&spans, t.param, t.n * pes, pes, true, "param", i)) != TP_OK ||
        (rc = add(&spans, t.grad, t.n * ges, ges, false, "grad", i)) != TP_OK ||
        (rc = add(&spans, t.m, t.n * ses, ses, true, "m", i)) != TP_OK ||
        (rc = add(&spans, t.v, t.n * ses, ses, true, "v", i)) != TP_OK ||
        (codes && (rc = add(&spans, t.m_scale, scales, 4, true, "m_scale", i)) != TP_OK) ||
        (codes && (rc = add(&spans, t.v_scale, scales, 4, true, "v_scale", i)) != TP_OK) ||
        (t.copy && (rc = add(&spans, t.copy, t.n * 2, 2, true, "copy", i)) != TP_OK))
      return rc;
    ts.push_back({t.param, t.copy, t.grad, t.m, t.v, codes ? t.m_scale : nullptr, codes ? t.v_scale : nullptr, t.n,
                  static_cast<float>(t.weight_decay), t.param_dtype == TP_F32, t.grad_dtype == TP_F32});
    bytes += static_cast<double>(t.n) * static_cast<double>(2 * pes + ges + 4 * ses + (t.copy ? 2 : 0));
  }
  if (a->parts) spans.push_back({a->parts, a->ranks * kGradParts * 8, false});
  if (a->norm_out) spans.push_back({a->norm_out, 4, true});
  if (a->step_dev) spans.push_back({a->step_dev, 8, false});
  if (a->lr_dev) spans.push_back({a->lr_dev, 4, false});
  if ((rc = apart(&spans)) != TP_OK) return rc;
  AdamArgs p;
  p.lr = static_cast<float>(a->lr);
  p.beta1 = static_cast<float>(a->beta1);
  p.beta2 = static_cast<float>(a->beta2);
  p.rest1 = static_cast<float>(1.0 - a->beta1);
  p.rest2 = static_cast<float>(1.0 - a->beta2);
  p.eps = static_cast<float>(a->eps);
  if (a->step_dev) {
    p.step = a->step_dev;
    p.log2_beta1 = std::log2(a->beta1);
    p.log2_beta2 = std::log2(a->beta2);
  } else {
    p.over1 = static_cast<float>(1.0 / (1.0 - std::pow(a->beta1, static_cast<double>(a->step))));
    p.over2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(a->beta2, static_cast<double>(a->step))));
  }
  p.lr_dev = a->lr_dev;
  p.parts = a->parts;
  p.ranks = a->ranks;
  p.max_norm = a->max_norm;
  p.clip_eps = a->clip_eps;
  p.norm_out = a->norm_out;
  p.skip = a->skip_nonfinite;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipEvent_t t0 = timing_begin(s);
  const hipError_t e = adamw_launch(ts.data(), static_cast<int64_t>(ts.size()), codes, p, s);
  if (e != hipSuccess) return hip_fail(e, "AdamW launch");
  timing_end(t0, s, TP_KERNEL_REDUCE, bytes);
  return TP_OK;
} catch (const std::bad_alloc&) {
  return no_memory();
}

int tp_adamw_unpack(const tp_adamw_state *states, int64_t num, tp_stream_t stream) try {
  clear_error();
  if (num < 0 || (num > 0 && !states)) return fail(TP_ERR_ARG, "need num >= 0 and an array of states");
  std::vector<AdamValues> ts;
  std::vector<Span> spans;
  double bytes = 0;
  for (int64_t i = 0; i < num; ++i) {
    const tp_adamw_state& t = states[i];
    const int64_t es = dtype_size(t.out_dtype);
    int rc;
    if (!es) return fail(TP_ERR_ARG, "tensor %lld: unknown dtype %d", (long long)i, t.out_dtype);
    if ((rc = check_count(t.n, i)) != TP_OK) return rc;
    if (t.n == 0) continue;
    const int64_t scales = (t.n + kAdamBlock - 1) / kAdamBlock * 4;
    if ((rc = add(&spans, t.m, t.n, 1, false, "m", i)) != TP_OK || (rc = add(&spans, t.v, t.n, 1, false, "v", i)) != TP_OK ||
        (rc = add(&spans, t.m_scale, scales, 4, false, "m_scale", i)) != TP_OK ||
        (rc = add(&spans, t.v_scale, scales, 4, false, "v_scale", i)) != TP_OK ||
        (rc = add(&spans, t.m_out, t.n * es, es, true, "m_out", i)) != TP_OK ||
        (rc = add(&spans, t.v_out, t.n * es, es, true, "v_out", i)) != TP_OK)
      return rc;
    ts.push_back({t.m, t.v, t.m_scale, t.v_scale, t.m_out, t.v_out, t.n, t.out_dtype == TP_F32});
    bytes += static_cast<double>(t.n) * static_cast<double>(2 + 2 * es);
  }
  const int rc = apart(&spans);
  if (rc != TP_OK) return rc;
  if (ts.empty()) return TP_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipEvent_t t0 = timing_begin(s);
  const hipError_t e = adamw_values_launch(ts.data(), static_cast<int64_t>(ts.size()), s);
  if (e != hipSuccess) return hip_fail(e, "AdamW state launch");
  timing_end(t0, s, TP_KERNEL_REDUCE, bytes);
  return TP_OK;
} catch (const std::bad_alloc&) {
  return no_memory();
}

}  // extern "C"
