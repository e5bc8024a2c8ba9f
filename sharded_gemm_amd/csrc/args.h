// Checks of matrix and workspace arguments that the entry points share.  Host code
// only.
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "common.h"

namespace tpshard {
namespace {

constexpr int64_t kMaxDim = int64_t{1} << 31;

[[maybe_unused]] int hip_fail(hipError_t e, const char *what) {
  return fail(TP_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// A matrix argument: rows x cols at row stride ld (0 = contiguous).
struct Mat {
  const void *p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0, es = 0;
  const char *name = "";
  int64_t bytes() const { return rows <= 0 || cols <= 0 || !p ? 0 : ((rows - 1) * ld + cols) * es; }
};

// Fills *m; the stride must cover a row, the pointer be aligned to its element.
[[maybe_unused]] int take(Mat *m, const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t es, bool needed) {
  *m = Mat{p, rows, cols, ld ? ld : cols, es, name};
  if (!p) return needed ? fail(TP_ERR_ARG, "%s must be non-NULL", name) : TP_OK;
  if (m->ld < cols) return fail(TP_ERR_ARG, "%s: row stride %lld < %lld", name, (long long)m->ld, (long long)cols);
  if (m->ld >= kMaxDim)
    return fail(TP_ERR_UNSUPPORTED, "%s: row stride %lld exceeds the kernels' range", name, (long long)m->ld);
  if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(es))
    return fail(TP_ERR_ARG, "%s is not aligned to its elements", name);
  return TP_OK;
}

// Whether two matrices share an element.  Column blocks of one larger matrix
// (one row pitch) interleave in memory without sharing any: then the columns'
// places within the pitch decide.
[[maybe_unused]] bool share(const Mat& a, const Mat& b) {
  if (!overlaps(a.p, a.bytes(), b.p, b.bytes())) return false;
  if (reinterpret_cast<uintptr_t>(b.p) < reinterpret_cast<uintptr_t>(a.p)) return share(b, a);
  const uintptr_t pitch = static_cast<uintptr_t>(a.ld * a.es);
  if (a.ld * a.es != b.ld * b.es) return true;
  const uintptr_t at = (reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % pitch;
  return at < static_cast<uintptr_t>(a.cols * a.es) || at + static_cast<uintptr_t>(b.cols * b.es) > pitch;
}

[[maybe_unused]] int disjoint(std::initializer_list<Mat> ins, std::initializer_list<Mat> outs) {
  for (const Mat *o = outs.begin(); o != outs.end(); ++o) {
    for (const Mat& in : ins)
      if (share(*o, in)) return fail(TP_ERR_ARG, "%s overlaps %s", o->name, in.name);
    for (const Mat *e = outs.begin(); e != o; ++e)
      if (share(*o, *e)) return fail(TP_ERR_ARG, "%s overlaps %s", o->name, e->name);
  }
  return TP_OK;
}

// An output's type: the operands', or fp32.
[[maybe_unused]] int check_out_dtype(int32_t out, int32_t dtype, const char *name) {
  if (out != dtype && out != TP_F32) return fail(TP_ERR_ARG, "%s = %d is neither dtype nor TP_F32", name, out);
  return TP_OK;
}

[[maybe_unused]] int check_ws(const void *ws, int64_t have, int64_t need) {
  if (!need) return TP_OK;
  if (!ws || have < need)
    return fail(TP_ERR_ARG, "the workspace holds %lld bytes, %lld are needed", (long long)(ws ? have : 0), (long long)need);
  if (reinterpret_cast<uintptr_t>(ws) & 15) return fail(TP_ERR_ARG, "ws is not 16-byte aligned");
  return TP_OK;
}

[[maybe_unused]] int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// An optional workspace: given at all, it has to be aligned and apart.
[[maybe_unused]] int take_ws(Mat *m, void *ws, int64_t bytes) {
  if (!ws || bytes <= 0) return TP_OK;
  if (reinterpret_cast<uintptr_t>(ws) & 15) return fail(TP_ERR_ARG, "ws is not 16-byte aligned");
  *m = Mat{ws, 1, bytes, bytes, 1, "ws"};
  return TP_OK;
}

}  // namespace
}  // namespace tpshard
