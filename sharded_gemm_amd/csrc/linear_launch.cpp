// Which kernel a product of the linear layer or the gated block runs on.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "linear.h"

namespace tpshard {

namespace {

bool aligned(const void *p, int64_t ld, int64_t es, int64_t elems) {
  return !p || (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(elems * es) == 0 && ld % elems == 0);
}

}  // namespace

bool lin_tiles_ok(const LinGemm& p) {
  if (p.f32 || p.K <= 0 || p.K % 32) return false;
  if (!aligned(p.a, p.lda, 2, 8) || !aligned(p.a2, p.lda, 2, 8) || !aligned(p.w, p.ldw, 2, 8) || !aligned(p.w2, p.ldw, 2, 8))
    return false;
  return (!p.a_t || p.M % 8 == 0) && (p.w_t || p.N % 8 == 0);
}

hipError_t lin_tiles_launch(const LinGemm& p, hipStream_t s) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  if (p.a_t) return lin_tiles_pair(p, s);
  switch (p.mode) {
    case kModeOne: return lin_tiles_one(p, s);
    case kModeDual: return lin_tiles_dual(p, s);
    case kModeCat: return lin_tiles_cat(p, s);
  }
  return hipErrorInvalidValue;
}

hipError_t lin_gemm_launch(LinGemm p, hipStream_t s, void *ws, int64_t ws_bytes) {
  const int64_t es = p.f32 ? 4 : 2, ces = p.c_f32 ? 4 : 2;
  p.vec = aligned(p.c, p.ldc, ces, 4) && aligned(p.c2, p.ldc, ces, 4) && aligned(p.res, p.ldres, es, 4) &&
          aligned(p.aux, p.ldaux, es, 4) && aligned(p.aux2, p.ldaux, es, 4) && aligned(p.bias, 4, 4, 4);
  if (lin_rows_ok(p)) return lin_rows_launch(p, ws, ws_bytes, s);
  if (lin_tiles_ok(p)) return lin_tiles_launch(p, s);
  return lin_staged_launch(p, s);
}

}  // namespace tpshard
