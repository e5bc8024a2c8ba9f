// Launch interface of the AdamW step (adamw_api.cpp validates; the kernels trust what
// reaches them), and the tables of tensors that travel in the kernels' arguments.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace tpshard {

constexpr int kAdamThreads = 256;
// Elements of a chunk: 16 per lane, in fours.  A wave's four times 64 lanes are a
// block of the 8-bit states, so blocks never cross waves.
constexpr int kAdamPer = 16, kAdamChunk = kAdamThreads * kAdamPer;
constexpr int kAdamBlock = 256;
constexpr int kMaxAdam = 40;   // tensors of a launch

// One tensor.  The states are fp32, or (ms, vs not null) codes and a scale a block.
struct AdamTensor {
  void *param, *copy;
  const void *grad;
  void *m, *v;
  float *ms, *vs;
  int64_t n;
  float decay;
  int32_t param_f32, grad_f32;
};
// Its codes as values, in fp32 or bf16.
struct AdamValues {
  const void *m, *v;
  const float *ms, *vs;
  void *m_out, *v_out;
  int64_t n;
  int32_t f32;
};

struct AdamTable {
  AdamTensor t[kMaxAdam];
  int64_t first[kMaxAdam + 1];   // chunks before tensor i
  int32_t num;
};
struct AdamValuesTable {
  AdamValues t[kMaxAdam];
  int64_t first[kMaxAdam + 1];
  int32_t num;
};

// The next tensors that hold anything, from *at on, as one launch's table.
template <typename Tensor, typename Table>
inline void next_adam(const Tensor *ts, int64_t num, int64_t *at, Table *t) {
  t->num = 0;
  t->first[0] = 0;
  for (; *at < num && t->num < kMaxAdam; ++*at) {
    if (ts[*at].n <= 0) continue;
    const int i = t->num++;
    t->t[i] = ts[*at];
    t->first[i + 1] = t->first[i] + (ts[*at].n + kAdamChunk - 1) / kAdamChunk;
  }
}

struct AdamArgs {
  float lr = 0, beta1 = 0, beta2 = 0, rest1 = 0, rest2 = 0, eps = 0;   // rest: 1 - beta
  float over1 = 1, over2 = 1;   // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t): where the step is the host's
  double log2_beta1 = 0, log2_beta2 = 0;
  const int64_t *step = nullptr;   // where it is the device's
  const float *lr_dev = nullptr;   // in lr's place
  const double *parts = nullptr;   // clipping, as grad_clip_launch
  int64_t ranks = 0;
  double max_norm = 0, clip_eps = 0;
  float *norm_out = nullptr;
  int32_t skip = 0;                // leave everything as it is where the norm is not finite
};
static_assert(sizeof(AdamTable) + sizeof(AdamArgs) < 4000 && sizeof(AdamValuesTable) < 4000, "kernel arguments");
hipError_t adamw_launch(const AdamTensor *ts, int64_t num, bool codes, const AdamArgs& a, hipStream_t s);
hipError_t adamw_values_launch(const AdamValues *ts, int64_t num, hipStream_t s);

}  // namespace tpshard
