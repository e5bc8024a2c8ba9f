// Launch interface of the AdamW step (adamw_api.cpp validates; the kernels trust what
// reaches them), and the tables of tensors that travel in the kernels' arguments.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace tpshard {

constexpr int kAdamThreads = 256;
constexpr int kAdamBlock = 256;   // elements of a wave's lanes by fours, so that blocks never cross waves
// Elements of a chunk, by each lane of a workgroup in fours.  Many in flight suit long
// streams, few the latency of a call with little for each CU.  MI355X, 16 : 4 a lane, us:
// fp32 states 201M elements 1028 : 1086, 20M 85 : 84, 1.8M 7.3 : 6.6; 8-bit states, fp32
// weights, 201M 569 : 605, 60M 178 : 167, 20M 52 : 49, 1.8M 9.7 : 7.9, 100 000 8.7 : 4.3; these as
// values in bf16, 201M 205 : 258.
constexpr int kAdamChunk = kAdamThreads * 16, kAdamShort = kAdamThreads * 4;
constexpr int64_t kAdamLong = int64_t{1} << 25;   // elements from which chunks are long
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
  int64_t first[kMaxAdam + 1];   // chunks before tensor i: whole ones where they are long
  int32_t num;
};
struct AdamValuesTable {
  AdamValues t[kMaxAdam];
  int64_t first[kMaxAdam + 1];
  int32_t num;
};

inline int64_t adam_chunk(const AdamTensor *ts, int64_t num) {
  int64_t n = 0;
  for (int64_t i = 0; i < num; ++i) n += ts[i].n;
  return n < kAdamLong ? kAdamShort : kAdamChunk;
}

// The next tensors that hold anything, from *at on, as one launch's table; whole: without their ends.
template <typename Tensor, typename Table>
inline void next_adam(const Tensor *ts, int64_t num, int64_t *at, Table *t, int64_t chunk, bool whole) {
  t->num = 0;
  t->first[0] = 0;
  for (; *at < num && t->num < kMaxAdam; ++*at) {
    if (ts[*at].n <= 0) continue;
    const int i = t->num++;
    t->t[i] = ts[*at];
    t->first[i + 1] = t->first[i] + (ts[*at].n + (whole ? 0 : chunk - 1)) / chunk;
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
static_assert(kMaxAdam <= 64, "a lane for each");
static_assert(sizeof(AdamTable) + sizeof(AdamArgs) < 4000 && sizeof(AdamValuesTable) < 4000, "kernel arguments");
hipError_t adamw_launch(const AdamTensor *ts, int64_t num, bool codes, const AdamArgs& a, hipStream_t s);
hipError_t adamw_values_launch(const AdamValues *ts, int64_t num, hipStream_t s);

}  // namespace tpshard
