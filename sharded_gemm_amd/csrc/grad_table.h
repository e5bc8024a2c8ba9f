// The tensors of one launch of the gradient norm or of clipping, cut into chunks.
#pragma once

#include <cstdint>

#include "linear.h"

namespace tpshard {

constexpr int kMaxTensors = 64;
constexpr int kGradThreads = 256;
// Elements of a chunk: 16 per lane.
constexpr int kGradPer = 16;
constexpr int kGradChunk = kGradThreads * kGradPer;

struct GradTable {
  const void *g[kMaxTensors];
  void *out[kMaxTensors];
  int64_t first[kMaxTensors + 1];   // chunks before tensor i
  int64_t n[kMaxTensors];
  uint64_t f32;                     // bit i: tensor i holds fp32
  int32_t num;
};
static_assert(sizeof(GradTable) < 3500, "kernel arguments");

// The next tensors that hold anything, from *at on, as one launch's table.
inline void next_table(const GradTensor *ts, int64_t num, int64_t *at, GradTable *t) {
  t->num = 0;
  t->f32 = 0;
  t->first[0] = 0;
  for (; *at < num && t->num < kMaxTensors; ++*at) {
    const GradTensor& x = ts[*at];
    if (x.n <= 0) continue;
    const int i = t->num++;
    t->g[i] = x.g;
    t->out[i] = x.out;
    t->n[i] = x.n;
    t->first[i + 1] = t->first[i] + (x.n + kGradChunk - 1) / kGradChunk;
    if (x.f32) t->f32 |= uint64_t{1} << i;
  }
}

}  // namespace tpshard
