// The global gradient norm over many tensors, and clipping by it.
//
//   n = sqrt(sum over ranks, tensors and elements of g^2)
//   g' = g * min(1, max_norm / (n + eps))
//
// Two launches: the first leaves kGradParts partial sums of squares, the second
// adds every rank's partials (each workgroup for itself: 8 KiB out of L2) and
// scales.  The squares are summed in 64 bits: they span twice the exponent range
// of the gradients (fp32 would overflow from 2^64 and lose those under 2^-75),
// and the vector units add doubles at half the fp32 rate, far above what memory
// delivers.  Workgroup b takes every kGradParts-th chunk of each tensor in turn,
// so the order of every sum depends on the sizes alone.
//
// Bound by HBM: 805 MB of fp32 in 126 us for the norm (6.4 TB/s) and 284 us for the
// scaling (5.7 TB/s read and written) on an MI355X; 7 MB in 3.4 + 5.3 us.
//
// The tensors' pointers travel in the kernel's arguments, kMaxTensors a launch:
// no table in device memory, nothing to copy, and a captured graph keeps them.
#include <vector>

#include "grad_table.h"
#include "linear_dev.h"

namespace tpshard {

using namespace lin;

namespace {

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sum over the workgroup, in every lane.
__device__ __forceinline__ double block_sum(double v, double *lds) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = lds[0];
#pragma unroll
  for (int w = 1; w < kGradThreads / 64; ++w) t += lds[w];
  __syncthreads();
  return t;
}

// The tensor that chunk `u` belongs to, from `i` on (chunks come in order).
__device__ __forceinline__ int tensor_of(const GradTable& t, int64_t u, int i) {
  while (u >= t.first[i + 1]) ++i;
  return i;
}

__device__ __forceinline__ double sq(float v) { return static_cast<double>(v) * static_cast<double>(v); }

__global__ void __launch_bounds__(kGradThreads) grad_sumsq_kernel(GradTable t, double *parts, int add) {
  __shared__ double lds[kGradThreads / 64];
  double s0 = 0.0, s1 = 0.0;
  int i = 0;
  for (int64_t u = blockIdx.x; u < t.first[t.num]; u += kGradParts) {
    i = tensor_of(t, u, i);
    const int64_t at = (u - t.first[i]) * kGradChunk, left = t.n[i] - at;
    if (t.f32 >> i & 1) {
      const uint32_t *g = static_cast<const uint32_t *>(t.g[i]) + at;
      if (left >= kGradChunk) {
        u32x4 v[kGradPer / 4];
#pragma unroll
        for (int q = 0; q < kGradPer / 4; ++q)
          v[q] = *reinterpret_cast<const u32x4_any *>(g + (q * kGradThreads + threadIdx.x) * 4);
#pragma unroll
        for (int q = 0; q < kGradPer / 4; ++q) {
          s0 += sq(__uint_as_float(v[q][0])) + sq(__uint_as_float(v[q][1]));
          s1 += sq(__uint_as_float(v[q][2])) + sq(__uint_as_float(v[q][3]));
        }
      } else {
        for (int64_t e = threadIdx.x; e < left; e += kGradThreads) s0 += sq(__uint_as_float(g[e]));
      }
    } else {
      const uint16_t *g = static_cast<const uint16_t *>(t.g[i]) + at;
      if (left >= kGradChunk) {
        u32x4 v[kGradPer / 8];
#pragma unroll
        for (int q = 0; q < kGradPer / 8; ++q)
          v[q] = *reinterpret_cast<const u32x4_any *>(g + (q * kGradThreads + threadIdx.x) * 8);
#pragma unroll
        for (int q = 0; q < kGradPer / 8; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s0 += sq(from_bf16(v[q][e] & 0xffffu));
            s1 += sq(from_bf16(v[q][e] >> 16));
          }
      } else {
        for (int64_t e = threadIdx.x; e < left; e += kGradThreads) s0 += sq(from_bf16(g[e]));
      }
    }
  }
  const double s = block_sum(s0 + s1, lds);
  if (threadIdx.x == 0) parts[blockIdx.x] = add ? parts[blockIdx.x] + s : s;
}

// One chunk of one tensor: loaded, then scaled and stored.
struct Chunk {
  u32x4 v[kGradPer / 4];
  const void *g;
  void *out;
  int64_t at, left;
  bool f32;
};

__device__ __forceinline__ void chunk_load(const GradTable& t, int64_t u, int i, Chunk& c) {
  c.g = t.g[i];
  c.out = t.out[i];
  c.at = (u - t.first[i]) * kGradChunk;
  c.left = t.n[i] - c.at;
  c.f32 = t.f32 >> i & 1;
  if (c.left < kGradChunk) return;
  if (c.f32) {
    const uint32_t *g = static_cast<const uint32_t *>(c.g) + c.at;
#pragma unroll
    for (int q = 0; q < kGradPer / 4; ++q) c.v[q] = *reinterpret_cast<const u32x4_any *>(g + (q * kGradThreads + threadIdx.x) * 4);
  } else {
    const uint16_t *g = static_cast<const uint16_t *>(c.g) + c.at;
#pragma unroll
    for (int q = 0; q < kGradPer / 8; ++q) c.v[q] = *reinterpret_cast<const u32x4_any *>(g + (q * kGradThreads + threadIdx.x) * 8);
  }
}

__device__ __forceinline__ void chunk_store(Chunk& c, float scale) {
  // Nothing below its limit changes where it lies.
  if (scale == 1.0f && c.out == c.g) return;
  if (c.f32) {
    const uint32_t *g = static_cast<const uint32_t *>(c.g) + c.at;
    uint32_t *o = static_cast<uint32_t *>(c.out) + c.at;
    if (c.left >= kGradChunk) {
#pragma unroll
      for (int q = 0; q < kGradPer / 4; ++q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c.v[q][e] = __float_as_uint(__uint_as_float(c.v[q][e]) * scale);
        __builtin_nontemporal_store(c.v[q], reinterpret_cast<u32x4_any *>(o + (q * kGradThreads + threadIdx.x) * 4));
      }
    } else {
      for (int64_t e = threadIdx.x; e < c.left; e += kGradThreads) o[e] = __float_as_uint(__uint_as_float(g[e]) * scale);
    }
  } else {
    const uint16_t *g = static_cast<const uint16_t *>(c.g) + c.at;
    uint16_t *o = static_cast<uint16_t *>(c.out) + c.at;
    if (c.left >= kGradChunk) {
#pragma unroll
      for (int q = 0; q < kGradPer / 8; ++q) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          c.v[q][e] = pack2(from_bf16(c.v[q][e] & 0xffffu) * scale, from_bf16(c.v[q][e] >> 16) * scale);
        __builtin_nontemporal_store(c.v[q], reinterpret_cast<u32x4_any *>(o + (q * kGradThreads + threadIdx.x) * 8));
      }
    } else {
      for (int64_t e = threadIdx.x; e < c.left; e += kGradThreads) o[e] = to_bf16(from_bf16(g[e]) * scale);
    }
  }
}

// Chunks are taken from the last to the first: the pass before went from first
// to last, and what it read last is still in the 256 MB cache on the memory side.
// The first chunk is on its way while the norm is added up.
__global__ void __launch_bounds__(kGradThreads) grad_clip_kernel(GradTable t, const double *parts, int64_t ranks,
                                                             double max_norm, double eps, float *norm_out) {
  __shared__ double lds[kGradThreads / 64];
  const int64_t chunks = t.first[t.num];
  int64_t u = chunks - 1 - blockIdx.x;
  int i = t.num - 1;
  auto find = [&]() {
    while (u < t.first[i]) --i;
  };
  Chunk c;
  if (u >= 0) {
    find();
    chunk_load(t, u, i, c);
  }
  double s = 0.0;
  for (int64_t q = threadIdx.x; q < ranks * kGradParts; q += kGradThreads) s += parts[q];
  const double norm = sqrt(block_sum(s, lds));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
  // A NaN norm makes a NaN scale; an infinite one a scale of zero.
  const double want = max_norm / (norm + eps);
  const float scale = want >= 1.0 ? 1.0f : static_cast<float>(want);
  while (u >= 0) {
    chunk_store(c, scale);
    u -= gridDim.x;
    if (u < 0) break;
    find();
    chunk_load(t, u, i, c);
  }
}

}  // namespace

hipError_t grad_sumsq_launch(const GradTensor *ts, int64_t num, double *parts, hipStream_t s) {
  int64_t at = 0;
  int add = 0;
  do {   // at least once: the partials are written even where there is nothing to add
    GradTable t;
    next_table(ts, num, &at, &t);
    hipLaunchKernelGGL(grad_sumsq_kernel, dim3(kGradParts), dim3(kGradThreads), 0, s, t, parts, add);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    add = 1;
  } while (at < num);
  return hipSuccess;
}

hipError_t grad_clip_launch(const GradTensor *ts, int64_t num, const double *parts, int64_t ranks, double max_norm,
                            double eps, float *norm_out, hipStream_t s) {
  // The tables of the pass before, from the last to the first.
  int64_t begin = 0, at = 0;
  std::vector<int64_t> starts;
  do {
    GradTable t;
    begin = at;
    next_table(ts, num, &at, &t);
    starts.push_back(begin);
  } while (at < num);
  for (size_t k = starts.size(); k-- > 0;) {
    GradTable t;
    at = starts[k];
    next_table(ts, num, &at, &t);
    const int64_t chunks = t.first[t.num];
    const int64_t grid = chunks < 1 ? 1 : chunks < 2048 ? chunks : 2048;
    hipLaunchKernelGGL(grad_clip_kernel, dim3(static_cast<unsigned>(grid)), dim3(kGradThreads), 0, s, t, parts, ranks,
                       max_norm, eps, norm_out);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    norm_out = nullptr;
  }
  return hipSuccess;
}

}  // namespace tpshard
