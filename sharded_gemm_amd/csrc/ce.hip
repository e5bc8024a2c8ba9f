// The vocabulary cross entropy's passes beside its products (ce_dev.h has their
// epilogues, ce_launch.cpp the schedule):
//
//   lse = ln sum_n e^{z_n} over a row's logits, from the {maximum, sum} pairs that the
//   products left; loss = lse - z_target.
//
// All are bound by what they move: pairs (8 bytes for each tile's columns of a row: 4096
// rows of 196 tiles 5 us), logits of few rows, X once (8192 x 4096 transposed 46 us, 2.9 TB/s: 64-byte
// rows of LDS tiles both ways, beside products of 4.6 ms), slices of dX (1021 x 1336, 3 or 4 of them, 6.3).
#include "ce.h"
#include "ce_dev.h"

namespace tpshard {

using namespace lin;
using namespace ce;

namespace {

constexpr int kThreads = 256;

// ---- logits of few rows ------------------------------------------------------------
// A workgroup reduces kCeStatCols logits of one row to a pair.
__global__ void __launch_bounds__(kThreads) ce_logits_kernel(CeLogits p) {
  constexpr int PER = kCeStatCols / kThreads;   // in fours, a row of fours at a time
  __shared__ float tops[kThreads / 64], sums[kThreads / 64];
  const int64_t m = blockIdx.y, n0 = static_cast<int64_t>(blockIdx.x) * kCeStatCols;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const float *z = p.z + m * p.ld;
  f32x4 v[PER / 4];
  float top = minus_inf();
#pragma unroll
  for (int q = 0; q < PER / 4; ++q) {
    const int64_t n = n0 + (q * kThreads + static_cast<int>(threadIdx.x)) * 4, left = p.n - n;
    v[q] = f32x4{minus_inf(), minus_inf(), minus_inf(), minus_inf()};
    if (left > 3) {
      v[q] = *reinterpret_cast<const f32x4 *>(z + n);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) v[q][e] = z[n + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, v[q][e]);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  const Against to(top);
  float s = 0.0f;
#pragma unroll
  for (int q = 0; q < PER / 4; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) s += exp2_(fmaf(v[q][e], to.by, -to.to));   // past the end: 2^-inf
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if (lane == 0) sums[wave] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = ((sums[0] + sums[1]) + (sums[2] + sums[3])) * exp2_(to.rest);
    *reinterpret_cast<f32x2 *>(p.part + 2 * (blockIdx.x * p.M + m)) = f32x2{top, s};
    const int t = column_of(p.targets[m], p.begin, p.n);
    if (t >= n0 && t < n0 + kCeStatCols) p.logit[m] = z[t];
  }
}

// ---- joining ---------------------------------------------------------------------
// R rows to a workgroup (16: a 128-byte line of pairs a slot; 1 where rows are few), the
// threads of a row over its slots, eight pairs in flight.
template <int R>
__global__ void __launch_bounds__(kThreads) ce_join_kernel(CeJoin p) {
  constexpr int Q = kThreads / R, U = 8;
  __shared__ f32x2 lds[kThreads];
  const int row = threadIdx.x % R, q = threadIdx.x / R;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * R + row;
  f32x2 a{minus_inf(), 0.0f};
  if (m < p.M) {
    const f32x2 *part = reinterpret_cast<const f32x2 *>(p.part) + m;
    int64_t i = q;
    for (; i + (U - 1) * Q < p.slots; i += U * Q) {
      f32x2 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = part[(i + u * Q) * p.M];
#pragma unroll
      for (int u = 0; u < U; ++u) a = join(a, v[u]);
    }
    for (; i < p.slots; i += Q) a = join(a, part[i * p.M]);
  }
  lds[threadIdx.x] = a;
  __syncthreads();
#pragma unroll
  for (int o = Q / 2; o > 0; o >>= 1) {
    if (q < o) lds[threadIdx.x] = a = join(a, lds[threadIdx.x + o * R]);
    __syncthreads();
  }
  if (q || m >= p.M) return;
  finish(p, m, a, p.logit[m]);
}

// Pieces' statistics: {max, sum of e^(z - max), target's logit or -inf}.
__global__ void __launch_bounds__(kThreads) ce_pieces_kernel(const float *stats, int64_t pieces, int64_t M,
                                                             const int64_t *targets, int64_t ignore, float *loss,
                                                             float *lse) {
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (m >= M) return;
  f32x2 a{minus_inf(), 0.0f};
  float logit = minus_inf();
  for (int64_t i = 0; i < pieces; ++i) {
    const float *p = stats + 3 * i * M + m;
    a = join(a, f32x2{p[0], p[M]});
    // (the target's piece; its logit may be a NaN)
    logit = p[2 * M] > logit || p[2 * M] != p[2 * M] ? p[2 * M] : logit;
  }
  const float total = lse_of(a);
  if (lse) lse[m] = total;
  if (loss) loss[m] = targets[m] == ignore ? 0.0f : total - logit;
}

// ---- the gradient's scale --------------------------------------------------------------
// By one workgroup of THREADS.
template <int THREADS>
__device__ __forceinline__ void scale_of(const CeScale& p) {
  for (int i = threadIdx.x; i < kMaxTickets; i += THREADS) p.tickets[i] = 0;
  if (!p.scale) return;
  __shared__ float tops[2][THREADS / 64];
  float g = 0.0f, h = 0.0f;
  auto larger = [](float top, float x) {
    x = fabsf(x);
    return x > top && x < __builtin_inff() ? x : top;   // (a NaN is neither)
  };
  constexpr int U = 8;   // tokens of a thread in flight
  for (int64_t m0 = threadIdx.x; m0 < p.M; m0 += U * THREADS) {
    int64_t id[U];
    float x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t m = m0 + u * THREADS < p.M ? m0 + u * THREADS : p.M - 1;
      id[u] = p.targets[m];
      x[u] = p.g ? p.g[m * p.g_step] : 1.0f;
      y[u] = p.h ? p.h[m * p.h_step] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (id[u] != p.ignore) {
        g = larger(g, x[u]);
        h = larger(h, y[u]);
      }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    g = fmaxf(g, __shfl_xor(g, o));
    h = fmaxf(h, __shfl_xor(h, o));
  }
  if ((threadIdx.x & 63) == 0) {
    tops[0][threadIdx.x >> 6] = g;
    tops[1][threadIdx.x >> 6] = h;
  }
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < THREADS / 64; ++w) {
    g = fmaxf(g, tops[0][w]);
    h = fmaxf(h, tops[1][w]);
  }
  g = fmaxf(g, h * 0x1p-64f);
  *p.scale = g < 0x1p-120f ? 1.0f : g;   // (its reciprocal has to be a number too)
}

__global__ void __launch_bounds__(1024) ce_scale_kernel(CeScale p) { scale_of<1024>(p); }

// ---- X, transposed, and padded copies --------------------------------------------------
// A padded copy's part of a workgroup.
__device__ __forceinline__ void pad_part(const CePad& p, int64_t block) {
  const int64_t per = p.cols / 8, i = block * kThreads + threadIdx.x;
  if (i >= p.rows * per) return;
  const int64_t r = i / per, c = i % per * 8, left = r < p.m ? p.n - c : 0;
  *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.to) + i * 8) =
      left > 0 ? load16<uint16_t>(static_cast<const uint16_t *>(p.from) + r * p.ld + c, left) : u32x4{0, 0, 0, 0};
}
// block: counted over both.
__device__ __forceinline__ void pad_parts(const CePads& p, int64_t block) {
  const int64_t first = (p.pad[0].rows * (p.pad[0].cols / 8) + kThreads - 1) / kThreads;
  if (block < first) pad_part(p.pad[0], block);
  else pad_part(p.pad[1], block - first);
}
__global__ void __launch_bounds__(kThreads) ce_pad_kernel(CePads p) { pad_parts(p, blockIdx.x); }

// 64 tokens x 64 columns through LDS; then the copies.  T: uint16_t or uint32_t.
template <typename T>
__global__ void __launch_bounds__(kThreads) ce_transpose_kernel(CeTranspose p, CePads pads) {
  constexpr int V = 16 / sizeof(T), E = 64, PITCH = E + 4 / sizeof(T);   // a row and a bank
  __shared__ T tile[E * PITCH];
  const int64_t blocks = (p.K + E - 1) / E * (p.rows / E);
  if (blockIdx.x >= blocks) return pad_parts(pads, blockIdx.x - blocks);
  if (blockIdx.x == 0) scale_of<kThreads>(p.scale);
  const int64_t tiles_k = (p.K + E - 1) / E, k0 = blockIdx.x % tiles_k * E, m0 = blockIdx.x / tiles_k * E;
#pragma unroll
  for (int q = 0; q < E * E / V / kThreads; ++q) {
    const int i = q * kThreads + threadIdx.x, r = i / (E / V), c = i % (E / V) * V;
    const int64_t m = m0 + r, left = p.K - k0 - c;
    u32x4 v{0, 0, 0, 0};
    if (m < p.M && left > 0 && p.targets[m] != p.ignore) v = load16<T>(static_cast<const T *>(p.X) + m * p.X_ld + k0 + c, left);
#pragma unroll
    for (int e = 0; e < V; ++e)
      tile[r * PITCH + c + e] = sizeof(T) == 4 ? static_cast<T>(v[e]) : static_cast<T>(v[e * sizeof(T) / 4] >> (16 * (e & 1)));
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < E * E / V / kThreads; ++q) {
    const int i = q * kThreads + threadIdx.x, k = i / (E / V), r = i % (E / V) * V;
    if (k0 + k >= p.K) continue;
    u32x4 v{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const uint32_t x = tile[(r + e) * PITCH + k];
      if constexpr (sizeof(T) == 4) v[e] = x;
      else v[e / 2] |= x << (16 * (e & 1));
    }
    *reinterpret_cast<u32x4 *>(static_cast<T *>(p.xt) + (k0 + k) * p.rows + m0 + r) = v;
  }
}

// ---- dX's sum over slices and pieces ------------------------------------------------
__global__ void __launch_bounds__(kThreads) ce_sum_kernel(CeSum p) {
  const int64_t per = (p.K + 3) / 4, i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.M * per) return;
  const int64_t m = i / per, k = i % per * 4, left = p.K - k;
  f32x4 v{0.f, 0.f, 0.f, 0.f};
  constexpr int B = 4;   // slices in flight
  for (int64_t s = 0; s < p.slices; s += B) {
    f32x4 x[B];
#pragma unroll
    for (int b = 0; b < B; ++b) x[b] = load4<float>(p.part, ((s + b) * p.M + m) * p.K + k, s + b < p.slices ? left : 0);
#pragma unroll
    for (int b = 0; b < B; ++b) v = v + x[b];
  }
  if (p.alpha) v = v * *p.alpha;
  if (p.base) v = load4<float>(p.base, m * p.base_ld + k, left) + v;
  if (p.out_f32) store4<float>(p.out, m * p.out_ld + k, v, left);
  else store4<uint16_t>(p.out, m * p.out_ld + k, v, left);
}

unsigned grid_of(int64_t n, int64_t by) { return static_cast<unsigned>((n + by - 1) / by); }

}  // namespace

hipError_t ce_logits_launch(const CeLogits& p, hipStream_t s) {
  hipLaunchKernelGGL(ce_logits_kernel, dim3(grid_of(p.n, kCeStatCols), static_cast<unsigned>(p.M)), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t ce_join_launch(const CeJoin& p, hipStream_t s) {
  if (p.M < 1024) hipLaunchKernelGGL(ce_join_kernel<1>, dim3(grid_of(p.M, 1)), dim3(kThreads), 0, s, p);
  else hipLaunchKernelGGL(ce_join_kernel<16>, dim3(grid_of(p.M, 16)), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t ce_pieces_launch(const float *stats, int64_t pieces, int64_t M, const int64_t *targets, int64_t ignore,
                            float *loss, float *lse, hipStream_t s) {
  hipLaunchKernelGGL(ce_pieces_kernel, dim3(grid_of(M, kThreads)), dim3(kThreads), 0, s, stats, pieces, M, targets, ignore, loss, lse);
  return hipGetLastError();
}

hipError_t ce_scale_launch(const CeScale& p, hipStream_t s) {
  hipLaunchKernelGGL(ce_scale_kernel, dim3(1), dim3(1024), 0, s, p);
  return hipGetLastError();
}

namespace {
unsigned pad_blocks(const CePads& p) {
  unsigned n = 0;
  for (int i = 0; i < p.num; ++i) n += grid_of(p.pad[i].rows * (p.pad[i].cols / 8), kThreads);
  return n;
}
}  // namespace

hipError_t ce_transpose_launch(const CeTranspose& p, const CePads& pads, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.K + 63) / 64 * (p.rows / 64)) + pad_blocks(pads));
  if (p.f32) hipLaunchKernelGGL(ce_transpose_kernel<uint32_t>, grid, dim3(kThreads), 0, s, p, pads);
  else hipLaunchKernelGGL(ce_transpose_kernel<uint16_t>, grid, dim3(kThreads), 0, s, p, pads);
  return hipGetLastError();
}

hipError_t ce_pad_launch(const CePads& p, hipStream_t s) {
  const unsigned n = pad_blocks(p);
  if (!n) return hipSuccess;
  hipLaunchKernelGGL(ce_pad_kernel, dim3(n), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t ce_sum_launch(const CeSum& p, hipStream_t s) {
  hipLaunchKernelGGL(ce_sum_kernel, dim3(grid_of(p.M * ((p.K + 3) / 4), kThreads)), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace tpshard
