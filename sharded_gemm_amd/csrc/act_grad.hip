// Gradients at the activation of the linear layer and of the gated block, and
// the bias gradient's column sums.
//
//   linear: dPre = dOut * act'(pre);         dbias[n] = sum over m of dPre[m, n]
//   gated : dU = dOut * act(G);              dG = dOut * U * act'(G)
//
// One pass over the inputs, memory-bound: a workgroup takes 512 columns by a
// slab of rows, each lane 8 columns (16 bytes of bf16) of every fourth row.
// The column sums add the unrounded fp32 values (dPre itself is rounded once to
// the operands' type, for the products that read it next); each slab leaves its
// own partial row and a second kernel adds the slabs in order, so no atomics
// decide the result.
#include "linear_dev.h"

namespace tpshard {

using namespace lin;

namespace {

constexpr int kLanes = 64, kGroups = 4, kCols = 8;
constexpr int kTileCols = kLanes * kCols;

// Eight elements at p; `left` exist (the rest read as zero).
template <typename T>
__device__ __forceinline__ void load8(const T *p, int64_t left, float (&v)[8]) {
  if (left >= 8) {
    if constexpr (sizeof(T) == 4) {
      const u32x4 a = *reinterpret_cast<const u32x4_any *>(p), b = *reinterpret_cast<const u32x4_any *>(p + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = __uint_as_float(a[e]);
        v[4 + e] = __uint_as_float(b[e]);
      }
    } else {
      const u32x4 a = *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = from_bf16(a[e] & 0xffffu);
        v[2 * e + 1] = from_bf16(a[e] >> 16);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? load1(p + e) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, int64_t left, const float (&v)[8]) {
  if (left >= 8) {
    if constexpr (sizeof(T) == 4) {
      u32x4 a, b;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = __float_as_uint(v[e]);
        b[e] = __float_as_uint(v[4 + e]);
      }
      *reinterpret_cast<u32x4_any *>(p) = a;
      *reinterpret_cast<u32x4_any *>(p + 4) = b;
    } else {
      *reinterpret_cast<u32x4_any *>(p) = u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) {
        if constexpr (sizeof(T) == 4) reinterpret_cast<float *>(p)[e] = v[e];
        else p[e] = to_bf16(v[e]);
      }
  }
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(kLanes * kGroups) act_grad_kernel(ActGrad p, int64_t rows_per_slab) {
  __shared__ float sums[GATED ? 1 : kGroups][GATED ? 1 : kTileCols];
  const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kTileCols + lane * kCols, left = p.N - n;
  const int64_t r0 = blockIdx.y * rows_per_slab, r1 = min(r0 + rows_per_slab, p.M);
  float col[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) col[e] = 0.f;
  with_act(p.act, [&](auto A) {
    constexpr int ACT = decltype(A)::value;
    if (left > 0) {
#pragma unroll 2
      for (int64_t m = r0 + grp; m < r1; m += kGroups) {
        float d[8], z[8], o[8];
        load8(static_cast<const T *>(p.d_out) + m * p.ld_dout + n, left, d);
        if (p.pre) load8(static_cast<const T *>(p.pre) + m * p.ld_pre + n, left, z);
        if constexpr (GATED) {
          float u[8], du[8];
          load8(static_cast<const T *>(p.up) + m * p.ld_pre + n, left, u);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const f32x2 a = act_both<ACT>(z[e]);
            du[e] = d[e] * a[0];
            o[e] = d[e] * u[e] * a[1];
          }
          store8(static_cast<T *>(p.d_up) + m * p.N + n, left, du);
          store8(static_cast<T *>(p.d_pre) + m * p.N + n, left, o);
        } else {
          if (ACT != TP_ACT_NONE && p.pre) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = d[e] * act_both<ACT>(z[e])[1];
            if (p.d_pre) store8(static_cast<T *>(p.d_pre) + m * p.N + n, left, o);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = d[e];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) col[e] += o[e];
        }
      }
    }
  });
  if constexpr (!GATED) {
    if (!p.parts) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[grp][lane * kCols + e] = col[e];
    __syncthreads();
    for (int i = threadIdx.x; i < kTileCols; i += kLanes * kGroups) {
      const int64_t c = static_cast<int64_t>(blockIdx.x) * kTileCols + i;
      if (c >= p.N) break;
      p.parts[blockIdx.y * p.N + c] = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
    }
  }
}

// colsum[n] (+)= sum over slabs of parts[slab][n]: 64 columns a workgroup, 16
// groups of slabs, joined in a fixed order.
constexpr int kSumGroups = 16;

__global__ void __launch_bounds__(64 * kSumGroups) colsum_kernel(const float *parts, int64_t slabs, int64_t N,
                                                                 float *out, int accumulate) {
  __shared__ float part[kSumGroups][64];
  const int lane = threadIdx.x % 64, grp = threadIdx.x / 64;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  float v = 0.f;
  if (n < N) {
#pragma unroll 4
    for (int64_t s = grp; s < slabs; s += kSumGroups) v += parts[s * N + n];
  }
  part[grp][lane] = v;
  __syncthreads();
  if (grp == 0 && n < N) {
    float t = part[0][lane];
#pragma unroll
    for (int g = 1; g < kSumGroups; ++g) t += part[g][lane];
    out[n] = accumulate ? out[n] + t : t;
  }
}

// Rows of a slab: 64 (16 rows a lane), more where a slab each would be more
// than 1024 of them (the grid's second dimension, and the partials' size).
int64_t slab_rows(int64_t M) {
  const int64_t r = (M + 1023) / 1024;
  return r < 64 ? 64 : r;
}

template <typename T>
hipError_t launch(const ActGrad& p, hipStream_t s) {
  const int64_t rows = slab_rows(p.M), slabs = (p.M + rows - 1) / rows;
  if (slabs > 0) {
    const dim3 grid(static_cast<unsigned>((p.N + kTileCols - 1) / kTileCols), static_cast<unsigned>(slabs));
    if (p.gated) hipLaunchKernelGGL((act_grad_kernel<T, true>), grid, dim3(kLanes * kGroups), 0, s, p, rows);
    else hipLaunchKernelGGL((act_grad_kernel<T, false>), grid, dim3(kLanes * kGroups), 0, s, p, rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.colsum) {
    hipLaunchKernelGGL(colsum_kernel, dim3(static_cast<unsigned>((p.N + 63) / 64)), dim3(64 * kSumGroups), 0, s, p.parts,
                       slabs, p.N, p.colsum, p.accumulate);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace

int64_t act_grad_slabs(int64_t M, int64_t) {
  const int64_t rows = slab_rows(M);
  return (M + rows - 1) / rows;
}

hipError_t act_grad_launch(const ActGrad& p, hipStream_t s) {
  if (p.N <= 0) return hipSuccess;
  return p.f32 ? launch<uint32_t>(p, s) : launch<uint16_t>(p, s);
}

}  // namespace tpshard
