// Gradients at the activation of the linear layer and of the gated block, and
// the bias gradient's column sums.
//
//   linear: dPre = dOut * act'(pre);         dbias[n] = sum over m of dPre[m, n]
//   gated : dU = dOut * act(G);              dG = dOut * U * act'(G)
//
// One pass over the inputs, memory-bound.  The gated form without row strides is
// one flat array, 8 elements a lane.  Otherwise a workgroup takes up to 512
// columns by a slab of rows, each lane 8 columns (16 bytes of bf16).  The column
// sums add the unrounded fp32 values; each slab leaves its own partial row and a
// second kernel adds the slabs in order, so no atomics decide the result.
//
// dPre, dU and dG are rounded once to the operands' type: the two products that
// read them next are bf16 matrix instructions then, at twice the rate of a product
// over two bf16 halves of each value (and nine times fp32's).  It adds one rounding
// to dX and dW: 2.35e-3 of the norm from exact where the stored result's own
// rounding is 1.66e-3.
//
// Measured on an MI355X (copy 5.2 TB/s): gated 8192 x 2048 bf16 30 us (5.6 TB/s),
// linear 8192 x 4096 with GeLU and its bias gradient 44 + 4 us (4.5 TB/s).
#include "linear_dev.h"

namespace tpshard {

using namespace lin;

namespace {

constexpr int kThreads = kActThreads, kCols = kActCols;

// Eight elements at p; `left` exist.  `on`: there are at least eight elements of
// the array from p on, so the missing ones are read from the next rows (and not
// used); otherwise they read as zero.
template <typename T>
__device__ __forceinline__ void load8(const T *p, int64_t left, bool on, float (&v)[8]) {
  if (left >= 8 || on) {
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

template <typename T, int ACT>
__device__ __forceinline__ void gated8(const float (&d)[8], const float (&z)[8], const float (&u)[8], float (&dg)[8],
                                       float (&du)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const f32x2 a = act_both<ACT>(z[e]);
    du[e] = d[e] * a[0];
    dg[e] = d[e] * u[e] * a[1];
  }
}

// The first workgroup clears the tickets of the products that follow.
__device__ __forceinline__ void zero_tickets(uint32_t *tickets) {
  if (tickets && blockIdx.x == 0 && blockIdx.y == 0)
    for (int64_t i = threadIdx.x; i < kMaxTickets; i += blockDim.x) tickets[i] = 0;
}

__global__ void __launch_bounds__(kThreads) zero_tickets_kernel(uint32_t *tickets) { zero_tickets(tickets); }

template <typename T>
__global__ void __launch_bounds__(kThreads) gated_grad_flat(ActGrad p) {
  zero_tickets(p.tickets);
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * kCols, left = p.M * p.N - at;
  if (left <= 0) return;
  float d[8], z[8], u[8], dg[8], du[8];
  load8(static_cast<const T *>(p.d_out) + at, left, false, d);
  load8(static_cast<const T *>(p.pre) + at, left, false, z);
  load8(static_cast<const T *>(p.up) + at, left, false, u);
  with_act(p.act, [&](auto A) { gated8<T, decltype(A)::value>(d, z, u, dg, du); });
  store8(static_cast<T *>(p.d_up) + at, left, du);
  store8(static_cast<T *>(p.d_pre) + at, left, dg);
}

// lanes: of a row (a power of two); the workgroup's 256 / lanes groups take the
// slab's rows in turn.
template <typename T, bool GATED>
__global__ void __launch_bounds__(kThreads) act_grad_kernel(ActGrad p, int64_t rows_per_slab, int lanes) {
  __shared__ float sums[GATED ? 1 : kThreads * kCols];
  zero_tickets(p.tickets);
  const int lane = threadIdx.x & (lanes - 1), grp = threadIdx.x / lanes, groups = kThreads / lanes;
  const int cols = lanes * kCols;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * cols + lane * kCols, left = p.N - n;
  const int64_t r0 = blockIdx.y * rows_per_slab, r1 = min(r0 + rows_per_slab, p.M);
  float col[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) col[e] = 0.f;
  with_act(p.act, [&](auto A) {
    constexpr int ACT = decltype(A)::value;
    if (left > 0) {
#pragma unroll 2
      for (int64_t m = r0 + grp; m < r1; m += groups) {
        // Seven more rows hold seven more elements, whatever their stride.
        const bool on = m + 7 < p.M;
        float d[8], z[8], o[8];
        load8(static_cast<const T *>(p.d_out) + m * p.ld_dout + n, left, on, d);
        if (p.pre) load8(static_cast<const T *>(p.pre) + m * p.ld_pre + n, left, on, z);
        if constexpr (GATED) {
          float u[8], du[8];
          load8(static_cast<const T *>(p.up) + m * p.ld_pre + n, left, on, u);
          gated8<T, ACT>(d, z, u, o, du);
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
    for (int e = 0; e < 8; ++e) sums[grp * cols + lane * kCols + e] = col[e];
    __syncthreads();
    for (int i = threadIdx.x; i < cols; i += kThreads) {
      const int64_t c = static_cast<int64_t>(blockIdx.x) * cols + i;
      if (c >= p.N) break;
      float v = sums[i];
      for (int g = 1; g < groups; ++g) v += sums[g * cols + i];
      p.parts[blockIdx.y * p.N + c] = v;
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

template <typename T>
hipError_t launch(const ActGrad& p, hipStream_t s) {
  const ActGrid g = act_grad_grid(p.M, p.N);
  if (p.M > 0) {
    const dim3 grid(static_cast<unsigned>(g.tiles), static_cast<unsigned>(g.slabs));
    const int64_t flat = (p.M * p.N + kThreads * kCols - 1) / (kThreads * kCols);
    if (p.gated && p.ld_dout == p.N && p.ld_pre == p.N && flat < (int64_t{1} << 23))
      hipLaunchKernelGGL((gated_grad_flat<T>), dim3(static_cast<unsigned>(flat)), dim3(kThreads), 0, s, p);
    else if (p.gated)
      hipLaunchKernelGGL((act_grad_kernel<T, true>), grid, dim3(kThreads), 0, s, p, g.rows, g.lanes);
    else
      hipLaunchKernelGGL((act_grad_kernel<T, false>), grid, dim3(kThreads), 0, s, p, g.rows, g.lanes);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.colsum) {
    hipLaunchKernelGGL(colsum_kernel, dim3(static_cast<unsigned>((p.N + 63) / 64)), dim3(64 * kSumGroups), 0, s, p.parts,
                       g.slabs, p.N, p.colsum, p.accumulate);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace

hipError_t zero_tickets_launch(uint32_t *tickets, hipStream_t s) {
  hipLaunchKernelGGL(zero_tickets_kernel, dim3(1), dim3(kThreads), 0, s, tickets);
  return hipGetLastError();
}

hipError_t act_grad_launch(const ActGrad& p, hipStream_t s) {
  if (p.N <= 0) return hipSuccess;
  return p.f32 ? launch<uint32_t>(p, s) : launch<uint16_t>(p, s);
}

}  // namespace tpshard
