// Device code that the linear layer's kernels share: activations, unaligned
// vector access and the product's epilogue.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tpshard.h"
#include "linear.h"

namespace tpshard {
namespace lin {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// The same vectors at an element's own alignment: gfx950 takes global accesses
// of any alignment, so odd strides and offsets keep 16-byte loads.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// ---- bf16 ------------------------------------------------------------------
// Round to nearest, ties to even, NaN kept (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
__device__ __forceinline__ uint16_t to_bf16(float f) { return static_cast<uint16_t>(pack2(f, 0.f)); }
__device__ __forceinline__ float from_bf16(uint32_t bits) { return __uint_as_float(bits << 16); }

template <typename T>
__device__ __forceinline__ float load1(const T *p) {
  if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float *>(p);
  else return from_bf16(*reinterpret_cast<const uint16_t *>(p));
}

// ---- 16 bytes ------------------------------------------------------------------
// 16 bytes of T at p, of which `left` elements exist (the rest read as zero).
template <typename T>
__device__ __forceinline__ u32x4 load16(const T *p, int64_t left) {
  constexpr int V = 16 / sizeof(T);
  if (left >= V) return *reinterpret_cast<const u32x4_any *>(p);
  u32x4 v{0, 0, 0, 0};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) v[e] = p[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) v[e >> 1] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
  }
  return v;
}

// ---- activations -------------------------------------------------------------
// All in fp32 on the hardware's exp2 and reciprocal (about 1 ulp each).
//  gelu_erf : x Phi(x); with a = |x|, q = Phi(-a) = e^{-x^2/2} t P(t), t = 1 / (1 + 0.21 a), Phi = 1 - q
//             for x >= 0, q below.  t P(t) is erfc(a / sqrt 2) e^{x^2/2} / 2, P of degree 8 fitted to it by
//             linear programming, minimax in the relative error over a <= 13.5 (1.4e-8; beyond, q
//             underflows).  So the tail is relatively exact too: with Abramowitz & Stegun's 7.1.26, four
//             terms shorter and within 1.5e-7 absolutely, x = -3 was off by 6e-5 and x = -8 by 1 %.
//  gelu_tanh: x s(2 v), v = sqrt(2/pi) (x + 0.044715 x^3), s the logistic function
//             (1 + tanh v = 2 s(2 v)).
//  silu     : x s(x).
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float logistic(float x) {
  // 1 / (1 + 2^{-x log2 e}): exp2 overflows to inf and the quotient to 0.
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

__device__ __forceinline__ float gelu_cdf(float x) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.21f, fabsf(x), 1.0f));
  float poly = fmaf(t, -0.0720329499f, 0.285448524f);
  poly = fmaf(t, poly, -0.334179842f);
  poly = fmaf(t, poly, 0.354022695f);
  poly = fmaf(t, poly, -0.0972383039f);
  poly = fmaf(t, poly, 0.126352044f);
  poly = fmaf(t, poly, 0.0687908271f);
  poly = fmaf(t, poly, 0.0851292977f);
  poly = fmaf(t, poly, 0.0837077095f);
  const float q = t * poly * __builtin_amdgcn_exp2f(x * (x * (-0.5f * kLog2e)));
  return x >= 0.0f ? 1.0f - q : q;
}

constexpr float kTanhA = 0.79788456080286535588f;   // sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_fwd(float x) {
  if constexpr (ACT == TP_ACT_GELU_ERF) return x * gelu_cdf(x);
  else if constexpr (ACT == TP_ACT_GELU_TANH) return x * logistic(2.0f * kTanhA * x * fmaf(kTanhB * x, x, 1.0f));
  else if constexpr (ACT == TP_ACT_SILU) return x * logistic(x);
  else if constexpr (ACT == TP_ACT_RELU) return x < 0.0f ? 0.0f : x;   // a NaN stays one
  else return x;
}

// (act(x), act'(x)).  Where the factor that x multiplies has run out (far x),
// the derivative is its limit, not inf * 0.
template <int ACT>
__device__ __forceinline__ f32x2 act_both(float x) {
  if constexpr (ACT == TP_ACT_GELU_ERF) {
    const float cdf = gelu_cdf(x);
    const float pdf = 0.39894228040143267794f * __builtin_amdgcn_exp2f(x * (x * (-0.5f * kLog2e)));
    return f32x2{x * cdf, pdf == 0.0f ? cdf : fmaf(x, pdf, cdf)};
  } else if constexpr (ACT == TP_ACT_GELU_TANH) {
    const float s = logistic(2.0f * kTanhA * x * fmaf(kTanhB * x, x, 1.0f));
    const float dv = 2.0f * kTanhA * fmaf(3.0f * kTanhB * x, x, 1.0f);
    const float ds = s * (1.0f - s);
    return f32x2{x * s, ds == 0.0f ? s : fmaf(x * dv, ds, s)};
  } else if constexpr (ACT == TP_ACT_SILU) {
    const float s = logistic(x);
    const float ds = s * (1.0f - s);
    return f32x2{x * s, ds == 0.0f ? s : fmaf(x, ds, s)};
  } else if constexpr (ACT == TP_ACT_RELU) {
    return f32x2{x < 0.0f ? 0.0f : x, x > 0.0f ? 1.0f : 0.0f};
  } else {
    return f32x2{x, 1.0f};
  }
}

template <int V>
struct Const {
  static constexpr int value = V;
};

// f(Const<act>): the activation becomes a compile-time constant of the code
// that uses it; `act` is uniform, so this is one scalar branch.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case TP_ACT_GELU_ERF: f(Const<TP_ACT_GELU_ERF>{}); break;
    case TP_ACT_GELU_TANH: f(Const<TP_ACT_GELU_TANH>{}); break;
    case TP_ACT_SILU: f(Const<TP_ACT_SILU>{}); break;
    case TP_ACT_RELU: f(Const<TP_ACT_RELU>{}); break;
    default: f(Const<TP_ACT_NONE>{}); break;
  }
}

// ---- several workgroups to a tile ---------------------------------------------
// Every workgroup of a tile leaves its partial sums; the one that finds all the
// others' done adds them, in their order, so that the result does not depend on
// who that is.  Nobody waits for anybody, and the ticket ends at zero again.
//
// The partials are device-scope accesses: such a store is past this XCD's own L2
// once vmcnt has counted it, and such a load does not read a stale line there,
// so no cache is written back or invalidated.  (A device fence writes the whole
// L2 back: one per wave made a 51 us product take 531.)
__device__ __forceinline__ void put_partial(float *p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float get_partial(const float *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void put_partial(f32x2 *p, f32x2 v) {
  __hip_atomic_store(reinterpret_cast<uint64_t *>(p), __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x2 get_partial(const f32x2 *p) {
  return __builtin_bit_cast(f32x2, __hip_atomic_load(reinterpret_cast<const uint64_t *>(p), __ATOMIC_RELAXED,
                                                     __HIP_MEMORY_SCOPE_AGENT));
}

// After this workgroup's put_partial calls: whether it is the tile's last.
__device__ __forceinline__ bool last_of_tile(uint32_t *ticket, uint32_t splits) {
  __shared__ uint32_t before;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  // Counts 0 .. splits - 1 and wraps to 0: even overlapping replays of one call,
  // which would spoil each other's result, leave the ticket at zero.
  if (threadIdx.x == 0) before = atomicInc(ticket, splits - 1);
  __syncthreads();
  return before + 1 == splits;
}

// out[i] = sum over y < splits, in order, of p[y * pitch + at(i)], with at least
// eight loads in flight at a time (a round trip to the memory side each batch).
template <int N, typename V, typename At>
__device__ __forceinline__ void sum_partials(const V *p, int64_t pitch, At&& at, int splits, V (&out)[N]) {
  constexpr int Y = N >= 8 ? 1 : 8 / N;   // splits of a batch
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = V{};
  for (int y0 = 0; y0 < splits; y0 += Y) {
    V v[Y][N];
#pragma unroll
    for (int y = 0; y < Y; ++y)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (y0 + y < splits) v[y][i] = get_partial(p + (y0 + y) * pitch + at(i));
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int y = 0; y < Y; ++y)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (y0 + y < splits) out[i] = out[i] + v[y][i];
  }
}

// The accumulators of workgroup (blockIdx.x, blockIdx.y): left as a partial; true
// in the tile's last workgroup, whose acc then holds the sum over all.
template <int THREADS, int TM, int TN>
__device__ __forceinline__ bool join_splits(const LinGemm& p, f32x4 (&acc)[TM][TN]) {
  constexpr int64_t PITCH = TM * TN * 2 * THREADS;   // f32x2 of one workgroup
  const int splits = gridDim.y;
  f32x2 *tile = reinterpret_cast<f32x2 *>(p.join) + static_cast<int64_t>(blockIdx.x) * splits * PITCH + threadIdx.x;
  f32x2 *mine = tile + blockIdx.y * PITCH;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        put_partial(mine + ((i * TN + j) * 2 + h) * THREADS, f32x2{acc[i][j][2 * h], acc[i][j][2 * h + 1]});
  if (!last_of_tile(p.tickets + blockIdx.x, splits)) return false;
  f32x2 sum[TM * TN * 2];
  sum_partials(tile, PITCH, [](int i) { return i * THREADS; }, splits, sum);
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = sum[(i * TN + j) * 2 + e / 2][e % 2];
  return true;
}

// ---- four columns of an output row ---------------------------------------------
// `left` of them exist.  Four go in one access at an element's own alignment;
// element by element where rows are odd, each of the four stores leaves a quarter
// of every line: 8191 x 333 x 2333 bf16 61 us against 47, two 8064 x 4333 fp32
// weight gradients over 128 rows 338 against 257.

template <typename T>
__device__ __forceinline__ f32x4 load4(const void *base, int64_t off, int64_t left) {
  const T *p = static_cast<const T *>(base) + off;
  f32x4 v{0.f, 0.f, 0.f, 0.f};
  if (left > 3) {
    if constexpr (sizeof(T) == 4) {
      v = *reinterpret_cast<const f32x4_any *>(p);
    } else {
      const u32x2 w = *reinterpret_cast<const u32x2_any *>(p);
      v = f32x4{from_bf16(w[0] & 0xffffu), from_bf16(w[0] >> 16), from_bf16(w[1] & 0xffffu), from_bf16(w[1] >> 16)};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) v[e] = load1(p + e);
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void store4(void *base, int64_t off, f32x4 v, int64_t left) {
  T *p = static_cast<T *>(base) + off;
  if (left > 3) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4_any *>(p) = v;
    else *reinterpret_cast<u32x2_any *>(p) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<float *>(p + e) = v[e];
        else *reinterpret_cast<uint16_t *>(p + e) = to_bf16(v[e]);
      }
  }
}

__device__ __forceinline__ void store4_c(const LinGemm& p, void *c, int64_t off, f32x4 v, int64_t left) {
  if (p.c_f32) {
    if (p.acc_c) v = load4<float>(c, off, left) + v;
    store4<float>(c, off, v, left);
  } else {
    store4<uint16_t>(c, off, v, left);
  }
}

// The epilogue of one lane's accumulators: acc[i][j] is row rm(i), columns
// cn(j) .. cn(j) + 3.  With kModeDual the first TN / 2 fragments of a row are
// the gate's and the rest the up projection's, at the same columns.
// T: the operands' type.  Loads of a row (residual, bias) come before its
// stores, which the compiler may not reorder by itself (the residual may be
// the output).
template <typename T, int MODE, int TM, int TN, typename RM, typename CN>
__device__ __forceinline__ void epilogue(const LinGemm& p, void *c, const f32x4 (&acc)[TM][TN], RM&& rm, CN&& cn) {
  constexpr int NJ = MODE == kModeDual ? TN / 2 : TN;
  if constexpr (MODE == kModeCat || MODE == kModePair) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int64_t m = rm(i), n = cn(j), left = p.N - n;
        if (m < p.M && left > 0) store4_c(p, c, m * p.ldc + n, acc[i][j], left);
      }
  } else {
    with_act(p.act, [&](auto A) {
      constexpr int ACT = decltype(A)::value;
      f32x4 bias[NJ];
      if constexpr (MODE == kModeOne) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int64_t n = cn(j), left = p.N - n;
          bias[j] = p.bias && left > 0 ? load4<float>(p.bias, n, left) : f32x4{0.f, 0.f, 0.f, 0.f};
        }
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int64_t m = rm(i);
        if (m >= p.M) continue;
        f32x4 res[NJ];
        if constexpr (MODE == kModeOne) {
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int64_t n = cn(j), left = p.N - n;
            res[j] = p.res && left > 0 ? load4<T>(p.res, m * p.ldres + n, left)
                                       : f32x4{0.f, 0.f, 0.f, 0.f};
          }
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int64_t n = cn(j), left = p.N - n;
          if (left <= 0) continue;
          f32x4 y;
          if constexpr (MODE == kModeDual) {
            const f32x4 g = acc[i][j], u = acc[i][j + NJ];
            if (p.aux) store4<T>(p.aux, m * p.ldaux + n, g, left);
            if (p.aux2) store4<T>(p.aux2, m * p.ldaux + n, u, left);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = act_fwd<ACT>(g[e]) * u[e];
          } else {
            const f32x4 pre = p.bias ? acc[i][j] + bias[j] : acc[i][j];
            if (p.aux) store4<T>(p.aux, m * p.ldaux + n, pre, left);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = act_fwd<ACT>(pre[e]);
            if (p.res) y = y + res[j];
          }
          store4_c(p, c, m * p.ldc + n, y, left);
        }
      }
    });
  }
}

}  // namespace lin
}  // namespace tpshard
