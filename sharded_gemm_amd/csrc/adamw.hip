// The AdamW step over many tensors, states in fp32 or in 8 bits.
//
//   g = grad * factor                       (clipping's, from the norm's partial sums)
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p - lr (decay p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// All in fp32, one pass: 28 bytes an element with fp32 states and gradients, 16 with
// 8-bit states, 2 more for a bf16 copy of the weights.  Bound by HBM.
//
// 8-bit states: blocks of 256 elements share a scale, the block's largest magnitude of
// m, and of sqrt(v).  Codes are square-law:
//   m = scale * sign(q) (q / 127)^2, q in [-127, 127];  sqrt(v) = scale * (q / 255)^2
// to the nearest q.  What the update has to resolve is sqrt(v), its divisor: half a
// step is 0.4 % of it at the block's largest element, 1.2 % at a tenth, 4 % at a
// hundredth, and the smallest code 1 / 65025 of it.  (An 8-bit float with 3 bits
// of mantissa is off by up to 6 % everywhere, an evenly spaced code ends at 1 / 510.)
// A second moment that is not zero keeps a code of 1 at least, or its element's next
// update would be divided by eps alone.  This step's update uses m and v before they
// are rounded.  A NaN or an infinity in a block makes its scale one, and so every
// value of the block.
//
// The tensors' pointers travel in the kernel's arguments, kMaxAdam a launch.
#include "adamw.h"
#include "linear.h"
#include "linear_dev.h"

namespace tpshard {

using namespace lin;

namespace {

typedef uint32_t u32_byte __attribute__((aligned(1)));

constexpr int kFours = kAdamPer / 4;

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Four values of fp32 or bf16 at element `at`, `left` of which exist.
template <bool F32>
__device__ __forceinline__ f32x4 get(const void *p, int64_t at, int64_t left) {
  if constexpr (F32) return load4<float>(p, at, left);
  else return load4<uint16_t>(p, at, left);
}
template <bool F32>
__device__ __forceinline__ void put(void *p, int64_t at, f32x4 v, int64_t left) {
  if constexpr (F32) store4<float>(p, at, v, left);
  else store4<uint16_t>(p, at, v, left);
}
__device__ __forceinline__ uint32_t get_codes(const void *p, int64_t at, int64_t left) {
  const uint8_t *b = static_cast<const uint8_t *>(p) + at;
  if (left > 3) return *reinterpret_cast<const u32_byte *>(b);
  uint32_t v = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) v |= static_cast<uint32_t>(b[e]) << (8 * e);
  return v;
}
__device__ __forceinline__ void put_codes(void *p, int64_t at, uint32_t v, int64_t left) {
  uint8_t *b = static_cast<uint8_t *>(p) + at;
  if (left > 3) {
    *reinterpret_cast<u32_byte *>(b) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) b[e] = static_cast<uint8_t>(v >> (8 * e));
  }
}

// ---- codes ----------------------------------------------------------------------
// A code that is off by one is a different state, so what leads to it is defined to the
// bit: each operation in fp32 and rounded by itself (no fma), divisions and square
// roots to the nearest.
#pragma clang fp contract(off)

__device__ __forceinline__ f32x4 m_of(uint32_t q, float scale) {
  f32x4 m;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float c = static_cast<float>(static_cast<int32_t>(q << (24 - 8 * e)) >> 24) * (1.0f / 127.0f);
    m[e] = c * fabsf(c) * scale;
  }
  return m;
}
// sqrt(v)
__device__ __forceinline__ f32x4 r_of(uint32_t q, float scale) {
  f32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float c = static_cast<float>(q >> (8 * e) & 0xffu) * (1.0f / 255.0f);
    r[e] = c * c * scale;
  }
  return r;
}

// The largest magnitude of a wave's values, by their bits: a NaN is above everything.
__device__ __forceinline__ float wave_top(f32x4 x) {
  uint32_t b = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) b = max(b, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) b = max(b, static_cast<uint32_t>(__shfl_xor(static_cast<int>(b), o)));
  return __uint_as_float(b);
}

// 1 / top; nothing under 2^-120 is told from zero (an m that small moves no weight, and the square root of an fp32
// is never that small).
__device__ __forceinline__ float over(float top) { return top < 0x1p-120f ? 0.0f : __builtin_amdgcn_rcpf(top); }

// round(codes * sqrt(x / top)), inv about 1 / top: from the hardware's reciprocal and root (an ulp each, so 1e-4 of
// a code at most) unless that is too near the middle between two codes to tell.
__device__ __forceinline__ float code_of(float x, float top, float inv, float codes) {
  const float c = codes * __builtin_amdgcn_sqrtf(x * inv);
  float q = rintf(c);
  if (fabsf(c - q) > 0.4995f && inv > 0.0f) q = rintf(codes * sqrtf(x / top));
  return fminf(q, codes);
}

__device__ __forceinline__ uint32_t m_codes(f32x4 m, float top) {
  const float inv = over(top);
  uint32_t q = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    q |= (static_cast<uint32_t>(static_cast<int32_t>(copysignf(code_of(fabsf(m[e]), top, inv, 127.0f), m[e]))) & 0xffu) << (8 * e);
  return q;
}
__device__ __forceinline__ uint32_t r_codes(f32x4 r, float top) {
  const float inv = over(top);
  uint32_t q = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    q |= static_cast<uint32_t>(r[e] > 0.0f ? fmaxf(code_of(r[e], top, inv, 255.0f), 1.0f) : 0.0f) << (8 * e);
  return q;
}

// ---- the step --------------------------------------------------------------------
struct Scalars {
  float factor, lr, lr1, over2;   // lr1: lr / (1 - b1^t)
};

// What a chunk's lanes load before the scalars are there.
template <bool CODES>
struct Loads {
  f32x4 p[kFours], g[kFours], m[CODES ? 1 : kFours], v[CODES ? 1 : kFours];
  uint32_t mq[CODES ? kFours : 1], vq[CODES ? kFours : 1];
  float ms[CODES ? kFours : 1], vs[CODES ? kFours : 1];
};

template <bool CODES, bool P32, bool G32>
__device__ __forceinline__ void load_as(const AdamTensor& t, int64_t at, int64_t n, Loads<CODES>& l) {
#pragma unroll
  for (int q = 0; q < kFours; ++q) {
    const int64_t i = at + (q * kAdamThreads + static_cast<int>(threadIdx.x)) * 4, left = n - i;
    l.p[q] = get<P32>(t.param, i, left);
    l.g[q] = get<G32>(t.grad, i, left);
    if constexpr (CODES) {
      l.mq[q] = get_codes(t.m, i, left);
      l.vq[q] = get_codes(t.v, i, left);
      l.ms[q] = left > 0 ? t.ms[i / kAdamBlock] : 0.0f;
      l.vs[q] = left > 0 ? t.vs[i / kAdamBlock] : 0.0f;
    } else {
      l.m[q] = get<true>(t.m, i, left);
      l.v[q] = get<true>(t.v, i, left);
    }
  }
}
template <bool CODES>
__device__ __forceinline__ void load(const AdamTensor& t, int64_t at, Loads<CODES>& l) {
  if (t.param_f32) {
    if (t.grad_f32) load_as<CODES, true, true>(t, at, t.n, l);
    else load_as<CODES, true, false>(t, at, t.n, l);
  } else {
    if (t.grad_f32) load_as<CODES, false, true>(t, at, t.n, l);
    else load_as<CODES, false, false>(t, at, t.n, l);
  }
}

template <bool CODES>
__device__ __forceinline__ void step(const AdamTensor& t, int64_t at, const AdamArgs& a, const Scalars& c, Loads<CODES>& l) {
  const float shrink = c.lr * t.decay;
#pragma unroll
  for (int q = 0; q < kFours; ++q) {
    const int64_t i = at + (q * kAdamThreads + static_cast<int>(threadIdx.x)) * 4, left = t.n - i;
    f32x4 m, v, r, p;
    if constexpr (CODES) {
      m = m_of(l.mq[q], l.ms[q]);
      v = r_of(l.vq[q], l.vs[q]);
      v = v * v;
    } else {
      m = l.m[q];
      v = l.v[q];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float g = l.g[q][e] * c.factor;
      m[e] = a.beta1 * m[e] + a.rest1 * g;
      v[e] = a.beta2 * v[e] + a.rest2 * g * g;
      r[e] = sqrtf(v[e]);
      const float move = c.lr1 * m[e] * __builtin_amdgcn_rcpf(fmaf(r[e], c.over2, a.eps));
      p[e] = fmaf(-shrink, l.p[q][e], l.p[q][e]) - move;
    }
    if (t.param_f32) put<true>(t.param, i, p, left);
    else put<false>(t.param, i, p, left);
    if (t.copy) put<false>(t.copy, i, p, left);
    if constexpr (CODES) {
      // Lanes past the end loaded zeros, and hold zeros.
      const float top_m = wave_top(m), top_r = wave_top(r);
      put_codes(t.m, i, m_codes(m, top_m), left);
      put_codes(t.v, i, r_codes(r, top_r), left);
      if ((threadIdx.x & 63) == 0 && left > 0) {
        t.ms[i / kAdamBlock] = top_m;
        t.vs[i / kAdamBlock] = top_r;
      }
    } else {
      put<true>(t.m, i, m, left);
      put<true>(t.v, i, v, left);
    }
  }
}

// Chunks are taken from the last to the first: the norm's pass went the other way, and
// what it read last is still in the cache on the memory side.  The first chunk is on
// its way while the norm is added up.
template <bool CODES>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(AdamTable t, AdamArgs a) {
  __shared__ double lds[kAdamThreads / 64];
  int64_t u = t.first[t.num] - 1 - blockIdx.x;
  int i = t.num - 1;
  auto find = [&]() {
    while (u < t.first[i]) --i;
  };
  Loads<CODES> l;
  if (u >= 0) {
    find();
    load<CODES>(t.t[i], (u - t.first[i]) * kAdamChunk, l);
  }
  Scalars c{1.0f, a.lr_dev ? *a.lr_dev : a.lr, 0.0f, a.over2};
  if (a.parts) {
    double s = 0.0;
    for (int64_t q = threadIdx.x; q < a.ranks * kGradParts; q += kAdamThreads) s += a.parts[q];
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    s = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    const double norm = sqrt(s);
    if (a.norm_out && blockIdx.x == 0 && threadIdx.x == 0) *a.norm_out = static_cast<float>(norm);
    if (a.skip && !__builtin_isfinite(norm)) return;
    const double want = a.max_norm / (norm + a.clip_eps);
    c.factor = want >= 1.0 ? 1.0f : static_cast<float>(want);   // a NaN norm makes a NaN factor
  }
  c.lr1 = c.lr * a.over1;
  if (a.step) {
    const int64_t at = *a.step;
    const double n = static_cast<double>(at > 1 ? at : 1);
    c.lr1 = static_cast<float>(static_cast<double>(c.lr) / (1.0 - exp2(n * a.log2_beta1)));
    c.over2 = static_cast<float>(1.0 / sqrt(1.0 - exp2(n * a.log2_beta2)));
  }
  while (u >= 0) {
    step<CODES>(t.t[i], (u - t.first[i]) * kAdamChunk, a, c, l);
    u -= gridDim.x;
    if (u < 0) break;
    find();
    load<CODES>(t.t[i], (u - t.first[i]) * kAdamChunk, l);
  }
}

__global__ void __launch_bounds__(kAdamThreads) adamw_values_kernel(AdamValuesTable t) {
  int i = 0;
  for (int64_t u = blockIdx.x; u < t.first[t.num]; u += gridDim.x) {
    while (u >= t.first[i + 1]) ++i;
    const AdamValues& x = t.t[i];
    const int64_t at = (u - t.first[i]) * kAdamChunk;
#pragma unroll
    for (int q = 0; q < kFours; ++q) {
      const int64_t e = at + (q * kAdamThreads + static_cast<int>(threadIdx.x)) * 4, left = x.n - e;
      if (left <= 0) continue;
      const f32x4 m = m_of(get_codes(x.m, e, left), x.ms[e / kAdamBlock]);
      const f32x4 r = r_of(get_codes(x.v, e, left), x.vs[e / kAdamBlock]), v = r * r;
      if (x.f32) {
        put<true>(x.m_out, e, m, left);
        put<true>(x.v_out, e, v, left);
      } else {
        put<false>(x.m_out, e, m, left);
        put<false>(x.v_out, e, v, left);
      }
    }
  }
}

// Workgroups of a launch: eight to a CU, each with several chunks in turn where there are more.
unsigned grid_of(int64_t chunks) { return static_cast<unsigned>(chunks < 1 ? 1 : chunks < 2048 ? chunks : 2048); }

}  // namespace

hipError_t adamw_launch(const AdamTensor *ts, int64_t num, bool codes, const AdamArgs& args, hipStream_t s) {
  int64_t at = 0;
  AdamArgs a = args;
  do {   // at least once: the norm is written even where there is nothing to step
    AdamTable t;
    next_adam(ts, num, &at, &t);
    const dim3 grid(grid_of(t.first[t.num]));
    if (codes) hipLaunchKernelGGL(adamw_kernel<true>, grid, dim3(kAdamThreads), 0, s, t, a);
    else hipLaunchKernelGGL(adamw_kernel<false>, grid, dim3(kAdamThreads), 0, s, t, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.norm_out = nullptr;
  } while (at < num);
  return hipSuccess;
}

hipError_t adamw_values_launch(const AdamValues *ts, int64_t num, hipStream_t s) {
  for (int64_t at = 0; at < num;) {
    AdamValuesTable t;
    next_adam(ts, num, &at, &t);
    if (!t.num) break;
    hipLaunchKernelGGL(adamw_values_kernel, dim3(grid_of(t.first[t.num])), dim3(kAdamThreads), 0, s, t);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace tpshard
