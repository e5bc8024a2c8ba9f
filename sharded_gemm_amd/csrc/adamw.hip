// The AdamW step over many tensors, states in fp32 or in 8 bits.
//
//   g = grad * factor                       (clipping's, from the norm's partial sums)
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p - lr (decay p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// All in fp32, one pass: 28 bytes an element with fp32 states and gradients, 16 with
// 8-bit states, 2 more for a bf16 copy of the weights.  Bound by HBM: 201M elements, MI355X,
// fp32 states 1028 us (5.5 TB/s), 8-bit ones 571 (5.6), with bf16 weights and gradients 814 (5.4) and
// 444 (4.5, bound by the instructions: some 60 an element); 8-bit states as bf16 values
// 206 (5.9).  1.8M elements 6.8 and 8.0, a launch's latency.
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

#include <algorithm>

#include "linear.h"
#include "linear_dev.h"

namespace tpshard {

using namespace lin;

namespace {

typedef uint32_t u32_byte __attribute__((aligned(1)));

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Elements of a chunk: 32-bit offsets from its start, which is the same for all lanes.
template <bool F32>
__device__ __forceinline__ const void *from(const void *p, int64_t at) {
  return static_cast<const char *>(p) + at * (F32 ? 4 : 2);
}
template <bool F32>
__device__ __forceinline__ void *from(void *p, int64_t at) {
  return static_cast<char *>(p) + at * (F32 ? 4 : 2);
}
__device__ __forceinline__ const uint8_t *codes_from(const void *p, int64_t at) { return static_cast<const uint8_t *>(p) + at; }

// Four values of fp32 or bf16 at element i, as they lie there.
template <bool F32>
__device__ __forceinline__ u32x4 get(const void *p, uint32_t i) {
  if constexpr (F32) return __builtin_bit_cast(u32x4, *reinterpret_cast<const f32x4_any *>(static_cast<const float *>(p) + i));
  const u32x2 w = *reinterpret_cast<const u32x2_any *>(static_cast<const uint16_t *>(p) + i);
  return u32x4{w[0], w[1], 0, 0};
}
__device__ __forceinline__ u32x4 widen(u32x4 w) { return u32x4{w[0] << 16, w[0] & 0xffff0000u, w[1] << 16, w[1] & 0xffff0000u}; }
// One by one, with the last of n in place of those past it, as fp32's bits.
template <bool F32>
__device__ __forceinline__ u32x4 get_last(const void *p, uint32_t i, uint32_t n) {
  u32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t at = min(i + e, n - 1);
    v[e] = F32 ? static_cast<const uint32_t *>(p)[at] : static_cast<uint32_t>(static_cast<const uint16_t *>(p)[at]) << 16;
  }
  return v;
}
// Zero from element `left` on.
__device__ __forceinline__ u32x4 first_of(u32x4 v, int left) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = e < left ? v[e] : 0u;
  return v;
}
template <bool F32>
__device__ __forceinline__ void put(void *p, uint32_t i, f32x4 v, int left) {
  if constexpr (F32) store4<float>(p, i, v, left);
  else store4<uint16_t>(p, i, v, left);
}
__device__ __forceinline__ uint32_t get_codes(const uint8_t *p, uint32_t i) { return *reinterpret_cast<const u32_byte *>(p + i); }
__device__ __forceinline__ u32x4 get_last_codes(const uint8_t *p, uint32_t i, uint32_t n) {
  u32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = p[min(i + e, n - 1)];
  return v;
}
__device__ __forceinline__ uint32_t pack(u32x4 v) { return v[0] | v[1] << 8 | v[2] << 16 | v[3] << 24; }
__device__ __forceinline__ void put_codes(uint8_t *b, uint32_t i, uint32_t v, int left) {
  b += i;
  if (left > 3) {
    *reinterpret_cast<u32_byte *>(b) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) b[e] = static_cast<uint8_t>(v >> (8 * e));
  }
}
// A lane's element of its four q in a chunk; the elements of a chunk at `at` of n.
__device__ __forceinline__ uint32_t element(int q) { return (q * kAdamThreads + threadIdx.x) * 4; }
template <int CHUNK>
__device__ __forceinline__ uint32_t elements(int64_t n, int64_t at) {
  return static_cast<uint32_t>(n - at < CHUNK ? n - at : CHUNK);
}

// The tensor of chunk u: tables hold up to 64, one to a lane, which holds the chunks up to its end.
struct Finder {
  int64_t end;
  template <typename Table>
  __device__ __forceinline__ explicit Finder(const Table& t) {
    const int lane = threadIdx.x & 63;
    end = lane < t.num ? t.first[lane + 1] : INT64_MAX;
  }
  __device__ __forceinline__ int operator()(int64_t u) const { return __popcll(__ballot(end <= u)); }
};

// ---- codes ----------------------------------------------------------------------
// A code that is off by one is a different state, so what leads to it is defined to the
// bit: each operation in fp32 and rounded by itself (no fma), divisions and square
// roots to the nearest.  Faster ways to the same codes are below.
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

// The largest of a wave's values of x >= 0, by their bits: a NaN is above everything.  Lanes of 16 join by data-parallel
// moves, which the maximum takes as an operand, and the rest by swaps.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t x) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_top(u32x4 x) {
  uint32_t b = max(max(x[0], x[1]), max(x[2], x[3]));
  b = max(b, moved<0xb1>(b));    // lane ^ 1
  b = max(b, moved<0x4e>(b));    // lane ^ 2
  b = max(b, moved<0x141>(b));   // 7 - lane of eight
  b = max(b, moved<0x140>(b));   // 15 - lane of sixteen
  auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  b = max(r[0], r[1]);
  r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(max(r[0], r[1]));
}
__device__ __forceinline__ u32x4 bits_of(f32x4 x) { return __builtin_bit_cast(u32x4, x); }

// The codes of four values: rounded c = sqrt(x k), from the hardware's root (x and k are off by an ulp at most, and the
// root by another: 1e-4 of a code in all), unless that is too near the middle between two codes to tell, or `all` is
// set: then exact(e).
template <typename F>
__device__ __forceinline__ f32x4 codes_of(f32x4 x, float k, bool all, F&& exact) {
  constexpr float kNear = 0.4998f;
  f32x4 q, off;
  float most = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float c = __builtin_amdgcn_sqrtf(x[e] * k);
    q[e] = rintf(c);
    off[e] = fabsf(c - q[e]);
    most = fmaxf(most, off[e]);
  }
  if (all || most > kNear) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (all || off[e] > kNear) q[e] = rintf(exact(e));
  }
  return q;
}

// round(127 sqrt(|m| / top)) with m's sign; nothing under 2^-112 is told from zero (an m that small moves no weight).
__device__ __forceinline__ uint32_t m_codes(f32x4 m, float top) {
  const float k = top < 0x1p-112f ? 0.0f : 16129.0f * __builtin_amdgcn_rcpf(top);
  f32x4 x;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = fabsf(m[e]);
  const f32x4 c = codes_of(x, k, top > 0x1p125f, [&](int e) { return 127.0f * sqrtf(x[e] / top); });   // (no 1 / top there)
  uint32_t q = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) q = __builtin_amdgcn_cvt_pk_u8_f32(copysignf(fminf(c[e], 127.0f), m[e]) + 128.0f, e, q);
  return q ^ 0x80808080u;
}
// round(255 sqrt(sqrt(v) / top)), 1 at least where v is not zero.  r: sqrt(v) to an ulp (0 for subnormals); v_top: the
// largest v, and top its root.
__device__ __forceinline__ uint32_t v_codes(f32x4 v, f32x4 r, float v_top, float top) {
  const f32x4 c = codes_of(r, 65025.0f * __builtin_amdgcn_rcpf(top), v_top < 0x1p-90f,
                           [&](int e) { return 255.0f * sqrtf(sqrtf(v[e]) / top); });
  uint32_t q = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) q = __builtin_amdgcn_cvt_pk_u8_f32(v[e] > 0.0f ? fmaxf(c[e], 1.0f) : 0.0f, e, q);
  return q;
}

// ---- the step --------------------------------------------------------------------
struct Scalars {
  float factor, lr, lr1, over2;   // lr1: lr / (1 - b1^t)
  bool root;                      // sqrt(v) of a subnormal v may be taken for 0: eps is far above it
};

// Long chunks are whole.  A tensor's end is taken in short ones, whose code goes element by element there: kept
// apart, it costs the stream no registers (106, 134 with ends in long chunks).
template <int CHUNK>
constexpr bool whole = CHUNK == kAdamChunk;

// What a chunk's lanes load before the scalars are there.  Whole chunks are kept as they
// lie in memory, so that nothing waits for a load until the step itself; a tensor's last
// chunk is converted, with zeros past the end.
template <bool CODES, int CHUNK>
struct Loads {
  static constexpr int kFours = CHUNK / kAdamThreads / 4;
  u32x4 p[kFours], g[kFours], m[CODES ? 1 : kFours], v[CODES ? 1 : kFours];
  uint32_t mq[CODES ? kFours : 1], vq[CODES ? kFours : 1];
  float ms[CODES ? kFours : 1], vs[CODES ? kFours : 1];
};

template <bool P32, bool G32, bool CODES, int CHUNK>
__device__ __forceinline__ void load_as(const AdamTensor& t, int64_t at, Loads<CODES, CHUNK>& l) {
  constexpr int kFours = Loads<CODES, CHUNK>::kFours;
  const uint32_t n = whole<CHUNK> ? CHUNK : elements<CHUNK>(t.n, at);
  const void *param = from<P32>(t.param, at), *grad = from<G32>(t.grad, at);
  const void *m32 = from<true>(t.m, at), *v32 = from<true>(t.v, at);
  const uint8_t *mc = codes_from(t.m, at), *vc = codes_from(t.v, at);
  const float *ms = CODES ? t.ms + at / kAdamBlock : nullptr, *vs = CODES ? t.vs + at / kAdamBlock : nullptr;
  if (n == CHUNK) {
#pragma unroll
    for (int q = 0; q < kFours; ++q) {
      const uint32_t i = element(q);
      l.p[q] = get<P32>(param, i);
      l.g[q] = get<G32>(grad, i);
      if constexpr (CODES) {
        l.mq[q] = get_codes(mc, i);
        l.vq[q] = get_codes(vc, i);
        l.ms[q] = ms[i / kAdamBlock];
        l.vs[q] = vs[i / kAdamBlock];
      } else {
        l.m[q] = get<true>(m32, i);
        l.v[q] = get<true>(v32, i);
      }
    }
    return;
  }
  u32x4 m[kFours], v[kFours];
#pragma unroll
  for (int q = 0; q < kFours; ++q) {
    const uint32_t i = element(q);
    l.p[q] = get_last<P32>(param, i, n);
    l.g[q] = get_last<G32>(grad, i, n);
    m[q] = CODES ? get_last_codes(mc, i, n) : get_last<true>(m32, i, n);
    v[q] = CODES ? get_last_codes(vc, i, n) : get_last<true>(v32, i, n);
    if constexpr (CODES) {
      l.ms[q] = ms[min(i, n - 1) / kAdamBlock];
      l.vs[q] = vs[min(i, n - 1) / kAdamBlock];
    }
  }
#pragma unroll
  for (int q = 0; q < kFours; ++q) {
    const int left = static_cast<int>(n - element(q));
    l.p[q] = first_of(l.p[q], left);
    l.g[q] = first_of(l.g[q], left);
    if constexpr (CODES) {
      l.mq[q] = pack(first_of(m[q], left));
      l.vq[q] = pack(first_of(v[q], left));
    } else {
      l.m[q] = first_of(m[q], left);
      l.v[q] = first_of(v[q], left);
    }
  }
}
template <bool CODES, int CHUNK>
__device__ __forceinline__ void load(const AdamTensor& t, int64_t at, Loads<CODES, CHUNK>& l) {
  if (t.param_f32) {
    if (t.grad_f32) load_as<true, true>(t, at, l);
    else load_as<true, false>(t, at, l);
  } else {
    if (t.grad_f32) load_as<false, true>(t, at, l);
    else load_as<false, false>(t, at, l);
  }
}

template <bool CODES, int CHUNK>
__device__ __forceinline__ void step(const AdamTensor& t, int64_t at, const AdamArgs& a, const Scalars& c, Loads<CODES, CHUNK>& l) {
  constexpr int kFours = Loads<CODES, CHUNK>::kFours;
  const float shrink = c.lr * t.decay;
  const uint32_t n = whole<CHUNK> ? CHUNK : elements<CHUNK>(t.n, at);
#pragma unroll
  for (int q = 0; q < kFours; ++q) {
    if (n == CHUNK && !t.param_f32) l.p[q] = widen(l.p[q]);
    if (n == CHUNK && !t.grad_f32) l.g[q] = widen(l.g[q]);
  }
#pragma unroll
  for (int q = 0; q < kFours; ++q) {
    const uint32_t i = element(q);
    const int left = whole<CHUNK> ? 4 : static_cast<int>(n - i);
    const f32x4 w = __builtin_bit_cast(f32x4, l.p[q]), dw = __builtin_bit_cast(f32x4, l.g[q]);
    f32x4 m, v, r, p;
    if constexpr (CODES) {
      m = m_of(l.mq[q], l.ms[q]);
      v = r_of(l.vq[q], l.vs[q]);
      v = v * v;
    } else {
      m = __builtin_bit_cast(f32x4, l.m[q]);
      v = __builtin_bit_cast(f32x4, l.v[q]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float g = dw[e] * c.factor;
      m[e] = a.beta1 * m[e] + a.rest1 * g;
      v[e] = a.beta2 * v[e] + a.rest2 * g * g;
      r[e] = CODES && c.root ? __builtin_amdgcn_sqrtf(v[e]) : sqrtf(v[e]);
      const float move = c.lr1 * m[e] * __builtin_amdgcn_rcpf(fmaf(r[e], c.over2, a.eps));
      p[e] = fmaf(-shrink, w[e], w[e]) - move;
    }
    if (t.param_f32) put<true>(from<true>(t.param, at), i, p, left);
    else put<false>(from<false>(t.param, at), i, p, left);
    if (t.copy) put<false>(from<false>(t.copy, at), i, p, left);
    if constexpr (CODES) {
      // Lanes past the end hold zeros.
      u32x4 size = bits_of(m);
#pragma unroll
      for (int e = 0; e < 4; ++e) size[e] &= 0x7fffffffu;
      const float top_m = wave_top(size), top_v = wave_top(bits_of(v)), top_r = sqrtf(top_v);
      put_codes(static_cast<uint8_t *>(t.m) + at, i, m_codes(m, top_m), left);
      put_codes(static_cast<uint8_t *>(t.v) + at, i, v_codes(v, r, top_v, top_r), left);
      if ((threadIdx.x & 63) == 0 && left > 0) {
        t.ms[at / kAdamBlock + i / kAdamBlock] = top_m;
        t.vs[at / kAdamBlock + i / kAdamBlock] = top_r;
      }
    } else {
      put<true>(from<true>(t.m, at), i, m, left);
      put<true>(from<true>(t.v, at), i, v, left);
    }
  }
}

// Chunks are taken from the last to the first: the norm's pass went the other way, and
// what it read last is still in the cache on the memory side.  The first chunk is on
// its way while the norm is added up.
template <bool CODES, int CHUNK>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(AdamTable t, AdamArgs a) {
  __shared__ double lds[kAdamThreads / 64];
  const Finder find(t);
  int64_t u = t.first[t.num] - 1 - blockIdx.x;
  int i = 0;
  Loads<CODES, CHUNK> l;
  if (u >= 0) {
    i = find(u);
    load(t.t[i], (u - t.first[i]) * CHUNK, l);
  }
  Scalars c{1.0f, a.lr_dev ? *a.lr_dev : a.lr, 0.0f, a.over2, false};
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
  c.root = a.eps > c.over2 * 0x1p-38f;
  while (u >= 0) {
    step(t.t[i], (u - t.first[i]) * CHUNK, a, c, l);
    u -= gridDim.x;
    if (u < 0) break;
    i = find(u);
    load(t.t[i], (u - t.first[i]) * CHUNK, l);
  }
  if constexpr (whole<CHUNK>) {   // what is left of each tensor: less than a chunk, so up to four short ones
    constexpr int S = CHUNK / kAdamShort;
#pragma unroll 1
    for (int w = blockIdx.x; w < t.num * S; w += gridDim.x) {
      const AdamTensor& x = t.t[w / S];
      const int64_t at = x.n / CHUNK * CHUNK + w % S * kAdamShort;
      if (at >= x.n) continue;
      Loads<CODES, kAdamShort> end;
      load(x, at, end);
      step(x, at, a, c, end);
    }
  }
}

__global__ void __launch_bounds__(kAdamThreads) adamw_values_kernel(AdamValuesTable t) {
  constexpr int kFours = kAdamChunk / kAdamThreads / 4;
  const Finder find(t);
  for (int64_t u = blockIdx.x; u < t.first[t.num]; u += gridDim.x) {
    const int i = find(u);
    const AdamValues& x = t.t[i];
    const int64_t at = (u - t.first[i]) * kAdamChunk;
    const uint32_t n = elements<kAdamChunk>(x.n, at);
    const uint8_t *mc = codes_from(x.m, at), *vc = codes_from(x.v, at);
    uint32_t mq[kFours], vq[kFours];
    float ms[kFours], vs[kFours];
#pragma unroll
    for (int q = 0; q < kFours; ++q) {
      const uint32_t block = min(element(q), n - 1) / kAdamBlock;
      ms[q] = x.ms[at / kAdamBlock + block];
      vs[q] = x.vs[at / kAdamBlock + block];
    }
    if (n == kAdamChunk) {
#pragma unroll
      for (int q = 0; q < kFours; ++q) {
        mq[q] = get_codes(mc, element(q));
        vq[q] = get_codes(vc, element(q));
      }
    } else {
#pragma unroll
      for (int q = 0; q < kFours; ++q) {
        mq[q] = pack(get_last_codes(mc, element(q), n));
        vq[q] = pack(get_last_codes(vc, element(q), n));
      }
    }
#pragma unroll
    for (int q = 0; q < kFours; ++q) {
      const int left = static_cast<int>(n - element(q));
      if (left <= 0) continue;
      const f32x4 m = m_of(mq[q], ms[q]), r = r_of(vq[q], vs[q]), v = r * r;
      if (x.f32) {
        put<true>(from<true>(x.m_out, at), element(q), m, left);
        put<true>(from<true>(x.v_out, at), element(q), v, left);
      } else {
        put<false>(from<false>(x.m_out, at), element(q), m, left);
        put<false>(from<false>(x.v_out, at), element(q), v, left);
      }
    }
  }
}

// Workgroups of a launch: one to a chunk, as far as that goes, for they balance themselves (201M elements, 2048 of them and
// 49152: fp32 states 1126 and 1036 us, 8-bit ones 670 and 572); fewer where each has several ranks' parts to add up.
constexpr int64_t kMostGroups = 65536;
unsigned grid_of(int64_t chunks, int64_t most) { return static_cast<unsigned>(chunks < 1 ? 1 : chunks < most ? chunks : most); }

template <int CHUNK>
void launch(const AdamTable& t, bool codes, const AdamArgs& a, hipStream_t s) {
  const int64_t most = a.parts ? std::max<int64_t>(kMostGroups / a.ranks, 2048) : kMostGroups;
  const dim3 grid(grid_of(std::max<int64_t>(t.first[t.num], whole<CHUNK> ? t.num * (CHUNK / kAdamShort) : 0), most));
  if (codes) hipLaunchKernelGGL((adamw_kernel<true, CHUNK>), grid, dim3(kAdamThreads), 0, s, t, a);
  else hipLaunchKernelGGL((adamw_kernel<false, CHUNK>), grid, dim3(kAdamThreads), 0, s, t, a);
}

}  // namespace

hipError_t adamw_launch(const AdamTensor *ts, int64_t num, bool codes, const AdamArgs& args, hipStream_t s) {
  const int64_t chunk = adam_chunk(ts, num);
  int64_t at = 0;
  AdamArgs a = args;
  do {   // at least once: the norm is written even where there is nothing to step
    AdamTable t;
    next_adam(ts, num, &at, &t, chunk, chunk == kAdamChunk);
    if (chunk == kAdamChunk) launch<kAdamChunk>(t, codes, a, s);
    else launch<kAdamShort>(t, codes, a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.norm_out = nullptr;
  } while (at < num);
  return hipSuccess;
}

hipError_t adamw_values_launch(const AdamValues *ts, int64_t num, hipStream_t s) {
  for (int64_t at = 0; at < num;) {
    AdamValuesTable t;
    next_adam(ts, num, &at, &t, kAdamChunk, false);
    if (!t.num) break;
    hipLaunchKernelGGL(adamw_values_kernel, dim3(grid_of(t.first[t.num], kMostGroups)), dim3(kAdamThreads), 0, s, t);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace tpshard
