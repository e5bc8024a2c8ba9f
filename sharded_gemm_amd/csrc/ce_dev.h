// Device code of the vocabulary cross entropy: row statistics of logits, how they
// combine, and the epilogues of the products whose output are logits.
//
// A set of logits of one row is held as {top, s}: its maximum, and s = sum of e^(z - top), so
//   ln sum e^z = top + ln s.
// A tile's terms are 2^(z log2 e - r), one fma and exp2 each, r = top log2 e as rounded to
// fp32: what rounding r changed is common to all of them, and one factor a row takes it out again.  From
// |top| = 2^30 on (kFar) that factor would pass 2^64; there logits that differ do so by 64
// and more, so the terms are 2^(z - top): one for each logit that equals the maximum, and nothing for
// the others.  Where the maximum is infinite the exponents are taken against 0: an infinite
// logit makes s infinite, a NaN makes it NaN, and minus infinity everywhere leaves 0.
#pragma once

#include "ce.h"
#include "linear_dev.h"

namespace tpshard {
namespace ce {

using lin::f32x2;
using lin::f32x4;
using lin::kLog2e;

constexpr float kLn2 = 0.693147180559945309417f;

__device__ __forceinline__ float minus_inf() { return -__builtin_inff(); }
constexpr float kFar = 0x1p30f;
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// How terms are taken against `top`: 2^(z by - to), times 2^rest in all.
struct Against {
  float by, to, rest;
  __device__ __forceinline__ explicit Against(float top) {
    const float t = __builtin_isinf(top) ? 0.0f : top;
    by = fabsf(t) < kFar ? kLog2e : 1.0f;
    to = t * by;
    rest = fmaf(-t, by, to);
  }
};

// (Equal maxima may be infinite ones; a set with nothing in it has minus infinity and 0.)
__device__ __forceinline__ f32x2 join(f32x2 a, f32x2 b) {
  const float top = fmaxf(a[0], b[0]), low = fminf(a[0], b[0]), away = top == low ? 0.0f : low - top;
  const bool first = a[0] == top;
  return f32x2{top, fmaf(first ? b[1] : a[1], exp2_(away * kLog2e), first ? a[1] : b[1])};
}

// ln sum e^z of the set.
__device__ __forceinline__ float lse_of(f32x2 a) {
  return fmaf(kLn2, __builtin_amdgcn_logf(a[1]), __builtin_isinf(a[0]) ? 0.0f : a[0]);
}

// The column of target t among the n that begin with id `begin`, or -1 (the subtraction may wrap).
__device__ __forceinline__ int column_of(int64_t t, int64_t begin, int64_t n) {
  const uint64_t c = static_cast<uint64_t>(t) - static_cast<uint64_t>(begin);
  return c < static_cast<uint64_t>(n) ? static_cast<int>(c) : -1;
}

// A row's outputs from the set of all its logits and its target's (where the piece holds it).
__device__ __forceinline__ void finish(const CeJoin& p, int64_t m, f32x2 a, float logit) {
  const int64_t id = p.targets[m];
  if (column_of(id, p.begin, p.V) < 0) logit = minus_inf();
  if (p.stats) {
    p.stats[m] = a[0];
    p.stats[p.M + m] = a[1];
    p.stats[2 * p.M + m] = logit;
  }
  const float lse = lse_of(a);
  if (p.lse) p.lse[m] = lse;
  if (p.loss) p.loss[m] = id == p.ignore ? 0.0f : lse - logit;
}

// The same lane's value in the other lane groups of 16 that share a row: f over x of lanes l, l ^ 16, l ^ 32, l ^ 48
// (the swaps are vector instructions; a shuffle goes through LDS).
template <typename F>
__device__ __forceinline__ float over_groups(float x, F&& f) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
  a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return f(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// kModeStats: the statistics of a tile's rows.  Four lanes and WAVES_N waves share a
// row: they join through `lds` (WAVES_N * BM pairs, the operand tiles' memory), so
// that a tile leaves one pair a row.
//
// A lane's share is max, fma, exp2 and add for each of its elements; the columns' bounds
// are only checked in tiles that reach past the last one.  Nothing else of a tile's
// time overlaps this one's, so latency counts: all targets are loaded at once, all rows
// go through each step together, and lanes join without LDS (4096 x 768 x 50000, W
// [V, K]: 304 us; a row after the other, joined by shuffles, 328; with the bounds checked
// everywhere 352.  The products alone take 260).
template <int BM, int WAVES_N, int THREADS, int TM, int TN, typename RM, typename CN>
__device__ __forceinline__ void stats(const CeGemm& p, char *lds, const f32x4 (&acc)[TM][TN], int64_t m0, int64_t slot,
                                      int wn, bool whole, RM&& rm, CN&& cn) {
  f32x2 *rows = reinterpret_cast<f32x2 *>(lds);
  const int lane = threadIdx.x & 63, N = static_cast<int>(p.cols);
  int64_t id[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) id[i] = p.targets[rm(i) < p.M ? rm(i) : p.M - 1];
  __syncthreads();   // the operand tiles have been read
  auto all = [&](auto checked) {
    constexpr bool CHECK = decltype(checked)::value != 0;
    float top[TM], s[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      top[i] = minus_inf();
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!CHECK || static_cast<int>(cn(j)) + e < N) top[i] = fmaxf(top[i], acc[i][j][e]);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) top[i] = over_groups(top[i], [](float x, float y) { return fmaxf(x, y); });
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const Against t(top[i]);
      s[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!CHECK || static_cast<int>(cn(j)) + e < N) s[i] += exp2_(fmaf(acc[i][j][e], t.by, -t.to));
      s[i] *= exp2_(t.rest);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      s[i] = over_groups(s[i], [](float x, float y) { return x + y; });
      if (lane < 16) rows[wn * BM + (rm(i) - m0)] = f32x2{top[i], s[i]};
    }
  };
  if (whole) all(lin::Const<0>{});
  else all(lin::Const<1>{});
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int t = rm(i) < p.M ? column_of(id[i], p.begin, p.cols) : -1;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int at = t - static_cast<int>(cn(j));
      if (static_cast<unsigned>(at) < 4u) {   // (t is a column or -1)
        const float z01 = at == 0 ? acc[i][j][0] : acc[i][j][1], z23 = at == 2 ? acc[i][j][2] : acc[i][j][3];
        p.logit[rm(i)] = at < 2 ? z01 : z23;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < BM; i += THREADS) {
    if (m0 + i >= p.M) continue;
    f32x2 a = rows[i];
#pragma unroll
    for (int w = 1; w < WAVES_N; ++w) a = join(a, rows[w * BM + i]);
    *reinterpret_cast<f32x2 *>(p.part + 2 * (slot * p.M + m0 + i)) = a;
  }
}

// kModeProb: the gradient at the logits, rounded to the operands' type T for the two
// products that read it.  In bf16 it is divided by the largest |g| first, which the
// products multiply back in fp32: most of a row's gradient is its target's entry, -g (1 -
// p), and where all g are alike (a mean) every one of them would be rounded the same
// way, up to 0.4 % of the result; divided, they round to -1 where targets are unlikely.
// Of likely ones what is off is independent from entry to entry: 2^-8 / sqrt(3) of the result's norm at
// most (0.0013 measured in an fp32 dX at a mean p of 0.25, 0.0015 at 0.6).
template <typename T, int TM, int TN, typename RM, typename CN>
__device__ __forceinline__ void prob(const CeGemm& p, const f32x4 (&acc)[TM][TN], RM&& rm, CN&& cn) {
  // Every row's loads before any store, which the compiler may not move them across.
  int64_t id[TM];
  float lses[TM], gs[TM], ghs[TM];
  const float scale = p.scale ? *p.scale : 1.0f;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t m = rm(i) < p.M ? rm(i) : p.M - 1;
    id[i] = p.targets[m];
    lses[i] = p.lse[m];
    const float g = p.g ? p.g[m * p.g_step] : 1.0f;
    gs[i] = g / scale;
    ghs[i] = (p.h ? g + p.h[m * p.h_step] : g) / scale;
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t m = rm(i);
    if (m >= p.pad_rows) continue;
    const float lse = lses[i], g = gs[i];
    const bool on = m < p.M && id[i] != p.ignore;
    const int t = column_of(id[i], p.begin, p.cols);
    // (z - lse) log2 e: in bf16 as one fma, as above (an infinite lse stays where it is); in fp32 the difference first, which is
    // exact where z and lse are close.
    const Against by(lse);
    const float to = __builtin_isinf(lse) ? lse : by.to, gh = sizeof(T) == 4 ? ghs[i] : ghs[i] * exp2_(by.rest);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int64_t n = cn(j), left = p.N - n;
      if (left <= 0) continue;
      f32x4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float z = acc[i][j][e];
        y[e] = gh * (sizeof(T) == 4 ? exp2_((z - lse) * kLog2e) : exp2_(fmaf(z, by.by, -to)));
      }
      const int at = t - static_cast<int>(n);
      if (static_cast<unsigned>(at) < 4u) {   // (t is a column or -1)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at == e) y[e] -= g;
      }
      const int64_t there = on ? p.cols - n : 0;
      if (there < 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e >= there) y[e] = 0.0f;
      }
      lin::store4<T>(p.c, m * p.ldc + n, y, left);
    }
  }
}

// kModeScaled.
template <int TM, int TN, typename RM, typename CN>
__device__ __forceinline__ void scaled(const ScaledGemm& p, const f32x4 (&acc)[TM][TN], RM&& rm, CN&& cn) {
  const float alpha = *p.alpha;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int64_t m = rm(i), n = cn(j), left = p.N - n;
      if (m < p.M && left > 0) lin::store4_c(p, p.c, m * p.ldc + n, acc[i][j] * alpha, left);
    }
}

}  // namespace ce
}  // namespace tpshard
