// The product for few rows (a decode step): M <= 64 tokens against a weight
// that is read once, so the weight's bytes bound it.
//
//   kModeOne  c = epi(X W)        kModeDual  c = act(X W) * (X W2)
//
// A workgroup owns 16 G output columns and all rows; its waves split K between
// them and join through LDS, so one launch does everything, with no partial
// sums in memory.  The weight never passes through LDS: each lane's loads are
// already an MFMA operand (v_mfma_f32_16x16x32_bf16 takes the weight first, so
// its 16 rows are output columns and its columns are tokens).
//  * k-contiguous weight ([N][K]): lane l loads 16 bytes (8 k) of column
//    l & 15 at k group l >> 4; G operands of 16 columns each.
//  * n-contiguous weight ([K][N]): lane l loads G columns, G (l & 15) on, of
//    eight k rows (8 (l >> 4) on); byte permutes pair the rows, which leaves the
//    8 k of each of the lane's G columns in a register quad: operand j holds
//    column G r + j in its row r.  No LDS transpose, half an instruction per
//    element.
// fp32 does the same with v_mfma_f32_16x16x4_f32, 4 k a lane.
// Rows past M repeat row M - 1, columns past N the last one (their results are
// dropped); k past the end reads as zero on both sides.
#include "linear_dev.h"

namespace tpshard {

using namespace lin;

namespace {

// 4 bf16 pairs or 4 floats: what one lane feeds to the MFMAs of a step.
template <typename T>
__device__ __forceinline__ f32x4 mma(u32x4 w, u32x4 x, f32x4 acc) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[e]), __uint_as_float(x[e]), acc, 0, 0, 0);
    return acc;
  }
}

// 16 bytes at p, of which `left` elements exist.
template <typename T>
__device__ __forceinline__ u32x4 load16(const T *p, int64_t left) {
  constexpr int V = 16 / sizeof(T);
  if (left >= V) return *reinterpret_cast<const u32x4_any *>(p);
  u32x4 v{0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e < left) {
      if constexpr (sizeof(T) == 4) v[e] = p[e];
      else v[e >> 1] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
    }
  return v;
}

// G elements of T at p as dwords, of which `left` exist.
template <typename T, int G>
struct Cols {
  static constexpr int D = G * sizeof(T) / 4;
  uint32_t d[D];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (D == 8) {
      const u32x4 a = *reinterpret_cast<const u32x4_any *>(p), b = *reinterpret_cast<const u32x4_any *>(p + G / 2);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        d[e] = a[e];
        d[4 + e] = b[e];
      }
    } else if constexpr (D == 4) {
      const u32x4 a = *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = a[e];
    } else if constexpr (D == 2) {
      const u32x2 a = *reinterpret_cast<const u32x2_any *>(p);
      d[0] = a[0];
      d[1] = a[1];
    } else {
      d[0] = *reinterpret_cast<const u32_any *>(p);
    }
  }
  __device__ __forceinline__ void load(const T *p, int64_t left) {
#pragma unroll
    for (int i = 0; i < D; ++i) d[i] = 0;
#pragma unroll
    for (int e = 0; e < G; ++e)
      if (e < left) {
        if constexpr (sizeof(T) == 4) d[e] = p[e];
        else d[e >> 1] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
      }
  }
};

// Most waves of a workgroup: past 16 rows the accumulators need more than the
// 128 registers that 16 waves leave each.
template <int MT>
constexpr int kWaves = MT == 1 ? 16 : 8;

template <typename T, bool WKC, bool DUAL, int G, int MT>
__global__ void __launch_bounds__(64 * kWaves<MT>) lin_rows_kernel(LinGemm p) {
  constexpr int PER = 16 / sizeof(T);          // k of a lane in a step
  constexpr int STEP = 4 * PER;                // k of a step
  constexpr int MATS = DUAL ? 2 : 1;
  constexpr int TC = 16 * G;
  // Steps whose loads are in flight together.
  constexpr int U = WKC ? (G * MATS * 4 + MT * 4 <= 12 ? 8 : G * MATS * 4 + MT * 4 <= 24 ? 4 : 2) : (G * MATS <= 4 ? 2 : 1);
  extern __shared__ float red[];               // [waves][MATS][M][TC]

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int l15 = lane & 15, q = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * TC;
  const T *X = static_cast<const T *>(p.a);

  // This wave's steps [s0, s1) of K's, and whether it ends with K's ragged one.
  const int64_t steps = (p.K + STEP - 1) / STEP;
  const int64_t s0 = steps * wave / waves, s1 = steps * (wave + 1) / waves;
  const int64_t s1_full = (s1 == steps && p.K % STEP) ? s1 - 1 : s1;

  const T *xp[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t m = 16 * t + l15;
    xp[t] = X + (m < p.M ? m : p.M - 1) * p.lda + PER * q;
  }
  const T *wp[MATS][WKC ? G : 1];
  int64_t left = 0;                             // columns of this lane that exist (n-contiguous)
#pragma unroll
  for (int a = 0; a < MATS; ++a) {
    const T *W = static_cast<const T *>(a ? p.w2 : p.w);
    if constexpr (WKC) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int64_t n = n0 + 16 * g + l15;
        wp[a][g] = W + (n < p.N ? n : p.N - 1) * p.ldw + PER * q;
      }
    } else {
      const int64_t n = n0 + G * l15;
      left = p.N - n;
      wp[a][0] = W + (left > 0 ? n : p.N - 1) + static_cast<int64_t>(PER) * q * p.ldw;
    }
  }
  const bool whole = n0 + TC <= p.N;

  f32x4 acc[MATS][G][MT];
#pragma unroll
  for (int a = 0; a < MATS; ++a)
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[a][g][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  if constexpr (WKC) {
    auto run = [&](int64_t s, auto n_steps, bool ragged) {
      constexpr int N = decltype(n_steps)::value;
      u32x4 w[N][MATS][G], x[N][MT];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t k = (s + i) * STEP, rest = ragged ? p.K - k - PER * q : PER;
#pragma unroll
        for (int a = 0; a < MATS; ++a)
#pragma unroll
          for (int g = 0; g < G; ++g) w[i][a][g] = load16<T>(wp[a][g] + k, rest);
#pragma unroll
        for (int t = 0; t < MT; ++t) x[i][t] = load16<T>(xp[t] + k, rest);
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int a = 0; a < MATS; ++a)
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[a][g][t] = mma<T>(w[i][a][g], x[i][t], acc[a][g][t]);
    };
    int64_t s = s0;
    for (; s + U <= s1_full; s += U) run(s, Const<U>{}, false);
    for (; s < s1_full; ++s) run(s, Const<1>{}, false);
    if (s < s1) run(s, Const<1>{}, true);
  } else {
    auto run = [&](int64_t s, auto n_steps, bool checked) {
      constexpr int N = decltype(n_steps)::value;
      Cols<T, G> w[N][MATS][PER];
      u32x4 x[N][MT];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t k = (s + i) * STEP, rest = p.K - k - PER * q;
#pragma unroll
        for (int a = 0; a < MATS; ++a)
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            const T *src = wp[a][0] + (k + e) * p.ldw;
            if (checked) w[i][a][e].load(src, e < rest ? left : 0);
            else w[i][a][e].load(src);
          }
#pragma unroll
        for (int t = 0; t < MT; ++t) x[i][t] = load16<T>(xp[t] + k, checked ? rest : PER);
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int a = 0; a < MATS; ++a)
#pragma unroll
          for (int g = 0; g < G; ++g) {
            u32x4 op;
            if constexpr (sizeof(T) == 2) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                op[e] = __builtin_amdgcn_perm(w[i][a][2 * e + 1].d[g >> 1], w[i][a][2 * e].d[g >> 1],
                                              (g & 1) ? 0x07060302u : 0x05040100u);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) op[e] = w[i][a][e].d[g];
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[a][g][t] = mma<T>(op, x[i][t], acc[a][g][t]);
          }
    };
    int64_t s = s0;
    if (whole) {
      for (; s + U <= s1_full; s += U) run(s, Const<U>{}, false);
      for (; s < s1_full; ++s) run(s, Const<1>{}, false);
    }
    for (; s < s1; ++s) run(s, Const<1>{}, true);
  }

  // Join the waves.  Lane l holds, of token 16 t + (l & 15), the operand rows
  // 4 (l >> 4) .. + 3.
  const int M = static_cast<int>(p.M);
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = 16 * t + l15;
    if (m < M) {
#pragma unroll
      for (int a = 0; a < MATS; ++a) {
        float *dst = red + (static_cast<int64_t>(wave * MATS + a) * M + m) * TC;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          if constexpr (WKC) {
            *reinterpret_cast<f32x4 *>(dst + 16 * g + 4 * q) = acc[a][g][t];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[(4 * q + e) * G + g] = acc[a][g][t][e];
          }
        }
      }
    }
  }
  __syncthreads();
  with_act(p.act, [&](auto A) {
    constexpr int ACT = decltype(A)::value;
    for (int i = threadIdx.x; i < M * TC; i += blockDim.x) {
      const int m = i / TC;
      const int64_t n = n0 + i % TC;
      if (n >= p.N) continue;
      float v[MATS];
#pragma unroll
      for (int a = 0; a < MATS; ++a) {
        v[a] = red[a * M * TC + i];
        for (int w = 1; w < waves; ++w) v[a] += red[(w * MATS + a) * M * TC + i];
      }
      auto put = [&](void *base, int64_t at, float y, bool f32) {
        if (f32) static_cast<float *>(base)[at] = y;
        else static_cast<uint16_t *>(base)[at] = to_bf16(y);
      };
      float y;
      if constexpr (DUAL) {
        if (p.aux) put(p.aux, m * p.ldaux + n, v[0], sizeof(T) == 4);
        if (p.aux2) put(p.aux2, m * p.ldaux + n, v[1], sizeof(T) == 4);
        y = act_fwd<ACT>(v[0]) * v[1];
      } else {
        const float pre = p.bias ? v[0] + p.bias[n] : v[0];
        if (p.aux) put(p.aux, m * p.ldaux + n, pre, sizeof(T) == 4);
        y = act_fwd<ACT>(pre);
        if (p.res) y += load1(static_cast<const T *>(p.res) + m * p.ldres + n);
      }
      put(p.c, m * p.ldc + n, y, p.c_f32);
    }
  });
}

// Waves of a workgroup: enough that each still has `least` steps, and that the
// join fits 64 KiB of LDS.
template <typename T, bool WKC, bool DUAL, int G, int MT>
hipError_t launch(const LinGemm& p, hipStream_t s) {
  constexpr int STEP = 64 / sizeof(T), TC = 16 * G, MATS = DUAL ? 2 : 1;
  const int64_t steps = (p.K + STEP - 1) / STEP, per_wave = MATS * p.M * TC * 4;
  int waves = kWaves<MT>;
  while (waves > 1 && (waves * 2 > steps || waves * per_wave > 64 * 1024)) waves /= 2;
  hipLaunchKernelGGL((lin_rows_kernel<T, WKC, DUAL, G, MT>), dim3(static_cast<unsigned>((p.N + TC - 1) / TC)),
                     dim3(64 * waves), static_cast<unsigned>(waves * per_wave), s, p);
  return hipGetLastError();
}

template <typename T, bool WKC, bool DUAL, int G>
hipError_t by_rows(const LinGemm& p, hipStream_t s) {
  if (p.M <= 16) return launch<T, WKC, DUAL, G, 1>(p, s);
  if (p.M <= 32) return launch<T, WKC, DUAL, G, 2>(p, s);
  return launch<T, WKC, DUAL, G, 4>(p, s);
}

template <typename T, bool DUAL>
hipError_t by_layout(const LinGemm& p, hipStream_t s) {
  if (p.w_t) return by_rows<T, true, DUAL, 1>(p, s);
  return p.N >= 8192 ? by_rows<T, false, DUAL, 4>(p, s) : by_rows<T, false, DUAL, 2>(p, s);
}

}  // namespace

bool lin_rows_ok(const LinGemm& p) {
  return p.M <= 64 && !p.a_t && p.K > 0 && (p.mode == kModeOne || p.mode == kModeDual) && !p.acc_c;
}

hipError_t lin_rows_launch(const LinGemm& p, hipStream_t s) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  const bool dual = p.mode == kModeDual;
  if (p.f32) return dual ? by_layout<uint32_t, true>(p, s) : by_layout<uint32_t, false>(p, s);
  return dual ? by_layout<uint16_t, true>(p, s) : by_layout<uint16_t, false>(p, s);
}

}  // namespace tpshard
