// The product for few rows (a decode step): up to 16 tokens, or 64, against a
// weight that is read once, so the weight's bytes bound it.
//
//   kModeOne  c = epi(X W)        kModeDual  c = act(X W) * (X W2)
//
// A workgroup owns 16 G output columns and all rows; its waves split K between
// them and join through LDS.  Given a workspace, several workgroups may split a
// tile's K too: each leaves its sums there, and the last to finish adds them up,
// still in the one launch.  The weight never passes through LDS: each lane's loads are
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
//
// Bound by HBM where the weight is large: on an MI355X (copy 5.2 TB/s) one token
// takes 30 us from 6144 to 12288 (151 MB, 5.0 TB/s) and 55 us through the gated
// block from 12288 to 6144 (302 MB, 5.5 TB/s); by latency where it is small: 768 x
// 768 4 us, gated 4096 -> 2048 (33.5 MB) 10 us (12 at 12 tokens), of which launch,
// first load and join take about 6.  fp32: 6144 -> 12288 (302 MB) 56 us (5.4 TB/s).  16 columns a tile for a k-contiguous weight, 128 bytes of
// columns for an n-contiguous one: with 64 bytes two workgroups on different XCDs
// fetch every line twice (gated 12288 -> 6144 93 us against 59).
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

template <typename T, bool WKC, bool DUAL, int G, int MT>
__global__ void __launch_bounds__(64 * kRowsWaves) lin_rows_kernel(LinGemm p) {
  constexpr int PER = 16 / sizeof(T);          // k of a lane in a step
  constexpr int STEP = 4 * PER;                // k of a step
  constexpr int MATS = DUAL ? 2 : 1;
  constexpr int TC = 16 * G;
  // Steps whose loads are in flight together.
  constexpr int REGS = (WKC ? 4 * G * MATS : PER * MATS * G * static_cast<int>(sizeof(T)) / 4) + 4 * MT;
  constexpr int U = REGS <= 12 ? 8 : REGS <= 24 ? 4 : REGS <= 32 ? 2 : 1;
  // [waves][MATS][M][TC]; four floats at a time go in and out.
  extern __shared__ __attribute__((aligned(16))) float red[];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int l15 = lane & 15, q = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * TC;
  const T *X = static_cast<const T *>(p.a);

  // This wave's steps [s0, s1) of K's (the workgroups of one tile split them
  // first), and whether it ends with K's ragged one.
  const int64_t steps = (p.K + STEP - 1) / STEP;
  const int64_t part = static_cast<int64_t>(blockIdx.y) * waves + wave, parts = static_cast<int64_t>(gridDim.y) * waves;
  const int64_t s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
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
      __builtin_amdgcn_sched_barrier(0);
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
      __builtin_amdgcn_sched_barrier(0);
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
  // Sum of cell i over the waves.
  auto joined = [&](int i) {
    float v = red[i];
    for (int w = 1; w < waves; ++w) v += red[w * MATS * M * TC + i];
    return v;
  };
  const int cells = MATS * M * TC, splits = gridDim.y;
  const float *from = nullptr;                  // the tile's partials, once all are there
  if (splits > 1) {
    float *mine = p.join + (static_cast<int64_t>(blockIdx.x) * splits + blockIdx.y) * cells;
    for (int i = threadIdx.x; i < cells; i += blockDim.x) put_partial(mine + i, joined(i));
    if (!last_of_tile(p.tickets + blockIdx.x, splits)) return;
    from = p.join + static_cast<int64_t>(blockIdx.x) * splits * cells;
  }
  with_act(p.act, [&](auto A) {
    constexpr int ACT = decltype(A)::value;
    // Two cells a lane at a time, so that their partials' loads travel together.
    const int all = M * TC, stride = blockDim.x;
    for (int i0 = threadIdx.x; i0 < all; i0 += 2 * stride) {
      const int cell[2] = {i0, i0 + stride < all ? i0 + stride : i0};
      float v[2 * MATS];
      if (from) {
        sum_partials(from, cells, [&](int k) { return (k % MATS) * all + cell[k / MATS]; }, splits, v);
      } else {
#pragma unroll
        for (int k = 0; k < 2 * MATS; ++k) v[k] = joined((k % MATS) * all + cell[k / MATS]);
      }
      auto put = [&](void *base, int64_t at, float y, bool f32) {
        if (f32) static_cast<float *>(base)[at] = y;
        else static_cast<uint16_t *>(base)[at] = to_bf16(y);
      };
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = cell[h] / TC;
        const int64_t n = n0 + cell[h] % TC;
        if (n >= p.N || (h && cell[1] == i0)) continue;
        float y;
        if constexpr (DUAL) {
          const float gate = v[h * MATS], up = v[h * MATS + 1];
          if (p.aux) put(p.aux, m * p.ldaux + n, gate, sizeof(T) == 4);
          if (p.aux2) put(p.aux2, m * p.ldaux + n, up, sizeof(T) == 4);
          y = act_fwd<ACT>(gate) * up;
        } else {
          const float pre = p.bias ? v[h] + p.bias[n] : v[h];
          if (p.aux) put(p.aux, m * p.ldaux + n, pre, sizeof(T) == 4);
          y = act_fwd<ACT>(pre);
          if (p.res) y += load1(static_cast<const T *>(p.res) + m * p.ldres + n);
        }
        put(p.c, m * p.ldc + n, y, p.c_f32);
      }
    }
  });
}

template <typename T, bool WKC, bool DUAL, int G>
hipError_t by_rows(const LinGemm& p, const RowsShape& h, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(h.tiles), static_cast<unsigned>(h.splits)), block(64 * h.waves);
  const unsigned lds = static_cast<unsigned>(h.waves * h.cells * 4);
  if (p.M <= 16) hipLaunchKernelGGL((lin_rows_kernel<T, WKC, DUAL, G, 1>), grid, block, lds, s, p);
  else if constexpr (!WKC) return hipErrorInvalidValue;
  else if (p.M <= 32) hipLaunchKernelGGL((lin_rows_kernel<T, WKC, DUAL, G, 2>), grid, block, lds, s, p);
  else hipLaunchKernelGGL((lin_rows_kernel<T, WKC, DUAL, G, 4>), grid, block, lds, s, p);
  return hipGetLastError();
}

template <typename T, bool DUAL>
hipError_t by_layout(const LinGemm& p, const RowsShape& h, hipStream_t s) {
  if (p.w_t) return by_rows<T, true, DUAL, 1>(p, h, s);
  return by_rows<T, false, DUAL, 8 / static_cast<int>(sizeof(T))>(p, h, s);
}

}  // namespace

hipError_t lin_rows_launch(const LinGemm& p, const RowsShape& h, hipStream_t s) {
  const bool dual = p.mode == kModeDual;
  if (p.f32) return dual ? by_layout<uint32_t, true>(p, h, s) : by_layout<uint32_t, false>(p, h, s);
  return dual ? by_layout<uint16_t, true>(p, h, s) : by_layout<uint16_t, false>(p, h, s);
}

}  // namespace tpshard
