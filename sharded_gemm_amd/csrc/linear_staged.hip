// The general product of the linear layer and the gated block: any operand
// layout, stride, alignment and size, bf16 and fp32.
//
//   kModeOne  c = epi(A W)              kModeDual  c = act(A W) * (A W2)
//   kModeCat  c = A W + A2 W2           kModePair  c = A W, c2 = A2 W2
//
// A workgroup of 4 or 8 waves owns a BM x BN tile of the output (kModeDual: BM x
// BN/2, with the gate's and the up projection's columns side by side in the W
// tile, so that each lane ends with both of an output's factors).  K is staged
// 128 bytes at a time (64 bf16, 32 fp32) through two LDS slots: the next
// stage's global loads are in registers while this one is multiplied.  Both
// tiles lie k-contiguous in LDS, 128 bytes a row, 16-byte chunk c of row r at
// c ^ ((r ^ r / 8) & 7), which keeps the writes of either source layout and the
// fragment reads on distinct banks; an operand that is row-contiguous in memory
// is transposed in registers on its way.  Elements past the edges read as zero,
// so the tile is zero-padded.
//
// bf16: v_mfma_f32_16x16x32_bf16.  fp32: v_mfma_f32_16x16x4_f32, four per
// 16-byte chunk; a lane group's chunk holds four consecutive k, which the four
// MFMAs take in turn (the order of a sum over k is free, and A and W agree).
//
// Measured on an MI355X: fp32 4096^3 1.03 ms (133 TFLOP/s, the library 150), 515 x
// 1021 x 1531 28 us (58); bf16 4097 x 4095 x 4097 270 us (509), the gated
// backward 1021 x 1337 -> 999 32 + 25 us.  Odd strides cost: a 16-byte load off a
// 4-byte boundary goes through the address unit a lane at a time.
#include "linear_dev.h"

namespace tpshard {

using namespace lin;

namespace {

constexpr int kRow = kStagedRow;          // LDS bytes of a tile row per stage

__device__ __forceinline__ uint32_t lds_at(int r, int c) {
  return static_cast<uint32_t>(r * kRow + ((c ^ ((r ^ (r >> 3)) & 7)) << 4));
}

// One operand's tile: ROWS output rows (or columns) by one stage of K.
// KC: k is contiguous in memory.  T: uint32_t (fp32) or uint16_t (bf16).
//
// Rows past the edge are clamped onto an existing one, and a row-contiguous
// group that reaches past it reads on into the next rows: both only feed
// outputs that are never stored.  So a stage is fetched without a check per
// element wherever it and the V rows after it lie inside K (there, reading V
// elements from any existing one stays within the operand whatever its stride);
// only the last stages of K are checked, and their missing elements are zero.
template <typename T, int ROWS, bool KC, int THREADS>
struct Tile {
  static constexpr int V = 16 / sizeof(T);          // elements of a 16-byte chunk
  static constexpr int KB = ROWS * 8 / THREADS;     // chunks (KC) or k rows (else) per thread
  static constexpr int NBLK = ROWS / V;             // groups of V rows
  static constexpr int BK = kRow / sizeof(T);
  static_assert(KB == 2, "tile rows");
  static_assert(KC || NBLK * (BK / KB) == THREADS, "one block of KB k rows per thread");

  const T *at[KC ? KB : 1];    // sources at k = 0
  int64_t ld;
  int left;                    // elements of the group that exist (row-contiguous)

  // where(r, &base, &index): the matrix and the row of tile row r; n: rows that exist.
  template <typename Where>
  __device__ __forceinline__ void init(int64_t ld_, int64_t n, Where&& where) {
    const int t = threadIdx.x;
    ld = ld_;
    left = V;
    const T *base;
    int64_t row;
    if constexpr (KC) {
#pragma unroll
      for (int q = 0; q < KB; ++q) {
        const int idx = t + THREADS * q;
        where(idx >> 3, &base, &row);
        at[q] = base + (row < n ? row : n - 1) * ld + (idx & 7) * V;
      }
    } else {
      where(t % NBLK * V, &base, &row);
      const int64_t rest = n - row;
      if (rest <= 0) {
        row = n - 1;
        left = 1;      // the clamped element itself: nothing lies behind the last row's
      } else if (rest < V) {
        left = static_cast<int>(rest);
      }
      at[0] = base + row + static_cast<int64_t>(t / NBLK * KB) * ld;
    }
  }

  // Stages that lie inside K as above.
  __device__ __forceinline__ static int64_t inside(int64_t K) { return K >= V ? (K - V) / BK : 0; }

  // The stage from k0 on; `shift`: from the first matrix to the one read (elements).
  __device__ __forceinline__ void load(int64_t k0, int64_t shift, u32x4 (&g)[KB]) const {
#pragma unroll
    for (int q = 0; q < KB; ++q)
      g[q] = *reinterpret_cast<const u32x4_any *>(KC ? at[KC ? q : 0] + shift + k0 : at[0] + shift + (k0 + q) * ld);
  }
  __device__ __forceinline__ void load_checked(int64_t k0, int64_t K, int64_t shift, u32x4 (&g)[KB]) const {
    const int t = threadIdx.x;
#pragma unroll
    for (int q = 0; q < KB; ++q) {
      if constexpr (KC) {
        g[q] = load16<T>(at[q] + shift + k0, K - k0 - ((t + THREADS * q) & 7) * V);
      } else {
        g[q] = load16<T>(at[0] + shift + (k0 + q) * ld, k0 + t / NBLK * KB + q < K ? left : 0);
      }
    }
  }

  __device__ __forceinline__ static void store(char *lds, const u32x4 (&g)[KB]) {
    const int t = threadIdx.x;
    if constexpr (KC) {
#pragma unroll
      for (int q = 0; q < KB; ++q) {
        const int idx = t + THREADS * q;
        *reinterpret_cast<u32x4 *>(lds + lds_at(idx >> 3, idx & 7)) = g[q];
      }
    } else {
      const int b = t % NBLK, kb = t / NBLK;
      const int byte = kb * KB * static_cast<int>(sizeof(T));
#pragma unroll
      for (int j = 0; j < V; ++j) {
        char *dst = lds + lds_at(b * V + j, byte >> 4) + (byte & 15);
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<u32x2 *>(dst) = u32x2{g[0][j], g[1][j]};
        } else {
          *reinterpret_cast<uint32_t *>(dst) =
              __builtin_amdgcn_perm(g[1][j >> 1], g[0][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
        }
      }
    }
  }
};

// 4 waves on 64 x 64, 8 on 128 x 128: two 16-byte chunks of each operand's stage a
// thread on both.  The 8 waves stay within 128 registers, so that two such
// workgroups share a CU (4 waves with 230 registers, both still storing element
// by element: 8191 x 333 x 2333 bf16 74 us against 61, 2049 x 2047 x 2049 63 against 58).
constexpr int threads_of(int edge) { return edge == 128 ? 512 : 256; }
constexpr int waves_simd(int edge) { return edge == 128 ? 4 : 2; }

template <typename T, int BM, int BN, bool AKC, bool WKC, int MODE>
__global__ void __launch_bounds__(threads_of(BM), waves_simd(BM)) lin_staged_kernel(LinGemm p) {
  constexpr int THREADS = threads_of(BM);
  using TA = Tile<T, BM, AKC, THREADS>;
  using TW = Tile<T, BN, WKC, THREADS>;
  constexpr int BK = TA::BK;
  constexpr int WAVES_N = THREADS / 128;                 // by two rows of waves
  constexpr int WM = BM / 2, WN = BN / WAVES_N, TM = WM / 16, TN = WN / 16;
  constexpr int BNO = MODE == kModeDual ? BN / 2 : BN;   // output columns of a tile
  constexpr int LDS_A = BM * kRow, STAGE = (BM + BN) * kRow;
  __shared__ __attribute__((aligned(16))) char smem[2 * STAGE];

  const int64_t tiles_m = (p.M + BM - 1) / BM, tiles_n = (p.N + BNO - 1) / BNO;
  int64_t tile = blockIdx.x;
  const bool second = MODE == kModePair && tile >= tiles_m * tiles_n;
  if (second) tile -= tiles_m * tiles_n;
  // Neighbouring workgroups share a W panel (tiles walk down the rows first).
  const int64_t m0 = tile % tiles_m * BM, n0 = tile / tiles_m * BNO;
  const T *A = static_cast<const T *>(second ? p.a2 : p.a), *W = static_cast<const T *>(second ? p.w2 : p.w);
  const T *W2 = static_cast<const T *>(p.w2);
  void *c = second ? p.c2 : p.c;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / WAVES_N, wn = wave % WAVES_N;

  TA ta;
  TW tw;
  ta.init(p.lda, p.M, [&](int r, const T **base, int64_t *row) {
    *base = A;
    *row = m0 + r;
  });
  tw.init(p.ldw, p.N, [&](int r, const T **base, int64_t *row) {
    // kModeDual: each wave's first half of the tile are the gate's columns, its
    // second half the up projection's.
    const bool up = MODE == kModeDual && r % WN >= WN / 2;
    *base = up ? W2 : W;
    *row = n0 + (MODE == kModeDual ? r / WN * (WN / 2) + r % (WN / 2) : r);
  });

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Regs {
    u32x4 a[TA::KB], w[TW::KB];
  };
  auto put = [&](int64_t st, const Regs& g) {
    char *slot = smem + (st & 1) * STAGE;
    TA::store(slot, g.a);
    TW::store(slot + LDS_A, g.w);
  };
  // All of a stage's fragments are read before its products where they fit
  // the registers (64 x 64).
  constexpr int AHEAD = BM == 64 ? 2 : 1;
  auto compute = [&](const char *stage) {
    const char *As = stage, *Ws = stage + LDS_A;
#pragma unroll
    for (int k0 = 0; k0 < 2; k0 += AHEAD) {
      u32x4 fa[AHEAD][TM], fw[AHEAD][TN];
#pragma unroll
      for (int kk = 0; kk < AHEAD; ++kk) {
        const int ch = (k0 + kk) * 4 + (lane >> 4);
#pragma unroll
        for (int i = 0; i < TM; ++i)
          fa[kk][i] = *reinterpret_cast<const u32x4 *>(As + lds_at(wm * WM + i * 16 + (lane & 15), ch));
#pragma unroll
        for (int j = 0; j < TN; ++j)
          fw[kk][j] = *reinterpret_cast<const u32x4 *>(Ws + lds_at(wn * WN + j * 16 + (lane & 15), ch));
      }
      if constexpr (AHEAD == 2) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int kk = 0; kk < AHEAD; ++kk) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fw[kk][j]),
                                                                  __builtin_bit_cast(bf16x8, fa[kk][i]), acc[i][j], 0, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
              for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(fw[kk][j][e]), __uint_as_float(fa[kk][i][e]),
                                                                 acc[i][j], 0, 0, 0);
        }
      }
    }
  };

  // Stages [first, last) of one pair of matrices.  64 x 64: stage st + 2 leaves
  // for the registers that stage st has left, stage st + 1 moves from its own to
  // LDS after stage st's products, so a load has two stages' time to arrive
  // (four gained nothing).  128 x 128: one stage ahead (two spill).
  // The unchecked stages have a loop of their own: where both kinds of fetch
  // meet, the compiler waits for the newest load too.
  auto run = [&](int64_t first, int64_t last, int64_t a_shift, int64_t w_shift) {
    const int64_t nst = last - first;
    if (nst <= 0) return;
    Regs g0, g1;
    auto fetch = [&](int64_t st, Regs& g) {
      ta.load((first + st) * BK, a_shift, g.a);
      tw.load((first + st) * BK, w_shift, g.w);
    };
    auto fetch_checked = [&](int64_t st, Regs& g) {
      ta.load_checked((first + st) * BK, p.K, a_shift, g.a);
      tw.load_checked((first + st) * BK, p.K, w_shift, g.w);
    };
    const int64_t free = min(TA::inside(p.K), last) - first;   // leading stages without checks
    if constexpr (BM == 128) {
      if (free > 0) fetch(0, g0); else fetch_checked(0, g0);
      put(0, g0);
      __syncthreads();
      int64_t st = 0;
      for (; st + 1 < free; ++st) {
        fetch(st + 1, g0);
        compute(smem + (st & 1) * STAGE);
        put(st + 1, g0);
        __syncthreads();
      }
      for (; st < nst; ++st) {
        if (st + 1 < nst) fetch_checked(st + 1, g0);
        compute(smem + (st & 1) * STAGE);
        if (st + 1 < nst) put(st + 1, g0);
        __syncthreads();
      }
      return;
    }
    auto step = [&](int64_t st, Regs& mine, const Regs& next) {
      if (st + 2 < nst) fetch_checked(st + 2, mine);
      compute(smem + (st & 1) * STAGE);
      if (st + 1 < nst) put(st + 1, next);
      __syncthreads();
    };
    int64_t st = 0;
    if (free >= 2) {
      fetch(0, g0);
      fetch(1, g1);
      put(0, g0);
      __syncthreads();
      for (; st + 3 < free; st += 2) {
        fetch(st + 2, g0);
        compute(smem);
        put(1, g1);
        __syncthreads();
        fetch(st + 3, g1);
        compute(smem + STAGE);
        put(0, g0);
        __syncthreads();
      }
    } else {
      fetch_checked(0, g0);
      if (nst > 1) fetch_checked(1, g1);
      put(0, g0);
      __syncthreads();
    }
    for (; st < nst; st += 2) {
      step(st, g0, g1);
      if (st + 1 < nst) step(st + 1, g1, g0);
    }
  };
  // This workgroup's share of the stages, over both pairs of matrices in kModeCat.
  const int64_t per = (p.K + BK - 1) / BK, all = MODE == kModeCat ? 2 * per : per;
  const int64_t st0 = all * blockIdx.y / gridDim.y, st1 = all * (blockIdx.y + 1) / gridDim.y;
  run(st0, min(st1, per), 0, 0);
  if constexpr (MODE == kModeCat)
    run(max(st0 - per, int64_t{0}), st1 - per, static_cast<const T *>(p.a2) - A, W2 - W);
  if (gridDim.y > 1 && !join_splits<THREADS>(p, acc)) return;

  auto rm = [&](int i) -> int64_t { return m0 + wm * WM + i * 16 + (lane & 15); };
  auto cn = [&](int j) -> int64_t {
    const int wcols = MODE == kModeDual ? WN / 2 : WN;
    return n0 + wn * wcols + j * 16 + 4 * (lane >> 4);
  };
  if constexpr (sizeof(T) == 4) epilogue<float, MODE>(p, c, acc, rm, cn);
  else epilogue<uint16_t, MODE>(p, c, acc, rm, cn);
}

template <typename T, bool AKC, bool WKC, int MODE>
hipError_t launch(const LinGemm& p, const StagedShape& h, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(h.tiles), static_cast<unsigned>(h.splits));
  if (h.edge == 128) hipLaunchKernelGGL((lin_staged_kernel<T, 128, 128, AKC, WKC, MODE>), grid, dim3(threads_of(128)), 0, s, p);
  else hipLaunchKernelGGL((lin_staged_kernel<T, 64, 64, AKC, WKC, MODE>), grid, dim3(threads_of(64)), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t dispatch(const LinGemm& p, const StagedShape& h, hipStream_t s) {
  const bool akc = !p.a_t, wkc = p.w_t != 0;
  switch (p.mode) {
    case kModeOne:
      if (akc) return wkc ? launch<T, true, true, kModeOne>(p, h, s) : launch<T, true, false, kModeOne>(p, h, s);
      break;
    case kModeDual:
      if (akc) return wkc ? launch<T, true, true, kModeDual>(p, h, s) : launch<T, true, false, kModeDual>(p, h, s);
      break;
    case kModeCat:
      if (akc) return wkc ? launch<T, true, true, kModeCat>(p, h, s) : launch<T, true, false, kModeCat>(p, h, s);
      break;
    case kModePair:
      if (!akc && !wkc) return launch<T, false, false, kModePair>(p, h, s);
      break;
  }
  if (p.mode == kModeOne && !akc && !wkc) return launch<T, false, false, kModeOne>(p, h, s);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t lin_staged_launch(const LinGemm& p, const StagedShape& h, hipStream_t s) {
  return p.f32 ? dispatch<uint32_t>(p, h, s) : dispatch<uint16_t>(p, h, s);
}

}  // namespace tpshard
