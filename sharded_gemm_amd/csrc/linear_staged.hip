// The general product of the linear layer and the gated block: any operand
// layout, stride, alignment and size, bf16 and fp32.
//
//   kModeOne  c = epi(A W)              kModeDual  c = act(A W) * (A W2)
//   kModeCat  c = A W + A2 W2           kModePair  c = A W, c2 = A2 W2
//
// A workgroup of 4 waves owns a BM x BN tile of the output (kModeDual: BM x
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
#include "linear_dev.h"

namespace tpshard {

using namespace lin;

namespace {

constexpr int kThreads = 256;
constexpr int kRow = 128;                 // LDS bytes of a tile row per stage

__device__ __forceinline__ uint32_t lds_at(int r, int c) {
  return static_cast<uint32_t>(r * kRow + ((c ^ ((r ^ (r >> 3)) & 7)) << 4));
}

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

// One operand's tile: ROWS output rows (or columns) by one stage of K.
// KC: k is contiguous in memory.  T: uint32_t (fp32) or uint16_t (bf16).
template <typename T, int ROWS, bool KC>
struct Tile {
  static constexpr int V = 16 / sizeof(T);          // elements of a 16-byte chunk
  static constexpr int KB = ROWS / 32;              // chunks (KC) or k rows (else) per thread
  static constexpr int NBLK = ROWS / V;             // groups of V rows
  static constexpr int BK = kRow / sizeof(T);
  static_assert(KB == 2 || KB == 4, "tile rows");
  static_assert(KC || NBLK * (BK / KB) == kThreads, "one block of KB k rows per thread");

  // at(r): element offset of tile row r at k = 0 (KC; < 0: no such row), or
  // group(b, &left): offset of the V rows of group b and how many exist.
  template <typename At>
  __device__ __forceinline__ static void load(const T *base, int64_t ld, int64_t k0, int64_t K, At&& at,
                                              u32x4 (&g)[KB]) {
    const int t = threadIdx.x;
    if constexpr (KC) {
#pragma unroll
      for (int q = 0; q < KB; ++q) {
        const int idx = t + kThreads * q, r = idx >> 3, c = idx & 7;
        const int64_t k = k0 + c * V;
        int64_t left = K - k, row;
        if (!at(r, &row)) left = 0;
        g[q] = load16<T>(base + row * ld + k, left);
      }
    } else {
      const int b = t % NBLK, kb = t / NBLK;
      int64_t col, left = at(b * V, &col);
#pragma unroll
      for (int q = 0; q < KB; ++q) {
        const int64_t k = k0 + kb * KB + q;
        g[q] = load16<T>(base + k * ld + col, k < K ? left : 0);
      }
    }
  }

  __device__ __forceinline__ static void store(char *lds, const u32x4 (&g)[KB]) {
    const int t = threadIdx.x;
    if constexpr (KC) {
#pragma unroll
      for (int q = 0; q < KB; ++q) {
        const int idx = t + kThreads * q;
        *reinterpret_cast<u32x4 *>(lds + lds_at(idx >> 3, idx & 7)) = g[q];
      }
    } else {
      const int b = t % NBLK, kb = t / NBLK;
      const int byte = kb * KB * static_cast<int>(sizeof(T));
#pragma unroll
      for (int j = 0; j < V; ++j) {
        char *dst = lds + lds_at(b * V + j, byte >> 4) + (byte & 15);
        if constexpr (sizeof(T) == 4) {
          if constexpr (KB == 4) *reinterpret_cast<u32x4 *>(dst) = u32x4{g[0][j], g[1][j], g[2][j], g[3][j]};
          else *reinterpret_cast<u32x2 *>(dst) = u32x2{g[0][j], g[1][j]};
        } else {
          uint32_t d[KB / 2];
#pragma unroll
          for (int e = 0; e < KB / 2; ++e) {
            const uint32_t lo = g[2 * e][j >> 1], hi = g[2 * e + 1][j >> 1];
            d[e] = (j & 1) ? ((lo >> 16) | (hi & 0xffff0000u)) : ((lo & 0xffffu) | (hi << 16));
          }
          if constexpr (KB == 4) *reinterpret_cast<u32x2 *>(dst) = u32x2{d[0], d[1]};
          else *reinterpret_cast<uint32_t *>(dst) = d[0];
        }
      }
    }
  }
};

template <typename T, int BM, int BN, bool AKC, bool WKC, int MODE>
__global__ void __launch_bounds__(kThreads) lin_staged_kernel(LinGemm p) {
  using TA = Tile<T, BM, AKC>;
  using TW = Tile<T, BN, WKC>;
  constexpr int BK = TA::BK, V = TA::V;
  constexpr int WM = BM / 2, WN = BN / 2, TM = WM / 16, TN = WN / 16;
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
  void *c = second ? p.c2 : p.c;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1;

  // A row r (KC) or the group of rows from r on: the first row's index, and
  // how many exist.
  auto a_at = [&](int r, int64_t *row) -> int64_t {
    const int64_t m = m0 + r;
    *row = m < p.M ? m : 0;
    return m < p.M ? p.M - m : 0;
  };
  // W tile row r: with kModeDual each wave's first half are the gate's columns
  // and its second half the up projection's.
  auto w_col = [&](int r) -> int64_t {
    if constexpr (MODE == kModeDual) return n0 + r / WN * (WN / 2) + r % (WN / 2);
    else return n0 + r;
  };
  auto w_at = [&](int r, int64_t *row) -> int64_t {
    const int64_t n = w_col(r);
    *row = n < p.N ? n : 0;
    return n < p.N ? p.N - n : 0;
  };

  u32x4 ga[TA::KB], gw[TW::KB];
  auto load = [&](int64_t k0, const T *Ab, const T *Wb) {
    TA::load(Ab, p.lda, k0, p.K, a_at, ga);
    if constexpr (MODE == kModeDual) {
      // Per thread: the matrix of the tile row (or group) it fetches.
      const T *W2 = static_cast<const T *>(p.w2);
      if constexpr (WKC) {
#pragma unroll
        for (int q = 0; q < TW::KB; ++q) {
          const int idx = threadIdx.x + kThreads * q, r = idx >> 3, ch = idx & 7;
          const int64_t k = k0 + ch * V;
          int64_t row, left = w_at(r, &row) ? p.K - k : 0;
          gw[q] = load16<T>((r % WN < WN / 2 ? Wb : W2) + row * p.ldw + k, left);
        }
      } else {
        const int b = threadIdx.x % TW::NBLK;
        TW::load(b * V % WN < WN / 2 ? Wb : W2, p.ldw, k0, p.K, w_at, gw);
      }
    } else {
      TW::load(Wb, p.ldw, k0, p.K, w_at, gw);
    }
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int64_t per = (p.K + BK - 1) / BK, nst = MODE == kModeCat ? 2 * per : per;
  auto fetch = [&](int64_t st) {
    if constexpr (MODE == kModeCat) {
      if (st >= per) {
        load((st - per) * BK, static_cast<const T *>(p.a2), static_cast<const T *>(p.w2));
        return;
      }
    }
    load(st * BK, A, W);
  };
  auto compute = [&](const char *stage) {
    const char *As = stage, *Ws = stage + LDS_A;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int ch = kk * 4 + (lane >> 4);
      u32x4 fa[TM], fw[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i)
        fa[i] = *reinterpret_cast<const u32x4 *>(As + lds_at(wm * WM + i * 16 + (lane & 15), ch));
#pragma unroll
      for (int j = 0; j < TN; ++j)
        fw[j] = *reinterpret_cast<const u32x4 *>(Ws + lds_at(wn * WN + j * 16 + (lane & 15), ch));
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fw[j]),
                                                                __builtin_bit_cast(bf16x8, fa[i]), acc[i][j], 0, 0, 0);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(fw[j][e]), __uint_as_float(fa[i][e]),
                                                               acc[i][j], 0, 0, 0);
      }
    }
  };

  if (nst > 0) {
    fetch(0);
    TA::store(smem, ga);
    TW::store(smem + LDS_A, gw);
  }
  __syncthreads();
  for (int64_t st = 0; st < nst; ++st) {
    char *cur = smem + (st & 1) * STAGE, *nxt = smem + ((st + 1) & 1) * STAGE;
    const bool more = st + 1 < nst;
    if (more) fetch(st + 1);
    compute(cur);
    if (more) {
      TA::store(nxt, ga);
      TW::store(nxt + LDS_A, gw);
    }
    __syncthreads();
  }

  auto rm = [&](int i) -> int64_t { return m0 + wm * WM + i * 16 + (lane & 15); };
  auto cn = [&](int j) -> int64_t {
    const int wcols = MODE == kModeDual ? WN / 2 : WN;
    return n0 + wn * wcols + j * 16 + 4 * (lane >> 4);
  };
  if constexpr (sizeof(T) == 4) epilogue<float, MODE>(p, c, acc, rm, cn);
  else epilogue<uint16_t, MODE>(p, c, acc, rm, cn);
}

constexpr int64_t kCUs = 256;

template <typename T, bool AKC, bool WKC, int MODE>
hipError_t launch(const LinGemm& p, hipStream_t s) {
  const int64_t products = MODE == kModePair ? 2 : 1, cols = MODE == kModeDual ? 2 * p.N : p.N;
  const int64_t big = (p.M + 127) / 128 * ((cols + 127) / 128) * products;
  const int64_t small = (p.M + 63) / 64 * ((cols + 63) / 64) * products;
  if (big >= kCUs)
    hipLaunchKernelGGL((lin_staged_kernel<T, 128, 128, AKC, WKC, MODE>), dim3(static_cast<unsigned>(big)),
                       dim3(kThreads), 0, s, p);
  else
    hipLaunchKernelGGL((lin_staged_kernel<T, 64, 64, AKC, WKC, MODE>), dim3(static_cast<unsigned>(small)),
                       dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t dispatch(const LinGemm& p, hipStream_t s) {
  const bool akc = !p.a_t, wkc = p.w_t != 0;
  switch (p.mode) {
    case kModeOne:
      if (akc) return wkc ? launch<T, true, true, kModeOne>(p, s) : launch<T, true, false, kModeOne>(p, s);
      break;
    case kModeDual:
      if (akc) return wkc ? launch<T, true, true, kModeDual>(p, s) : launch<T, true, false, kModeDual>(p, s);
      break;
    case kModeCat:
      if (akc) return wkc ? launch<T, true, true, kModeCat>(p, s) : launch<T, true, false, kModeCat>(p, s);
      break;
    case kModePair:
      if (!akc && !wkc) return launch<T, false, false, kModePair>(p, s);
      break;
  }
  if (p.mode == kModeOne && !akc && !wkc) return launch<T, false, false, kModeOne>(p, s);
  return hipErrorInvalidValue;
}

}  // namespace

// Launches are capped at 2^32 threads: 2^23 tiles of 64 x 64 (twice that many
// workgroups of 256 threads where two products share a launch).
bool lin_grid_ok(int64_t M, int64_t N) { return ((M + 63) / 64) * ((N + 63) / 64) < (int64_t{1} << 22); }

hipError_t lin_staged_launch(const LinGemm& p, hipStream_t s) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  return p.f32 ? dispatch<uint32_t>(p, s) : dispatch<uint16_t>(p, s);
}

}  // namespace tpshard
