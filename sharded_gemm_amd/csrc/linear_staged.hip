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
//
// Rows past the edge are clamped onto an existing one, and a row-contiguous
// group that reaches past it reads on into the next rows: both only feed
// outputs that are never stored.  So a stage is fetched without a check per
// element wherever it and the V rows after it lie inside K (there, reading V
// elements from any existing one stays within the operand whatever its stride);
// only the last stages of K are checked, and their missing elements are zero.
template <typename T, int ROWS, bool KC>
struct Tile {
  static constexpr int V = 16 / sizeof(T);          // elements of a 16-byte chunk
  static constexpr int KB = ROWS / 32;              // chunks (KC) or k rows (else) per thread
  static constexpr int NBLK = ROWS / V;             // groups of V rows
  static constexpr int BK = kRow / sizeof(T);
  static_assert(KB == 2 || KB == 4, "tile rows");
  static_assert(KC || NBLK * (BK / KB) == kThreads, "one block of KB k rows per thread");

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
        const int idx = t + kThreads * q;
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

  // `shift`: from the first matrix to the one read (elements).
  __device__ __forceinline__ void load(int64_t k0, int64_t K, int64_t shift, u32x4 (&g)[KB]) const {
    const int t = threadIdx.x;
    if (k0 + BK + V <= K) {
#pragma unroll
      for (int q = 0; q < KB; ++q)
        g[q] = *reinterpret_cast<const u32x4_any *>(KC ? at[KC ? q : 0] + shift + k0 : at[0] + shift + (k0 + q) * ld);
    } else {
#pragma unroll
      for (int q = 0; q < KB; ++q) {
        if constexpr (KC) {
          g[q] = load16<T>(at[q] + shift + k0, K - k0 - ((t + kThreads * q) & 7) * V);
        } else {
          g[q] = load16<T>(at[0] + shift + (k0 + q) * ld, k0 + t / NBLK * KB + q < K ? left : 0);
        }
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
          for (int e = 0; e < KB / 2; ++e)
            d[e] = __builtin_amdgcn_perm(g[2 * e + 1][j >> 1], g[2 * e][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
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
  constexpr int BK = TA::BK;
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
  const T *W2 = static_cast<const T *>(p.w2);
  void *c = second ? p.c2 : p.c;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1;

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

  const int64_t per = (p.K + BK - 1) / BK, all = MODE == kModeCat ? 2 * per : per;
  const int64_t st0 = all * blockIdx.y / gridDim.y, nst = all * (blockIdx.y + 1) / gridDim.y - st0;
  const int64_t a_far = MODE == kModeCat ? static_cast<const T *>(p.a2) - A : 0, w_far = MODE == kModeCat ? W2 - W : 0;
  struct Regs {
    u32x4 a[TA::KB], w[TW::KB];
  };
  auto fetch = [&](int64_t st, Regs& g) {
    st += st0;
    const bool far = MODE == kModeCat && st >= per;
    const int64_t k0 = (far ? st - per : st) * BK;
    ta.load(k0, p.K, far ? a_far : 0, g.a);
    tw.load(k0, p.K, far ? w_far : 0, g.w);
  };
  auto put = [&](int64_t st, const Regs& g) {
    char *slot = smem + (st & 1) * STAGE;
    TA::store(slot, g.a);
    TW::store(slot + LDS_A, g.w);
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

  // Stage st + 2 leaves for the registers that stage st has left, stage st + 1
  // moves from its own to LDS after stage st's products: a load has two stages'
  // time to arrive.
  Regs g0, g1;
  auto step = [&](int64_t st, Regs& mine, const Regs& next) {
    if (st + 2 < nst) fetch(st + 2, mine);
    compute(smem + (st & 1) * STAGE);
    if (st + 1 < nst) put(st + 1, next);
    __syncthreads();
  };
  if (nst > 0) fetch(0, g0);
  if (nst > 1) fetch(1, g1);
  if (nst > 0) put(0, g0);
  __syncthreads();
  for (int64_t st = 0; st < nst; st += 2) {
    step(st, g0, g1);
    if (st + 1 < nst) step(st + 1, g1, g0);
  }
  if (gridDim.y > 1 && !join_splits<kThreads>(p, acc)) return;

  auto rm = [&](int i) -> int64_t { return m0 + wm * WM + i * 16 + (lane & 15); };
  auto cn = [&](int j) -> int64_t {
    const int wcols = MODE == kModeDual ? WN / 2 : WN;
    return n0 + wn * wcols + j * 16 + 4 * (lane >> 4);
  };
  if constexpr (sizeof(T) == 4) epilogue<float, MODE>(p, c, acc, rm, cn);
  else epilogue<uint16_t, MODE>(p, c, acc, rm, cn);
}

constexpr int64_t kCUs = 256;

// The tile's edge (128 where every CU gets such a tile, else 64) and the
// workgroups that split its K.
struct Shape {
  int edge, splits;
  int64_t tiles;
};
Shape shape_of(const LinGemm& p) {
  Shape h{128, 1, lin_tiles_count(p, 128, 128)};
  if (h.tiles >= kCUs) return h;
  h.edge = 64;
  h.tiles = lin_tiles_count(p, 64, 64);
  const int64_t stages = (p.K * (p.f32 ? 4 : 2) + kRow - 1) / kRow * (p.mode == kModeCat ? 2 : 1);
  while (h.splits < 16 && h.tiles * h.splits < 2 * kCUs && stages >= 2 * h.splits * 8) h.splits *= 2;
  return h;
}

template <typename T, bool AKC, bool WKC, int MODE>
hipError_t launch(const LinGemm& p, const Shape& h, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(h.tiles), static_cast<unsigned>(h.splits));
  if (h.edge == 128) hipLaunchKernelGGL((lin_staged_kernel<T, 128, 128, AKC, WKC, MODE>), grid, dim3(kThreads), 0, s, p);
  else hipLaunchKernelGGL((lin_staged_kernel<T, 64, 64, AKC, WKC, MODE>), grid, dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t dispatch(const LinGemm& p, const Shape& h, hipStream_t s) {
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

// Launches are capped at 2^32 threads: 2^23 tiles of 64 x 64 (twice that many
// workgroups of 256 threads where two products share a launch).
bool lin_grid_ok(int64_t M, int64_t N) { return ((M + 63) / 64) * ((N + 63) / 64) < (int64_t{1} << 22); }

int64_t lin_staged_ws(const LinGemm& p) {
  const Shape h = shape_of(p);
  return h.splits > 1 ? kTicketBytes + h.tiles * h.splits * 64 * 64 * 4 : 0;
}

hipError_t lin_staged_launch(LinGemm p, void *ws, int64_t ws_bytes, hipStream_t s) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  Shape h = shape_of(p);
  if (!ws || ws_bytes < lin_staged_ws(p)) h.splits = 1;
  if (h.splits > 1) {
    p.tickets = static_cast<uint32_t *>(ws);
    p.join = reinterpret_cast<float *>(static_cast<char *>(ws) + kTicketBytes);
  }
  return p.f32 ? dispatch<uint32_t>(p, h, s) : dispatch<uint16_t>(p, h, s);
}

}  // namespace tpshard
