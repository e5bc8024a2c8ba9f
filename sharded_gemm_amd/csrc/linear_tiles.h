// The tiled bf16 kernels of the linear layer and the gated block, on gemm.hip's
// building blocks (gemm_tiles.h).  One translation unit instantiates each mode.
//
// Bound by MFMA on large problems.  On an MI355X: the gated forward 4096 x 12288 ->
// 6144 with both pre-activations kept 846 us (1.46 PFLOP/s; a bf16 8192^3 library
// product reaches 1.39), the gated backward 8192 x 4096 -> 2048's input gradient
// over both weights 205 us (1.34) and its two weight gradients 253 us (1.09: both
// operands come through the transposing LDS read).  Two products for the gate and
// the up projection would read X twice and pass both results through memory.
#pragma once

#include "ce_dev.h"
#include "gemm_tiles.h"
#include "linear_dev.h"

namespace tpshard {
namespace {

// The W tile of a stage.  kModeDual: two tiles of BN / 2 columns, the gate's and
// the up projection's, one after the other, so that every DMA piece comes from
// one matrix; a wave's fragments take the same columns of both.
template <int BN, int BK, bool WT, int MODE>
struct WTile {
  static constexpr bool DUAL = MODE == kModeDual;
  using H = OpTile<DUAL ? BN / 2 : BN, BK, WT>;
  __device__ __forceinline__ static bool second(int piece) { return DUAL && piece >= H::PIECES; }
  __device__ __forceinline__ static int64_t src(int piece, int lane, int64_t n0, int64_t N, int64_t ld) {
    return H::src(DUAL ? piece % H::PIECES : piece, lane, n0, N, ld);
  }
  // Fragment j of wave column wn.
  template <typename C>
  __device__ __forceinline__ static bf16x8_t frag(const TP_LDS char *base, int wn, int j, int kk, int lane) {
    if constexpr (DUAL) {
      constexpr int NJ = C::TN / 2;
      return H::frag(base + (j < NJ ? 0 : H::BYTES), wn * (C::WN / 2) + j % NJ * 16, kk, lane);
    } else {
      return H::frag(base, wn * C::WN + j * 16, kk, lane);
    }
  }
};

// Rows that an operand's groups can be read to: whole groups of 8 of a row-contiguous one.
template <bool KC>
__device__ __forceinline__ int64_t rows_of(int64_t n) { return KC ? n : (n + 7) / 8 * 8; }

// What a workgroup computes: its tile, and its part of K.
struct Place {
  int m0, n0;
  bool second;          // kModePair's second product
  int st0, st1;         // its stages
};

template <int BM, int BNO, int BK, int MODE>
__device__ __forceinline__ Place place_of(const LinGemm& p) {
  const int tiles_m = static_cast<int>((p.M + BM - 1) / BM), tiles_n = static_cast<int>((p.N + BNO - 1) / BNO);
  const int ntiles = tiles_m * tiles_n;
  int bid = blockIdx.x;
  Place q;
  q.second = MODE == kModePair && bid >= ntiles;
  if (q.second) bid -= ntiles;
  int tm, tn;
  tile_coords(bid, ntiles, tiles_m, tiles_n, &tm, &tn);
  q.m0 = tm * BM;
  q.n0 = tn * BNO;
  const int nst = static_cast<int>(p.K / BK) * (MODE == kModeCat ? 2 : 1);
  q.st0 = static_cast<int>(static_cast<int64_t>(nst) * blockIdx.y / gridDim.y);
  q.st1 = static_cast<int>(static_cast<int64_t>(nst) * (blockIdx.y + 1) / gridDim.y);
  return q;
}

// Ring kernel (gemm_tiles.h, ring_loop): tiles for problems that fill the chip
// with smaller ones only, any K that is a multiple of BK.
template <int BM, int BN, int BK, int S, int MODE, bool AT, bool WT, int WAVES_M, int WAVES_N>
__global__ void __launch_bounds__(64 * WAVES_M * WAVES_N, 1) lin_ring_kernel(LinArgs<MODE> p) {
  using C = DmaCfg<BM, BN, BK, S, AT, WT, WAVES_M, WAVES_N>;
  using TA = typename C::TA;
  using TW = typename C::TW;
  using WO = WTile<BN, BK, WT, MODE>;
  constexpr int KK = C::KK, BNO = MODE == kModeDual ? BN / 2 : BN;
  __shared__ __attribute__((aligned(1024))) char smem[S * C::STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  const Place pl = place_of<BM, BNO, BK, MODE>(p);
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((TP_LDS char *)smem));
  const uint16_t *A = static_cast<const uint16_t *>(pl.second ? p.a2 : p.a);
  const uint16_t *W = static_cast<const uint16_t *>(pl.second ? p.w2 : p.w);
  const uint16_t *W2 = static_cast<const uint16_t *>(p.w2);
  const uint16_t *A2 = static_cast<const uint16_t *>(p.a2);
  int64_t a_src[C::A_PW], w_src[C::W_PW];
#pragma unroll
  for (int q = 0; q < C::A_PW; ++q) a_src[q] = TA::src(wave * C::A_PW + q, lane, pl.m0, rows_of<!AT>(p.M), p.lda);
#pragma unroll
  for (int q = 0; q < C::W_PW; ++q)
    w_src[q] = WO::src(min(wave + q * C::NW, TW::PIECES - 1), lane, pl.n0, rows_of<WT>(p.N), p.ldw);
  const int64_t a_step = TA::step(p.lda), w_step = TW::step(p.ldw);
  const int half = static_cast<int>(p.K / BK);
  auto issue = [&](int st, int slot) {
    const uint32_t base = lds0 + slot * C::STAGE;
    const uint16_t *Ab = A, *Wb = W;
    int at = pl.st0 + st;
    if (MODE == kModeCat && at >= half) {
      Ab = A2;
      Wb = W2;
      at -= half;
    }
#pragma unroll
    for (int q = 0; q < C::A_PW; ++q) lds_dma16(Ab + a_src[q] + at * a_step, base + (wave * C::A_PW + q) * 1024);
#pragma unroll
    for (int q = 0; q < C::W_PW; ++q)
      if (C::W_REM == 0 || q + 1 < C::W_PW || wave < C::W_REM)
        lds_dma16((WO::second(wave + q * C::NW) ? W2 : Wb) + w_src[q] + at * w_step,
                  base + TA::BYTES + (wave + q * C::NW) * 1024);
  };
  const bool dma_hi = C::W_REM == 0 || wave < C::W_REM;
  auto wait_stages = [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (dma_hi) wait_vmcnt<N * C::L_HI>(); else wait_vmcnt<N * C::L_LO>();
  };
  auto read = [&](int u, bf16x8_t (&fa)[C::TM], bf16x8_t (&fb)[C::TN]) {
    const int kk = KK == 1 ? 0 : (u & 1);
    const TP_LDS char *base = (const TP_LDS char *)smem + ((u / KK) % S) * C::STAGE;
#pragma unroll
    for (int i = 0; i < C::TM; ++i) fa[i] = TA::frag(base, wm * C::WM + i * 16, kk, lane);
#pragma unroll
    for (int j = 0; j < C::TN; ++j) fb[j] = WO::template frag<C>(base + TA::BYTES, wn, j, kk, lane);
  };
  f32x4_t acc[C::TM][C::TN];
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto mma = [&](const bf16x8_t (&fa)[C::TM], const bf16x8_t (&fb)[C::TN]) {
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
#pragma unroll
      for (int i = 0; i < C::TM; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
  };
  const int pending = 0;
  if (pl.st1 > pl.st0) ring_loop<C, S, false>(pl.st1 - pl.st0, issue, wait_stages, read, mma, [] {}, pending);
  if (gridDim.y > 1 && !lin::join_splits<C::THREADS>(p, acc)) return;

  auto rm = [&](int i) -> int64_t { return pl.m0 + wm * C::WM + i * 16 + (lane & 15); };
  auto cn = [&](int j) -> int64_t {
    return pl.n0 + wn * (MODE == kModeDual ? C::WN / 2 : C::WN) + j * 16 + 4 * (lane >> 4);
  };
  if constexpr (MODE == kModeStats)
    ce::stats<BM, C::WAVES_N, C::THREADS>(p, smem, acc, pl.m0, p.slot0 + pl.n0 / BN, wn, pl.n0 + BN <= p.cols, rm, cn);
  else if constexpr (MODE == kModeProb) ce::prob<uint16_t>(p, acc, rm, cn);
  else if constexpr (MODE == kModeScaled) ce::scaled(p, acc, rm, cn);
  else lin::epilogue<uint16_t, MODE>(p, pl.second ? p.c2 : p.c, acc, rm, cn);
}

// Ping-pong kernel (gemm_tiles.h, pps_loop) on 256-row tiles.
template <int BM, int BN, int MODE, bool AT, bool WT, int WGM = 2>
__global__ void __launch_bounds__(512, 1) lin_pps_kernel(LinArgs<MODE> p) {
  constexpr int BK = 64, NG = 4, SA = 3, SW = 2;
  using C = DmaCfg<BM, BN, BK, 2, AT, WT, WGM, 8 / WGM>;
  using TA = typename C::TA;
  using TW = typename C::TW;
  using WO = WTile<BN, BK, WT, MODE>;
  constexpr int A_PW = TA::PIECES / NG, W_PW = TW::PIECES / NG, BNO = MODE == kModeDual ? BN / 2 : BN;
  constexpr int W_BASE = SA * TA::BYTES;
  static_assert(TA::PIECES % NG == 0 && TW::PIECES % NG == 0, "DMA split");
  static_assert(MODE != kModeDual || WO::H::PIECES % W_PW == 0, "a wave's pieces come from one matrix");
  static_assert(SA * TA::BYTES + SW * TW::BYTES <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) char smem[SA * TA::BYTES + SW * TW::BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  const bool grpA = wave < 4;
  const Place pl = place_of<BM, BNO, BK, MODE>(p);
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((TP_LDS char *)smem));
  const uint32_t step = static_cast<uint32_t>((grpA ? TA::step(p.lda) : TW::step(p.ldw)) * 2);
  const void *a_base = pl.second ? p.a2 : p.a;
  const void *w_base = pl.second || WO::second((wave & 3) * W_PW) ? p.w2 : p.w;
  const int half = static_cast<int>(p.K / BK), st0 = MODE == kModeSlices ? pl.st0 : 0;
  auto dma_a = [&](int q, int st, int slot_st) {
    const uint32_t src = static_cast<uint32_t>(TA::src((wave & 3) * A_PW + q, lane, pl.m0, rows_of<!AT>(p.M), p.lda) * 2);
    const bool far = MODE == kModeCat && st >= half;
    lds_dma16_s(far ? p.a2 : a_base, src + (far ? st - half : st + st0) * step,
                lds0 + (slot_st % SA) * TA::BYTES + ((wave & 3) * A_PW + q) * 1024);
  };
  auto dma_w = [&](int q, int st, int slot_st) {
    const uint32_t src = static_cast<uint32_t>(WO::src((wave & 3) * W_PW + q, lane, pl.n0, rows_of<WT>(p.N), p.ldw) * 2);
    const bool far = MODE == kModeCat && st >= half;
    lds_dma16_s(far ? p.w2 : w_base, src + (far ? st - half : st + st0) * step,
                lds0 + W_BASE + (slot_st % SW) * TW::BYTES + ((wave & 3) * W_PW + q) * 1024);
  };
  auto read_a = [&](int i, int kk, int st) {
    return TA::frag((const TP_LDS char *)smem + (st % SA) * TA::BYTES, wm * C::WM + i * 16, kk, lane);
  };
  auto read_w = [&](int j, int kk, int st) {
    return WO::template frag<C>((const TP_LDS char *)smem + W_BASE + (st % SW) * TW::BYTES, wn, j, kk, lane);
  };
  f32x4_t acc[C::TM][C::TN];
  auto init_acc = [&]() {
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  };
  pps_loop<C, A_PW, W_PW>(grpA, pl.st1 - st0, acc, dma_a, dma_w, read_a, read_w, init_acc);

  auto rm = [&](int i) -> int64_t { return pl.m0 + wm * C::WM + i * 16 + (lane & 15); };
  auto cn = [&](int j) -> int64_t {
    return pl.n0 + wn * (MODE == kModeDual ? C::WN / 2 : C::WN) + j * 16 + 4 * (lane >> 4);
  };
  if constexpr (MODE == kModeStats)
    ce::stats<BM, C::WAVES_N, C::THREADS>(p, smem, acc, pl.m0, p.slot0 + pl.n0 / BN, wn, pl.n0 + BN <= p.cols, rm, cn);
  else if constexpr (MODE == kModeProb) ce::prob<uint16_t>(p, acc, rm, cn);
  else if constexpr (MODE == kModeScaled) ce::scaled(p, acc, rm, cn);
  else if constexpr (MODE == kModeSlices)
    lin::epilogue<uint16_t, MODE>(p, static_cast<float *>(p.c) + blockIdx.y * p.M * p.ldc, acc, rm, cn);
  else lin::epilogue<uint16_t, MODE>(p, pl.second ? p.c2 : p.c, acc, rm, cn);
}

// ---- launchers -----------------------------------------------------------------

template <int BM, int BN, int BK, int S, int MODE, bool AT, bool WT, int WAVES_M, int WAVES_N>
hipError_t launch_ring(const LinGemm& p, int splits, hipStream_t s) {
  hipLaunchKernelGGL((lin_ring_kernel<BM, BN, BK, S, MODE, AT, WT, WAVES_M, WAVES_N>),
                     dim3(static_cast<unsigned>(lin_tiles_count(p, BM, BN)), static_cast<unsigned>(splits)),
                     dim3(64 * WAVES_M * WAVES_N), 0, s,
                     lin_args<MODE>(p));
  return hipGetLastError();
}

template <int BM, int BN, int MODE, bool AT, bool WT, int WGM = 2>
hipError_t launch_lin_pps(const LinGemm& p, hipStream_t s, int slices = 1) {
  hipLaunchKernelGGL((lin_pps_kernel<BM, BN, MODE, AT, WT, WGM>),
                     dim3(static_cast<unsigned>(lin_tiles_count(p, BM, BN)), static_cast<unsigned>(slices)), dim3(512), 0, s,
                     lin_args<MODE>(p));
  return hipGetLastError();
}

template <int MODE, bool AT, bool WT>
hipError_t dispatch_tiles(const LinGemm& p, const TilePick& t, hipStream_t s) {
  constexpr bool dual = MODE == kModeDual;
  constexpr int WGM = AT ? 4 : 2;
  switch (t.tile) {
    case kTile256:
      if constexpr (!AT || WT) return launch_lin_pps<256, 256, MODE, AT, WT, WGM>(p, s);
      break;
    case kTile192:
      if constexpr (!dual) return launch_lin_pps<256, 192, MODE, AT, WT, WGM>(p, s);
      break;
    case kTile128w: return launch_lin_pps<256, 128, MODE, AT, WT, AT || WT ? 4 : 2>(p, s);
    case kTile128: return launch_ring<128, 128, 32, 8, MODE, AT, WT, 2, 4>(p, t.splits, s);
    case kTile64: return launch_ring<64, dual ? 128 : 64, 64, 3, MODE, AT, WT, 2, 2>(p, t.splits, s);
    case kTile64short: return launch_ring<64, dual ? 128 : 64, 64, 2, MODE, AT, WT, 2, 2>(p, t.splits, s);
    case kTile32:
      if constexpr (MODE == kModeStats) return launch_ring<32, 64, 64, 4, MODE, AT, WT, 2, 2>(p, t.splits, s);
      break;
    case kTile64k32:   // (a^T w^T: K is tokens, in multiples of 64)
      if constexpr (!AT || !WT) return launch_ring<64, dual ? 128 : 64, 32, 4, MODE, AT, WT, 2, 2>(p, t.splits, s);
      break;
  }
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace tpshard
