// Device building blocks of the bf16 GEMMs: operand tiles in LDS, the DMA that
// fills them and the two main loops (a ring of stages; the ping-pong of two wave
// groups).  gemm.hip's header comment describes the design.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace tpshard {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

#define TP_LDS __attribute__((address_space(3)))

namespace {

constexpr int kCUs = 256;

// ---- XCD-aware tile order ------------------------------------------------
// Workgroups are dealt round-robin to the 8 XCDs, each with its own L2.
// Hand XCD x a contiguous range of logical tiles, then walk tiles in groups
// of kGroupM tile rows so neighbours share operand panels in that L2.
constexpr int kXcds = 8;
constexpr int kGroupM = 4;

__device__ __forceinline__ void tile_coords(int bid, int ntiles, int tiles_m, int tiles_n, int *tm, int *tn) {
  const int per = ntiles / kXcds, rem = ntiles % kXcds;
  const int x = bid % kXcds, i = bid / kXcds;
  const int t = x * per + (x < rem ? x : rem) + i;
  const int in_group = kGroupM * tiles_n;
  const int g = t / in_group;
  const int first_m = g * kGroupM;
  const int gm = (tiles_m - first_m) < kGroupM ? (tiles_m - first_m) : kGroupM;
  const int local = t - g * in_group;
  *tm = first_m + local % gm;
  *tn = local / gm;
}

// ---- LDS-DMA ring ---------------------------------------------------------

// One LDS-DMA load: this lane's 16 bytes at g land at LDS byte address
// lds + 16 * lane.  lds must be wave-uniform (it goes to M0).
__device__ __forceinline__ void lds_dma16(const void *g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g),
               "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory");
}

// s_waitcnt vmcnt(N) (expcnt and lgkmcnt left alone).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// s_waitcnt lgkmcnt(0) (vmcnt and expcnt left alone).
__device__ __forceinline__ void wait_lgkmcnt0() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
}

// One operand's tile of a stage in LDS.  ROWS is the output extent it feeds
// (BM for A, BN for W).
//  * KC (k-contiguous in memory): ROWS LDS rows of BK k (2 * BK bytes each);
//    chunk c of row r sits at c ^ swz(r), so that the 8 rows a DMA instruction
//    or a 16-lane read group touches hit distinct banks; fragments are one
//    ds_read_b128 per lane (row = lane & 15, k chunk = lane >> 4).
//  * otherwise (row/column-contiguous): BK LDS rows (one per k) of ROWS
//    elements; chunk c of k-row r sits at c ^ 2 (r & 3), so the 4 k-rows a
//    transposing read touches hit distinct banks; a fragment is two
//    ds_read_b64_tr_b16 (lane 4 r + q of group g reads k-row 8 g + r (+4),
//    columns 4 q .. 4 q + 3; lane j of the group then holds column j, 4 k).
// DMA pieces are 1 KiB: lane l of piece p covers tile bytes 1024 p + 16 l.
template <int ROWS, int BK, bool KC>
struct OpTile {
  static constexpr int BYTES = ROWS * BK * 2;
  static constexpr int PIECES = BYTES / 1024;
  static constexpr int RB = KC ? BK * 2 : ROWS * 2;   // bytes per LDS row
  static_assert(BYTES % 1024 == 0 && RB % 16 == 0, "operand tile");
  static_assert(KC || (RB / 16) % 8 == 0, "row-contiguous tiles need 8-chunk rows for their swizzle");

  __device__ __forceinline__ static int swz(int r) {
    return KC ? (BK == 32 ? ((r >> 1) & 3) : (r & 7)) : 2 * (r & 3);
  }
  // Element offset, from the operand base at k = 0, of this lane's 16 bytes
  // of piece `piece` for the tile whose first row (m or n) is row0.  Rows (KC)
  // or 8-column groups (otherwise) past nrows are clamped onto valid memory:
  // they only feed outputs that are never stored.
  __device__ __forceinline__ static int64_t src(int piece, int lane, int64_t row0, int64_t nrows, int64_t ld) {
    const int byte = piece * 1024 + lane * 16;
    const int r = byte / RB, c = ((byte % RB) >> 4) ^ swz(r);
    if constexpr (KC) {
      const int64_t g = (row0 + r < nrows) ? row0 + r : nrows - 1;
      return g * ld + c * 8;
    } else {
      const int64_t g = (row0 + c * 8 < nrows) ? row0 + c * 8 : nrows - 8;
      return static_cast<int64_t>(r) * ld + g;
    }
  }
  // Element advance of the source per stage (k0 -> k0 + BK).
  __device__ __forceinline__ static int64_t step(int64_t ld) { return KC ? BK : BK * ld; }
  // MFMA operand fragment of the 16 rows starting at tile row `row`, k-step kk.
  __device__ __forceinline__ static bf16x8_t frag(const TP_LDS char *base, int row, int kk, int lane) {
    if constexpr (KC) {
      const int r = row + (lane & 15), c = kk * 4 + (lane >> 4);
      return *(const TP_LDS bf16x8_t *)(base + r * RB + ((c ^ swz(r)) << 4));
    } else {
      const int col = row + 4 * (lane & 3);
      const int k = kk * 32 + 8 * (lane >> 4) + ((lane & 15) >> 2);
      const int o = k * RB + (((col >> 3) ^ swz(k)) << 4) + (col & 7) * 2;   // k + 4: same swizzle
      const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TP_LDS i16x4_t *)(base + o));
      const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TP_LDS i16x4_t *)(base + o + 4 * RB));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// AT: A given transposed (m-contiguous); WT: W given transposed (k-contiguous).
template <int BM, int BN, int BK, int S, bool AT, bool WT, int WAVES_M_ = 2, int WAVES_N_ = 4>
struct DmaCfg {
  using TA = OpTile<BM, BK, !AT>;
  using TW = OpTile<BN, BK, WT>;
  static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, NW = WAVES_M * WAVES_N, THREADS = 64 * NW;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 16, TN = WN / 16;
  static constexpr int KK = BK / 32;                   // MFMA k-steps per stage
  static constexpr int STAGE = TA::BYTES + TW::BYTES;
  // The A pieces split evenly over the waves; the W pieces are dealt
  // round-robin, so when they do not divide evenly the first W_REM waves
  // issue one more than the rest.
  static constexpr int A_PW = TA::PIECES / NW;
  static constexpr int W_PW = (TW::PIECES + NW - 1) / NW, W_REM = TW::PIECES % NW;
  static constexpr int L_HI = A_PW + W_PW, L_LO = W_REM ? L_HI - 1 : L_HI;   // per-wave DMA count
  static_assert((BK == 32 || BK == 64) && WN % 16 == 0 && WM % 16 == 0, "tile shape");
  static_assert(A_PW >= 1 && TA::PIECES % NW == 0 && TW::PIECES >= NW, "DMA split");
  static_assert((S - 1) * L_HI < 64, "vmcnt range");
  static_assert(S * STAGE <= 160 * 1024, "LDS");
};

// The main loop over the stages of a tile: fragments of step u + 1 are read
// while step u multiplies.
//
// Stage t lives in slot t % S.  The barrier that opens stage t (after this
// wave's loads of stage t have landed: vmcnt) also proves every wave has
// read stage t-1 into registers (lgkmcnt(0) before it: the DMA is invisible
// to the compiler's own waits), so stage t+S-1 is issued into its slot.
//
// issue(st, slot) starts this wave's DMA of a stage; wait_stages(n) waits until
// at most n stages of it are in flight; read(u, fa, fb) fetches step u's
// fragments; mma(fa, fb) multiplies.  With PF the caller streams other vectors
// in beside the stages: prefetch() issues at most one load right after a
// stage's DMA and *pf_pending says whether it did (the next opening may leave
// exactly that one in flight).
template <typename C, int S, bool PF, typename Issue, typename Wait, typename Read, typename Mma, typename Prefetch>
__device__ __forceinline__ void ring_loop(int nst, Issue&& issue, Wait&& wait_stages, Read&& read, Mma&& mma,
                                          Prefetch&& prefetch, const int& pf_pending) {
  constexpr int KK = C::KK;
  const int nu = nst * KK;
  auto open_stage = [&](int st) {
    if constexpr (PF) {
      if (pf_pending) wait_vmcnt<1>(); else wait_vmcnt<0>();
    } else {
      if (st + S - 2 < nst) wait_stages(std::integral_constant<int, S - 2>{}); else wait_vmcnt<0>();
    }
    wait_lgkmcnt0();
    __syncthreads();
    if (st + S - 1 < nst) issue(st + S - 1, (st + S - 1) % S);
    if constexpr (PF) prefetch();
  };
#pragma unroll
  for (int st = 0; st < S; ++st)
    if (st < nst) issue(st, st);
  if (nst >= S) wait_stages(std::integral_constant<int, S - 1>{}); else wait_vmcnt<0>();
  __syncthreads();
  bf16x8_t fa0[C::TM], fb0[C::TN], fa1[C::TM], fb1[C::TN];
  read(0, fa0, fb0);
  int u = 0;
  for (; u + 2 <= nu; u += 2) {
    if ((u + 1) % KK == 0) open_stage((u + 1) / KK);
    read(u + 1, fa1, fb1);
    mma(fa0, fb0);
    if (u + 2 < nu) {
      if ((u + 2) % KK == 0) open_stage((u + 2) / KK);
      read(u + 2, fa0, fb0);
    }
    mma(fa1, fb1);
  }
  if (u < nu) mma(fa0, fb0);
}

// ---- ping-pong ------------------------------------------------------------

// DMA of 16 bytes at sbase + voff (32-bit byte offset) into LDS M0 + 16 * lane.
__device__ __forceinline__ void lds_dma16_s(const void *sbase, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(sbase),
               "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory");
}
// Barriers of the schedule, each with the wait it needs folded in, so no LDS
// read or DMA can be moved across it.
__device__ __forceinline__ void barrier_lgkm0() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void barrier_vm0() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void barrier_raw() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// s_waitcnt vmcnt(n * L) for a run-time n in [0, NMAX] (the count must be an
// immediate), folded with the barrier that follows it.
template <int L, int NMAX>
__device__ __forceinline__ void barrier_vm_n(int n) {
  if constexpr (NMAX == 0) {
    barrier_vm0();
  } else {
    if (n >= NMAX) {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(NMAX * L) : "memory");
      __builtin_amdgcn_sched_barrier(0);
    } else {
      barrier_vm_n<L, NMAX - 1>(n);
    }
  }
}

// The ping-pong kernel (bf16_gemm_pps): 8 waves (WGM x 8/WGM) on a 256-row
// tile, K staged 64 at a time.  Waves 0-3 (group A, tile rows 0..127) and
// 4-7 (group B, rows 128..255) run one barrier apart; wave w sits on SIMD
// w % 4, so each SIMD holds one wave of each group and feeds its matrix pipe
// from one while the other reads LDS.  With a single two-slot ring every DMA
// of stage s would have to leave in the one phase that follows the barrier
// after which both groups are done with stage s-2 and precedes the one after
// which group A reads stage s-1, the phase in which group A reads LDS: the
// issue of a stage's 40-64 DMA instructions (about 15 cycles each through the
// CU's address unit) then held up group A's reads while group B waited at the
// barrier (MI355X phase stamps on the 175B GEMM1 shape: about 830 of 2950
// cycles per stage).  Here the A tile has a ring of three slots and W's tile a
// ring of two, and each group issues its tile between its own MFMAs:
//   A: a0 a1 | #0 | R_0 #1 M_0+a2 #2 | R_1 #3 M_1+a3 #4 | ...
//   B: w0    | #0 | w1 #1 R_0 #2 M_0+w2 #3 R_1 #4 M_1+w3 ...
// (aS, wS: the A / W tile of stage S; R reads, M multiplies).  Group A's
// A tile of stage t+2 overwrites stage t-1's slot after #2t+1, group B's W
// tile of stage t+1 stage t-1's slot after #2t; both groups finished reading
// stage t-1 by #2t.  Before #2t+2, after which group A reads stage t+1, group
// A waits for its A tile of stage t+1 (stage t+2's stays in flight) and group
// B for its W tile of stage t+1.  Every MFMA phase carries its DMA, so the
// loop has one body and one MFMA chain per group (duplicated chains made the
// compiler spill): where the stage it would fetch does not exist, it fetches
// the last stage again, into the slot of the nominal stage, which nothing
// reads any more.  Same accumulation order as every other kernel, so the
// results are the same bits.  Measured on MI355X against the single-ring
// form: 7-15% faster on every 256 x 192 and 256 x 128 shape here, forward and
// backward, 8% on 256 x 256 and 9-14% with the accumulating epilogue.
// dma_a / dma_w(q, st, slot_st): piece q of this wave's share of stage st's A / W
// tile, into the slot of stage slot_st; read_a / read_w(i, kk, st): fragment i of
// step kk; init_acc() sets the accumulators before a group's first product.
template <typename C, int A_PW, int W_PW, typename DmaA, typename DmaW, typename ReadA, typename ReadW, typename Init>
__device__ __forceinline__ void pps_loop(bool grpA, int nst, f32x4_t (&acc)[C::TM][C::TN], DmaA&& dma_a, DmaW&& dma_w,
                                         ReadA&& read_a, ReadW&& read_w, Init&& init_acc) {
  constexpr int KK = C::KK;
  bf16x8_t fa[KK][C::TM], fb[KK][C::TN];
  auto read_stage = [&](int st) {
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
      for (int i = 0; i < C::TM; ++i) fa[kk][i] = read_a(i, kk, st);
#pragma unroll
      for (int j = 0; j < C::TN; ++j) fb[kk][j] = read_w(j, kk, st);
    }
  };
  // The stage's MFMAs with ND DMA pieces of stage `dst` spread between them:
  // piece q after MFMA number (q + 1/2) * NF / ND (ND = 0: none; measured
  // 1.5-3% faster than starting at the first MFMA).  Everything is
  // compile-time, so the chain is one basic block; the scheduling barriers
  // keep each DMA where it is written.
  constexpr int NF = KK * C::TN * C::TM;
  auto mma_stage = [&](auto nd, auto is_a, int dst, int dslot) {
    constexpr int ND = decltype(nd)::value;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
      for (int j = 0; j < C::TN; ++j)
#pragma unroll
        for (int i = 0; i < C::TM; ++i) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[kk][j], fa[kk][i], acc[i][j], 0, 0, 0);
          if constexpr (ND > 0) {
            const int f = (kk * C::TN + j) * C::TM + i;
#pragma unroll
            for (int q = 0; q < ND; ++q)
              if (f == q * NF / ND + NF / (2 * ND)) {
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (decltype(is_a)::value) dma_a(q, dst, dslot); else dma_w(q, dst, dslot);
                __builtin_amdgcn_sched_barrier(0);
              }
          }
        }
  };
  using I0 = std::integral_constant<int, 0>;
  using IA = std::integral_constant<int, A_PW>;
  using IW = std::integral_constant<int, W_PW>;
  using T = std::true_type;
  using F = std::false_type;

  // Every MFMA phase carries its DMA, so the loop has one body: in the last
  // iterations, where the stage it would fetch does not exist, it fetches the
  // last stage again into a slot that nothing reads any more (A: the slot of
  // stage t-1, W: that of stage t-1, both finished by #2t), and the waits
  // stay as in the steady state.
  const int last = nst - 1;
  if (nst > 0) {
    if (grpA) {
#pragma unroll
      for (int q = 0; q < A_PW; ++q) dma_a(q, 0, 0);
#pragma unroll
      for (int q = 0; q < A_PW; ++q) dma_a(q, min(1, last), 1);
      wait_vmcnt<A_PW>();
    } else {
#pragma unroll
      for (int q = 0; q < W_PW; ++q) dma_w(q, 0, 0);
      wait_vmcnt<0>();
    }
  }
  barrier_raw();                                     // #0
  if (grpA) {
    init_acc();
    for (int t = 0; t < nst; ++t) {
      read_stage(t);
      barrier_lgkm0();                               // #2t+1
      mma_stage(IA{}, T{}, min(t + 2, last), t + 2);   // stage t+2's A tile, slot (t+2) % 3
      barrier_vm_n<A_PW, 1>(1);                      // #2t+2: stage t+1's A tile landed
    }
  } else if (nst > 0) {
#pragma unroll
    for (int q = 0; q < W_PW; ++q) dma_w(q, min(1, last), 1);
    barrier_raw();                                   // #1
    read_stage(0);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");   // #2
    __builtin_amdgcn_sched_barrier(0);
    init_acc();
    for (int t = 1; t < nst; ++t) {
      mma_stage(IW{}, F{}, min(t + 1, last), t + 1);   // stage t+1's W tile, slot (t+1) % 2
      barrier_raw();                                 // #2t+1
      read_stage(t);
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");   // #2t+2
      __builtin_amdgcn_sched_barrier(0);
    }
    mma_stage(I0{}, F{}, 0, 0);
  } else {
    init_acc();
  }
  wait_vmcnt<0>();                                   // the repeated fetches of the last stage
}

}  // namespace

}  // namespace tpshard
