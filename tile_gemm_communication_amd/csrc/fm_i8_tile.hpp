// fm_i8_tile.hpp -- macro-tiles of 8-bit products on v_mfma_i32_32x32x32_i8.
//
// Four waves, 2 x 2 over a BM x BN tile of C = A W^T; both operands lie with k in a row,
// so one layout and one read serve both.  A K step is 128 bytes of every row; LDS holds
// AHEAD + 1 steps of A's rows and AHEAD of W's, filled by direct-to-LDS loads.  A step
// has four sub-steps of one instruction depth (32).  The fragments of a sub-step are
// read two sub-steps ahead, four register slots in turn:
//   sub-steps 0, 1  MFMAs, reading sub-steps 2, 3 of this stage, and A's loads of
//                   stage kt + AHEAD into the place of stage kt - 1;
//   wait, barrier   the next stage has landed, this one is drained;
//   sub-steps 2, 3  MFMAs, reading sub-steps 0, 1 of the next stage, and W's loads of
//                   stage kt + AHEAD into this one's place.
// So the loads come evenly, a quarter a sub-step; one memory operation follows each
// MFMA (sched_barrier keeps the order), and the matrix cores do not wait for a burst of
// them.  A 256 x 256 step is 64 MFMAs of 32 cycles a wave on 32 LDS reads: LDS is busy for
// three quarters of that time, the loads' path for half.
//
// 16-byte chunk c of row m is stored at chunk c ^ ((m ^ m >> 3) & 7), which spreads the
// reads of eight rows over all banks; the loads realise it by which chunk a lane fetches.
// The first MFMA operand is W, so lane l holds row l % 32 of C and, for item 4 r + q,
// column 8 r + 4 (l / 32) + q: runs of four columns.
#pragma once

#include "fm_i8_choice.hpp"
#include "fm_tile.hpp"

namespace fm {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

template <int BM, int BN, int AHEAD>
struct I8Tile {
  static constexpr int WM = BM / 2, WN = BN / 2;
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int A_STAGE = BM * kI8Step, W_STAGE = BN * kI8Step;
  static constexpr int W_AT = (AHEAD + 1) * A_STAGE;
  static constexpr int A_DMA = BM / 32, W_DMA = BN / 32;   // loads of a wave, 8 rows each
  static constexpr int DMA = A_DMA + W_DMA;
  static constexpr int READS = FM + FN, MFMAS = FM * FN;
  static constexpr int LDS_BYTES = W_AT + AHEAD * W_STAGE;
  static_assert(BM % 64 == 0 && BN % 64 == 0 && AHEAD >= 2 && LDS_BYTES <= 160 * 1024, "tile size");

  char* smem;
  uint32_t lds0;
  int lane, w, wm, wn, KT, tail;   // tail: bytes of the last step, 0 if whole
  const char *a_base, *w_base;
  uint32_t off[DMA];               // a lane's byte in each of its loads' rows
  uint32_t ra[4][2], rw[4][2];     // LDS offsets of a fragment by sub-step and block parity
  i32x16 acc[FM][FN];
  i32x4 fa[4][FM], fw[4][FN];

  __device__ __forceinline__ I8Tile(char* s, int64_t K) : smem(s) {
    lane = threadIdx.x & 63;
    w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    wm = w >> 1;
    wn = w & 1;
    lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)s);
    KT = (int)cdiv(K, kI8Step);
    tail = (int)(K % kI8Step);
    const int r32 = lane & 31, hi = lane >> 5, s0 = swz_a(r32);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        // row wm * WM + 32 i + r32: its swizzle is s0 ^ 4 (number of the 32-row block & 1)
        ra[ks][p] = (wm * WM + r32) * kI8Step + (((2 * ks + hi) ^ s0 ^ (4 * ((p + wm * FM) & 1))) << 4);
        rw[ks][p] = W_AT + (wn * WN + r32) * kI8Step +
                    (((2 * ks + hi) ^ s0 ^ (4 * ((p + wn * FN) & 1))) << 4);
      }
  }

  // Load d of this wave fills rows 8 (w DMA' + d) .. + 7 of A or W, DMA' loads each.
  __device__ __forceinline__ int dma_row(int d) const {
    return d < A_DMA ? w * (BM / 4) + 8 * d + (lane >> 3) : w * (BN / 4) + 8 * (d - A_DMA) + (lane >> 3);
  }
  __device__ __forceinline__ int dma_chunk(int d) const { return (lane & 7) ^ swz_a(dma_row(d)); }

  // Rows past the last (`rows`, `cols`: those that exist) are read as the last.
  __device__ __forceinline__ void set_tile(const char* a, int rows, const char* wt, int cols, int64_t K) {
    a_base = a;
    w_base = wt;
#pragma unroll
    for (int d = 0; d < DMA; ++d) {
      const int r = min(dma_row(d), (d < A_DMA ? rows : cols) - 1);
      off[d] = (uint32_t)r * (uint32_t)K + dma_chunk(d) * 16;
    }
  }

  __device__ __forceinline__ uint32_t dma_at(int d, int buf) const {
    return d < A_DMA ? buf * A_STAGE + w * (BM / 4) * kI8Step + d * 1024
                     : W_AT + buf * W_STAGE + w * (BN / 4) * kI8Step + (d - A_DMA) * 1024;
  }
  // Load d of stage kt into place buf.  LAST: in the last step a lane whose chunk lies
  // past K loads its row's first chunk of the step instead.
  template <bool LAST>
  __device__ __forceinline__ void dma_item(int d, int kt, int buf) {
    uint32_t at = off[d];
    if constexpr (LAST) {
      const int c = dma_chunk(d) * 16;
      if (kt == KT - 1 && tail && c >= tail) at -= c;
    }
    dma16(at, (d < A_DMA ? a_base : w_base) + (int64_t)kt * kI8Step, lds0 + dma_at(d, buf));
  }
  // Its chunks past K count as zeros: A's are cleared, once this wave's loads have landed.
  __device__ __forceinline__ void clear_tail(int buf) {
#pragma unroll
    for (int d = 0; d < A_DMA; ++d)
      if (dma_chunk(d) * 16 >= tail)
        *reinterpret_cast<u32x4*>(smem + dma_at(d, buf) + lane * 16) = u32x4{0, 0, 0, 0};
  }

  __device__ __forceinline__ void read_item(int q, int abuf, int wbuf, int ks, int slot) {
    // A and W in turn, as the first MFMAs need them
    const int pairs = 2 * (FM < FN ? FM : FN);
    const bool is_a = q < pairs ? q % 2 == 0 : FM > FN;
    const int j = q < pairs ? q / 2 : q - pairs / 2;
    if (is_a)
      fa[slot][j] = *reinterpret_cast<const i32x4*>(smem + abuf * A_STAGE + ra[ks][j & 1] + j * 32 * kI8Step);
    else
      fw[slot][j] = *reinterpret_cast<const i32x4*>(smem + wbuf * W_STAGE + rw[ks][j & 1] + j * 32 * kI8Step);
  }

  // MFMAs on slot m; reads of sub-step ks into slot r; loads d0 .. d1 - 1 of stage kt into
  // place dbuf (LOAD 0: none, 2: perhaps the last stage).
  template <bool READ, int LOAD>
  __device__ __forceinline__ void substep(int m, int abuf, int wbuf, int ks, int r, int kt, int dbuf, int d0,
                                          int d1) {
    static_for<MFMAS>([&](auto qc) {
      constexpr int q = decltype(qc)::value;
      constexpr int i = q / FN, j = q % FN;
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[m][j], fa[m][i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (READ && q < READS) {
        read_item(q, abuf, wbuf, ks, r);
        __builtin_amdgcn_sched_barrier(0);
      }
      // the loads spread over the MFMAs, from the last on
      const int n = d1 - d0, from = n * q / MFMAS, to = n * (q + 1) / MFMAS;
      if (LOAD && to > from) {
#pragma unroll
        for (int d = from; d < to; ++d) dma_item<LOAD == 2>(d0 + d, kt, dbuf);
        __builtin_amdgcn_sched_barrier(0);
      }
    });
    if (READ) {   // smaller tiles have fewer MFMAs than reads
#pragma unroll
      for (int q = MFMAS; q < READS; ++q) read_item(q, abuf, wbuf, ks, r);
    }
  }

  // KIND 0 loads stage kt + AHEAD, 1 that stage as the last, 2 nothing, 3 is the last step.
  // (ac, an, ap: places of A's stages kt, kt + 1 and kt - 1; wc, wx: of W's kt and kt + 1.)
  template <int KIND>
  __device__ __forceinline__ void step(int kt, int ac, int an, int ap, int wc, int wx) {
    constexpr int LOAD = KIND == 0 ? 1 : KIND == 1 ? 2 : 0;
    substep<true, LOAD>(0, ac, wc, 2, 2, kt + AHEAD, ap, 0, A_DMA / 2);
    substep<true, LOAD>(1, ac, wc, 3, 3, kt + AHEAD, ap, A_DMA / 2, A_DMA);
    // behind stage kt + 1 come those up to kt + AHEAD - 1 and A's of kt + AHEAD
    if constexpr (KIND < 2) wait_vmcnt<(AHEAD - 2) * DMA + A_DMA>();
    else wait_vmcnt<0>();
    if (KIND == 2 && tail && kt + 2 == KT) clear_tail(an);
    wait_lgkm_mem();
    __syncthreads();
    substep<KIND != 3, LOAD>(2, an, wx, 0, 0, kt + AHEAD, wc, A_DMA, A_DMA + W_DMA / 2);
    substep<KIND != 3, LOAD>(3, an, wx, 1, 1, kt + AHEAD, wc, A_DMA + W_DMA / 2, DMA);
  }

  // The whole sum.  Behind it every wave has passed the last barrier, but its last
  // fragments may still be on their way from LDS.
  __device__ __forceinline__ void run() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = i32x16{};
    if (KT == 0) return;
    const int ahead = min(AHEAD, KT);
#pragma unroll 1
    for (int s = 0; s < ahead; ++s) {
#pragma unroll
      for (int d = 0; d < DMA; ++d) dma_item<true>(d, s, s);
    }
    if (KT >= AHEAD) wait_vmcnt<(AHEAD - 1) * DMA>();
    else wait_vmcnt<0>();
    if (tail && KT == 1) clear_tail(0);
    wait_lgkm_mem();
    __syncthreads();
#pragma unroll
    for (int q = 0; q < READS; ++q) read_item(q, 0, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < READS; ++q) read_item(q, 0, 0, 1, 1);
    int kt = 0, ac = 0, an = 1, ap = AHEAD, wc = 0, wx = 1;
    auto turn = [&] {
      ++kt;
      ap = ac;
      ac = an;
      an = an == AHEAD ? 0 : an + 1;
      wc = wx;
      wx = wx + 1 == AHEAD ? 0 : wx + 1;
    };
    for (; kt + AHEAD + 1 < KT; turn()) step<0>(kt, ac, an, ap, wc, wx);
    if (kt + AHEAD < KT) {
      step<1>(kt, ac, an, ap, wc, wx);
      turn();
    }
    for (; kt + 1 < KT; turn()) step<2>(kt, ac, an, ap, wc, wx);
    step<3>(kt, ac, an, ap, wc, wx);
  }
};

}  // namespace fm
