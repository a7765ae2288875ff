// fm_i8_tile.hpp -- macro-tiles of 8-bit products on v_mfma_i32_32x32x32_i8.
//
// Four waves, 2 x 2 over a BM x BN tile of C = A W^T; both operands lie with k in a row,
// so one layout and one read serve both.  A K step is 128 bytes of every row; LDS holds
// NSTAGE steps of [A rows | W rows], filled by direct-to-LDS loads.  A step has four
// sub-steps of one instruction depth (32).  The fragments of a sub-step are read two
// sub-steps ahead, four register slots in turn:
//   sub-steps 0, 1  MFMAs, reading sub-steps 2, 3 of this stage;
//   wait, barrier   the next stage has landed, this one is drained;
//   sub-steps 2, 3  MFMAs, reading sub-steps 0, 1 of the next stage, and the loads of
//                   stage kt + NSTAGE into this one's place.
// One memory operation follows each MFMA (sched_barrier keeps the order), so that the
// matrix cores do not wait for a burst of them.  A 256 x 256 step is 64 MFMAs of 32
// cycles a wave on 32 LDS reads: LDS is busy for half of that time.
//
// 16-byte chunk c of row m is stored at chunk c ^ ((m ^ m >> 3) & 7), which spreads the
// reads of eight rows over all banks; the loads realise it by which chunk a lane fetches.
// The first MFMA operand is W, so lane l holds row l % 32 of C and, for item 4 r + q,
// column 8 r + 4 (l / 32) + q: runs of four columns.
#pragma once

#include "fm_tile.hpp"

namespace fm {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kI8Step = 128;   // bytes of k in a stage

template <int BM, int BN, int NSTAGE>
struct I8Tile {
  static constexpr int WM = BM / 2, WN = BN / 2;
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int STAGE = (BM + BN) * kI8Step, W_AT = BM * kI8Step;
  static constexpr int A_DMA = BM / 32, DMA = (BM + BN) / 32;   // loads of a wave, 8 rows each
  static constexpr int READS = FM + FN, MFMAS = FM * FN;
  static constexpr int LDS_BYTES = NSTAGE * STAGE;
  static_assert(BM % 64 == 0 && BN % 64 == 0 && LDS_BYTES <= 160 * 1024, "tile size");

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
    return buf * STAGE + (d < A_DMA ? w * (BM / 4) * kI8Step + d * 1024
                                    : W_AT + w * (BN / 4) * kI8Step + (d - A_DMA) * 1024);
  }
  __device__ __forceinline__ void dma_item(int d, int kt, int buf) {
    dma16(off[d], (d < A_DMA ? a_base : w_base) + (int64_t)kt * kI8Step, lds0 + dma_at(d, buf));
  }
  // A stage that may be the last step: a lane whose chunk lies past K loads its row's first
  // chunk of the step instead.
  __device__ __forceinline__ void dma_last(int kt, int buf, bool last = true) {
#pragma unroll
    for (int d = 0; d < DMA; ++d) {
      const uint32_t c = dma_chunk(d) * 16;
      dma16(last && tail && c >= (uint32_t)tail ? off[d] - c : off[d],
            (d < A_DMA ? a_base : w_base) + (int64_t)kt * kI8Step, lds0 + dma_at(d, buf));
    }
  }
  // Its chunks past K count as zeros: A's are cleared, once this wave's loads have landed.
  __device__ __forceinline__ void clear_tail(int buf) {
#pragma unroll
    for (int d = 0; d < A_DMA; ++d)
      if (dma_chunk(d) * 16 >= tail)
        *reinterpret_cast<u32x4*>(smem + dma_at(d, buf) + lane * 16) = u32x4{0, 0, 0, 0};
  }

  __device__ __forceinline__ void read_item(int q, int buf, int ks, int slot) {
    const char* s = smem + buf * STAGE;
    // A and W in turn, as the first MFMAs need them
    const int pairs = 2 * (FM < FN ? FM : FN);
    const bool is_a = q < pairs ? q % 2 == 0 : FM > FN;
    const int j = q < pairs ? q / 2 : q - pairs / 2;
    if (is_a) fa[slot][j] = *reinterpret_cast<const i32x4*>(s + ra[ks][j & 1] + j * 32 * kI8Step);
    else fw[slot][j] = *reinterpret_cast<const i32x4*>(s + rw[ks][j & 1] + j * 32 * kI8Step);
  }

  // MFMAs on slot `m`; reads of sub-step ks of buffer nbuf into slot r; loads d0 .. d1 - 1
  // of stage dk into buffer dbuf.
  template <bool READ, bool LOAD>
  __device__ __forceinline__ void substep(int m, int nbuf, int ks, int r, int dk, int dbuf, int d0, int d1) {
    static_for<MFMAS>([&](auto qc) {
      constexpr int q = decltype(qc)::value;
      constexpr int i = q / FN, j = q % FN;
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[m][j], fa[m][i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (READ && q < READS) {
        read_item(q, nbuf, ks, r);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (LOAD && d0 + q < d1) {
        dma_item(d0 + q, dk, dbuf);
        __builtin_amdgcn_sched_barrier(0);
      }
    });
    if (READ) {   // smaller tiles have fewer MFMAs than memory operations
#pragma unroll
      for (int q = MFMAS; q < READS; ++q) read_item(q, nbuf, ks, r);
    }
    if (LOAD) {
#pragma unroll
      for (int d = d0 + MFMAS; d < d1; ++d) dma_item(d, dk, dbuf);
    }
  }

  // KIND 0 loads stage kt + NSTAGE, 1 that stage as the last, 2 nothing, 3 is the last step.
  template <int KIND>
  __device__ __forceinline__ void step(int kt, int cur, int nxt) {
    substep<true, false>(0, cur, 2, 2, 0, 0, 0, 0);
    substep<true, false>(1, cur, 3, 3, 0, 0, 0, 0);
    if constexpr (KIND < 2) wait_vmcnt<(NSTAGE - 2) * DMA>();
    else wait_vmcnt<0>();
    if (KIND == 2 && tail && kt + 2 == KT) clear_tail(nxt);
    wait_lgkm_mem();
    __syncthreads();
    if constexpr (KIND == 1) dma_last(kt + NSTAGE, cur);
    substep<KIND != 3, KIND == 0>(2, nxt, 0, 0, kt + NSTAGE, cur, 0, DMA / 2);
    substep<KIND != 3, KIND == 0>(3, nxt, 1, 1, kt + NSTAGE, cur, DMA / 2, DMA);
  }

  // The whole sum.  Behind it every wave has passed the last barrier, but may still
  // read no more than registers: LDS is free.
  __device__ __forceinline__ void run() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = i32x16{};
    if (KT == 0) return;
    const int ahead = min(NSTAGE, KT);
#pragma unroll 1
    for (int s = 0; s < ahead; ++s) dma_last(s, s, s + 1 == KT);
    if (KT >= NSTAGE) wait_vmcnt<(NSTAGE - 1) * DMA>();
    else wait_vmcnt<0>();
    if (tail && KT == 1) clear_tail(0);
    wait_lgkm_mem();
    __syncthreads();
#pragma unroll
    for (int q = 0; q < READS; ++q) read_item(q, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < READS; ++q) read_item(q, 0, 1, 1);
    int kt = 0, cur = 0;
    auto next = [&](int b) { return b + 1 == NSTAGE ? 0 : b + 1; };
    for (; kt + NSTAGE + 1 < KT; ++kt) {
      step<0>(kt, cur, next(cur));
      cur = next(cur);
    }
    if (kt + NSTAGE < KT) {
      step<1>(kt, cur, next(cur));
      cur = next(cur);
      ++kt;
    }
    for (; kt + 1 < KT; ++kt) {
      step<2>(kt, cur, next(cur));
      cur = next(cur);
    }
    step<3>(kt, cur, next(cur));
  }
};

}  // namespace fm
