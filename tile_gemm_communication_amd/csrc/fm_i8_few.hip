// fm_i8_few.hip -- 8-bit products of few rows: the weights stream through once.
//
// A block takes 8 C8 columns, as many as make one block a compute unit, and all rows of
// x; its waves share the sum over k, wave w the 128-byte steps w, w + NWV, ...  Each wave
// keeps a ring of S steps in its own part of LDS, filled by direct-to-LDS loads of eight
// whole 128-byte pieces of rows, so that S - 1 steps are in flight without a register or
// a barrier; the waves' sums (whole numbers: exact in any order) meet in LDS at the end.
// Bound by the weights' bytes: 1 x 6144 x 12288 (k x columns) 12.3 us, 6.1 TB/s, with the
// weights in the Infinity Cache, 14.8 from HBM; 45 x 12288 x 6144 14.5 and 21.8, where a wave's
// loads of x and W return in one order (macro-tiles took 24.8 and the k loop's latency).
//
// v_mfma_i32_16x16x64_i8: lane l holds 16 bytes of row l % 16 from k = 16 (l / 16) on of
// either operand, and of the result column l % 16, rows 4 (l / 16) .. + 3.  W comes first,
// so a lane has four neighbouring columns of one row of C.
#include <algorithm>

#include "fm_i8.hpp"
#include "fm_i8_tile.hpp"
#include "fm_sched.hpp"

namespace fm {
namespace {

constexpr int kFewLds = 152 * 1024;

// What a block quantises for itself: at most 32 pieces of 512 values (four a wave; 17 KiB
// of codes).  A wave's pieces come one after another (each load has its own branch, and is
// waited for at its end), and the first weights' loads go out behind the last.  1 x 12288 x
// 6144: 14.7 us, the product alone 12.3, with a launch of its own before it 17.6; of 96 pieces
// (8 x 6144) it would take 23, against 15.9.
constexpr int kQuantPiece = 512, kQuantHeld = 4, kQuantMost = 8 * kQuantHeld;
constexpr int kFewQuantRows = 8, kFewCodes = 17 * 1024;

// X8, C8: eights of x's rows and of columns.  QUANT: the block quantises 16-bit rows first
// and keeps the codes; else codes are streamed beside the weights.
template <int X8, int C8, bool QUANT>
struct FewShape {
  static constexpr int X_LOADS = QUANT ? 0 : X8, LOADS = X_LOADS + C8;   // 1 KiB each
  static constexpr int NWV = LOADS <= 9 ? 8 : 4;
  static constexpr int X_BYTES = QUANT ? kFewCodes : 0;
  static constexpr int FIT = (kFewLds - X_BYTES) / (NWV * LOADS * 1024);
  static constexpr int S = FIT < 4 ? FIT : 4;
  static constexpr int FM = (X8 + 1) / 2, FN = (C8 + 1) / 2;   // 16 x 16 results
  static constexpr int RING = NWV * S * LOADS * 1024, SUMS = NWV * FM * FN * 1024;
  static constexpr int LDS = RING > SUMS ? RING : SUMS;
  static_assert(S >= 2, "two steps in flight");
};

__host__ __device__ inline int code_pitch(int K) { return (K + 255) / 256 * 256 + 64; }

// Four results of a row from column n on.
struct Finish4 {
  f32x4 scale, bias;
};

__device__ __forceinline__ Finish4 columns4(const I8Args& a, int64_t n) {
  Finish4 f = {*reinterpret_cast<const f32x4*>(a.w_scale + n), {0.f, 0.f, 0.f, 0.f}};
  if (a.bias)
    f.bias = a.dt == FM_F16 ? load4<F16>(static_cast<const _Float16*>(a.bias) + n)
                            : load4<BF16>(static_cast<const __bf16*>(a.bias) + n);
  return f;
}

__device__ __forceinline__ void store_row4(const I8Args& a, const Finish4& f, i32x4 sum, float sa, int64_t at) {
  f32x4 v[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[0][i] = (float)sum[i] * (sa * f.scale[i]) + f.bias[i];
  activate_all(v, a.act);
  if (a.c == FM_F32) store4<F32>(reinterpret_cast<float*>(a.C) + at, v[0]);
  else if (a.c == FM_F16) store4<F16>(reinterpret_cast<_Float16*>(a.C) + at, v[0]);
  else store4<BF16>(reinterpret_cast<__bf16*>(a.C) + at, v[0]);
}

// The rows of x as codes at `codes`, zeros from K to the end of the last step, and their
// scales.  x's loads come first, then start() (the weights' first loads, in flight during
// the arithmetic), so that x does not wait for the weights.  Ends behind a barrier.
template <class F>
__device__ __forceinline__ void quantise_rows(const I8Args& a, int w, int lane, int KT, char* codes,
                                              uint32_t* tops, float* scales, F&& start) {
  const int K = (int)a.K, M = (int)a.M, pieces = (K + kQuantPiece - 1) / kQuantPiece;
  const int total = M * pieces, pitch = code_pitch(K);
  u32x4 v[kQuantHeld];
#pragma unroll
  for (int i = 0; i < kQuantHeld; ++i) {
    const int g = i * 8 + w, row = g / pieces, e = (g - row * pieces) * kQuantPiece + lane * 8;
    v[i] = u32x4{0, 0, 0, 0};
    if (g < total && e < K) v[i] = *reinterpret_cast<const u32x4*>(a.A + ((int64_t)row * K + e) * 2);
  }
  start();
  auto widened = [&](const u32x4& r, int h) {
    const u32x2 p = {r[2 * h], r[2 * h + 1]};
    return a.dt == FM_F16 ? widen<F16>(__builtin_bit_cast(f16x4, p)) : widen<BF16>(__builtin_bit_cast(bf16x4, p));
  };
#pragma unroll
  for (int i = 0; i < kQuantHeld; ++i) {
    const int g = i * 8 + w;
    if (g >= total) break;
    uint32_t top = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 x = widened(v[i], h);
#pragma unroll
      for (int k = 0; k < 4; ++k) top = max(top, magnitude(x[k]));
    }
    top = group_umax<64>(top);
    if (lane == 0) tops[g] = top;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQuantHeld; ++i) {
    const int g = i * 8 + w, row = g / pieces, e = (g - row * pieces) * kQuantPiece + lane * 8;
    if (g >= total) break;
    const RowQuant r = row_quant(group_umax<64>(lane < pieces ? tops[row * pieces + lane] : 0u));
    if (e == 0) scales[row] = r.scale;
    if (e < KT * kI8Step)
      *reinterpret_cast<u32x2*>(codes + row * pitch + e) = u32x2{quant4(widened(v[i], 0), r), quant4(widened(v[i], 1), r)};
  }
  __syncthreads();
}

template <int X8, int C8, bool QUANT>
__global__ __launch_bounds__((64 * FewShape<X8, C8, QUANT>::NWV)) void gemm_i8_few(const I8Args a) {
  using Sh = FewShape<X8, C8, QUANT>;
  constexpr int NWV = Sh::NWV, S = Sh::S, LOADS = Sh::LOADS, XL = Sh::X_LOADS, FM = Sh::FM, FN = Sh::FN;
  static_assert(!QUANT || NWV == 8, "pieces go to eight waves");
  __shared__ __attribute__((aligned(16))) char smem[Sh::LDS + Sh::X_BYTES];
  __shared__ uint32_t s_tops[QUANT ? kQuantMost : 1];
  __shared__ float s_scale[kFewQuantRows];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int M = (int)a.M, K = (int)a.K;
  // where the blocks are a multiple of 8, an XCD takes neighbouring columns: 64 x 8192 x 8192
  // 14.3 us, dealt out in turn 21.0 (rows of W whose pitch is a power of two); 32 x 4096 x 4096
  // 5.5 and 6.7; 24 x 6144 x 6144 8.7 and 8.5; other numbers of blocks are dealt out in turn
  const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(xcd_slot(blockIdx.x, gridDim.x)) * (8 * C8);
  const int cols = (int)min((int64_t)(8 * C8), a.N - n0);
  const int KT = (K + kI8Step - 1) / kI8Step, tail = K % kI8Step;
  const char* const wt = a.W + n0 * K;
  char* const ring = smem + w * (S * LOADS * 1024);
  char* const codes = smem + Sh::LDS;
  const uint32_t ring0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)ring);

  // Load d: rows 8 d .. + 7 of x, then of W; rows past the last are read as the last.
  // Chunk c of row r lies at chunk c ^ swz_a(r).
  uint32_t off[LOADS];
#pragma unroll
  for (int d = 0; d < LOADS; ++d) {
    const int r = 8 * (d < XL ? d : d - XL) + (lane >> 3);
    off[d] = (uint32_t)min(r, (d < XL ? M : cols) - 1) * (uint32_t)K + (((lane & 7) ^ swz_a(r)) << 4);
  }
  auto load = [&](int kt, int slot) {
    const int64_t k = (int64_t)kt * kI8Step;
#pragma unroll
    for (int d = 0; d < LOADS; ++d) {
      // past K a lane loads its row's first chunk of the step instead
      const int c = (((lane & 7) ^ swz_a(8 * (d < XL ? d : d - XL) + (lane >> 3))) << 4);
      const uint32_t at = kt == KT - 1 && tail && c >= tail ? off[d] - c : off[d];
      dma16(at, (d < XL ? a.A : wt) + k, ring0 + (slot * LOADS + d) * 1024);
    }
  };
  // Fragment (16 rows from 16 g on, half h of the step) of x (from = 0) or W (from = XL)
  // in a slot; an odd number of eights reads its last one twice.
  auto fragment = [&](const char* s, int from, int eights, int g, int h) {
    const int r = lane & 15, e = 2 * g + (2 * g + 1 < eights ? r >> 3 : 0);
    const int row = 8 * e + (r & 7), c = (4 * h + (lane >> 4)) ^ swz_a(row);
    return *reinterpret_cast<const i32x4*>(s + (from + e) * 1024 + (r & 7) * kI8Step + c * 16);
  };

  i32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  const int steps = KT > w ? (KT - w + NWV - 1) / NWV : 0;   // this wave's
  auto start = [&] {
    for (int i = 0; i < S && i < steps; ++i) load(w + i * NWV, i);
  };
  if constexpr (QUANT) quantise_rows(a, w, lane, KT, codes, s_tops, s_scale, start);
  else start();
  int slot = 0;
  for (int i = 0; i < steps; ++i) {
    if (i + S <= steps) wait_vm_mem<(S - 1) * LOADS>();
    else wait_vm_mem<0>();
    const int kt = w + i * NWV;
    const char* s = ring + slot * LOADS * 1024;
    if (!QUANT && kt == KT - 1 && tail) {   // x counts as 0 past K
#pragma unroll
      for (int d = 0; d < XL; ++d)
        if (((((lane & 7) ^ swz_a(8 * d + (lane >> 3))) << 4)) >= tail)
          *reinterpret_cast<u32x4*>(const_cast<char*>(s) + d * 1024 + lane * 16) = u32x4{0, 0, 0, 0};
      wait_lgkm_mem();
    }
    i32x4 fx[2][FM], fw[2][FN];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int g = 0; g < FN; ++g) fw[h][g] = fragment(s, XL, C8, g, h);
#pragma unroll
      for (int g = 0; g < FM; ++g) {
        if constexpr (QUANT)
          fx[h][g] = *reinterpret_cast<const i32x4*>(codes + min(lane & 15, M - 1) * code_pitch(K) + kt * kI8Step +
                                                     (4 * h + (lane >> 4)) * 16);
        else fx[h][g] = fragment(s, 0, X8, g, h);
      }
    }
    wait_lgkm_mem();   // read before the slot is filled again
    if (i + S < steps) load(kt + S * NWV, slot);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[h][n], fx[h][m], acc[m][n], 0, 0, 0);
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  __syncthreads();
  i32x4* const sums = reinterpret_cast<i32x4*>(smem);
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int n = 0; n < FN; ++n) sums[((w * FM + m) * FN + n) * 64 + lane] = acc[m][n];
  __syncthreads();
  for (int t = threadIdx.x; t < FM * FN * 64; t += 64 * NWV) {
    const int l = t & 63, m = (t / 64 / FN) * 16 + (l & 15), n = (t / 64 % FN) * 16 + 4 * (l >> 4);
    if (m >= M || n >= cols) continue;
    i32x4 sum = sums[t];
#pragma unroll
    for (int o = 1; o < NWV; ++o) sum += sums[o * (FM * FN * 64) + t];
    store_row4(a, columns4(a, n0 + n), sum, QUANT ? s_scale[m % kFewQuantRows] : a.a_scale[m],
               (int64_t)m * a.N + n0 + n);
  }
}

// One block a unit up to 12288 columns on 256 units; a block takes most of a unit's LDS, so
// more columns take a second, partly filled round: 1 x 6144 x 12288 (k x columns) 12.3 us,
// 14336 17.1, 16384 21.0, 28672 35.5.
template <int X8, bool QUANT>
void launch_columns(const I8Args& a, hipStream_t stream) {
  const int64_t eights = a.N / 8, per = cdiv(eights, device_cu_count());
#define FM_FEW(C8)                                                                            \
  hipLaunchKernelGGL((gemm_i8_few<X8, C8, QUANT>), dim3((unsigned)cdiv(eights, C8)),              \
                     dim3(64 * FewShape<X8, C8, QUANT>::NWV), 0, stream, a)
  if (per <= 1) FM_FEW(1);
  else if (per <= 2) FM_FEW(2);
  else if (per <= 3) FM_FEW(3);
  else if (per <= 4) FM_FEW(4);
  else FM_FEW(6);
#undef FM_FEW
}

}  // namespace

void launch_i8_few(const I8Args& a, hipStream_t stream) {
  if (a.M <= 8) launch_columns<1, false>(a, stream);
  else if (a.M <= 16) launch_columns<2, false>(a, stream);
  else if (a.M <= 32) launch_columns<4, false>(a, stream);
  else if (a.M <= 48) launch_columns<6, false>(a, stream);
  else launch_columns<8, false>(a, stream);
}

bool i8_few_quantises(int64_t M, int64_t K) {
  return M <= kFewQuantRows && K > 0 && M * cdiv(K, kQuantPiece) <= kQuantMost &&
         M * code_pitch((int)K) <= kFewCodes;
}

void launch_i8_few_quant(const I8Args& a, hipStream_t stream) { launch_columns<1, true>(a, stream); }

}  // namespace fm
