// fm_i8_tiles.hip -- 8-bit products of many rows, on the macro-tiles of fm_i8_tile.hpp.
//
// 4096 x 12288 x 6144 245 to 260 us by the card, 2.4 to 2.5 POP/s: the matrix cores are busy in
// 65% of the cycles at the 1.7 GHz that the power limit leaves (a loop on registers alone
// reaches 3.5 POP/s).
#include <algorithm>

#include "fm_i8.hpp"
#include "fm_i8_choice.hpp"
#include "fm_i8_tile.hpp"
#include "fm_sched.hpp"

namespace fm {
namespace {

struct TileArgs : I8Args {
  int tiles_m, tiles_n, group_m;
};

// A lane's eight columns.
struct Columns {
  f32x4 scale[2], bias[2];
};

// A persistent grid of macro-tiles (fm_sched.hpp's order).  The epilogue turns the sums of
// each 32-row block of a wave around through its own part of LDS, so that a lane finishes
// eight neighbouring columns of several rows and stores cover whole pieces of rows.
template <typename E, typename O, int BM, int BN, int AHEAD>
__global__ __launch_bounds__(256, 1) void gemm_i8_tiles(const TileArgs a) {
  using Tile = I8Tile<BM, BN, AHEAD>;
  // bytes of a staged row, and lanes that take one, eight columns each (rounded up, so that
  // a lane keeps its columns)
  constexpr int PITCH = Tile::WN * 4 + 16, LPR = Tile::WN == 96 ? 16 : Tile::WN / 8;
  static_assert(4 * 32 * PITCH + (BM + 2 * BN) * 4 <= Tile::LDS_BYTES && 32 * LPR % 64 == 0, "staging");
  __shared__ __attribute__((aligned(16))) char smem[Tile::LDS_BYTES];
  Tile t(smem, a.K);
  const int r32 = t.lane & 31, hi = t.lane >> 5;
  char* stage = smem + t.w * 32 * PITCH;
  float* s_row = reinterpret_cast<float*>(smem + 4 * 32 * PITCH);
  float *s_scale = s_row + BM, *s_bias = s_scale + BN;
  const int total = a.tiles_m * a.tiles_n;
  for (int L = xcd_slot(blockIdx.x, gridDim.x); L < total; L += gridDim.x) {
    int tm, tn;
    band_coords(L, a.tiles_m, a.tiles_n, a.group_m, tm, tn);
    // the operands' bases must sit in scalar registers for the loads
    tm = __builtin_amdgcn_readfirstlane(tm);
    tn = __builtin_amdgcn_readfirstlane(tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int rows = (int)min((int64_t)BM, a.M - m0), cols = (int)min((int64_t)BN, a.N - n0);
    t.set_tile(a.A + m0 * a.K, rows, a.W + n0 * a.K, cols, a.K);
    // the tile's scales and biases are on their way during the sum
    const int ir = min((int)threadIdx.x, rows - 1), ic = min((int)threadIdx.x, cols - 1);
    const float row_scale = a.a_scale[m0 + ir], col_scale = a.w_scale[n0 + ic];
    const float col_bias = a.bias ? (float)static_cast<const typename Elem<E>::type*>(a.bias)[n0 + ic] : 0.f;
    t.run();
    __syncthreads();   // every wave has read its last fragments
    if (threadIdx.x < BM) s_row[threadIdx.x] = row_scale;
    if (threadIdx.x < BN) {
      s_scale[threadIdx.x] = col_scale;
      s_bias[threadIdx.x] = col_bias;
    }
    __syncthreads();
    const int x = t.lane % LPR * 8, n = t.wn * Tile::WN + x;
    const bool mine = x < Tile::WN && n < cols;
    Columns c = {};
    if (mine) {
      load8<F32>(s_scale + n, c.scale);
      load8<F32>(s_bias + n, c.bias);
    }
#pragma unroll
    for (int i = 0; i < Tile::FM; ++i) {
      asm volatile("" ::: "memory");   // one block's registers after another's
#pragma unroll
      for (int j = 0; j < Tile::FN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const i32x16& s = t.acc[i][j];
          *reinterpret_cast<i32x4*>(stage + r32 * PITCH + (32 * j + 8 * r + 4 * hi) * 4) =
              i32x4{s[4 * r], s[4 * r + 1], s[4 * r + 2], s[4 * r + 3]};
        }
      wave_lds_sync();
      // several rows' reads first, then their arithmetic: one wave a SIMD has no other to
      // cover LDS's latency
      constexpr int ROWS = 32 * LPR / 64, G = ROWS < 4 ? ROWS : 4;
#pragma unroll 1
      for (int q = 0; q < ROWS; q += G) {
        f32x4 v[2 * G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int y = (q + g) * (64 / LPR) + t.lane / LPR;
          const i32x4* p = reinterpret_cast<const i32x4*>(stage + y * PITCH + min(x, Tile::WN - 8) * 4);
          const float sa = s_row[t.wm * Tile::WM + 32 * i + y];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) v[2 * g + h][k] = (float)p[h][k] * (sa * c.scale[h][k]) + c.bias[h][k];
        }
        activate_all(v, a.act);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int m = t.wm * Tile::WM + 32 * i + (q + g) * (64 / LPR) + t.lane / LPR;
          if (m < rows && mine) {
            const f32x4 o[2] = {v[2 * g], v[2 * g + 1]};
            store8<O>(reinterpret_cast<typename Elem<O>::type*>(a.C) + (m0 + m) * a.N + n0 + n, o);
          }
        }
      }
      wave_lds_sync();
    }
    __syncthreads();   // before the next tile's loads land in LDS
  }
}

template <typename E, typename O, int BM, int BN, int AHEAD>
void launch_grid(const I8Args& g, int resident, hipStream_t stream) {
  TileArgs a = {g};
  a.tiles_m = (int)cdiv(a.M, BM);
  a.tiles_n = (int)cdiv(a.N, BN);
  a.group_m = std::min(8, a.tiles_m);
  const int64_t total = (int64_t)a.tiles_m * a.tiles_n, most = (int64_t)device_cu_count() * resident;
  hipLaunchKernelGGL((gemm_i8_tiles<E, O, BM, BN, AHEAD>), dim3((unsigned)std::min(total, most)), dim3(256), 0,
                     stream, a);
}

template <typename E, typename O>
void launch_types(const I8Args& a, hipStream_t stream) {
  const int i = choose_tile(a.M, a.N, a.K, device_cu_count()), r = kTileChoices[i].resident;
  switch (i) {
    case 0: return launch_grid<E, O, 64, 64, 4>(a, r, stream);
    case 1: return launch_grid<E, O, 64, 128, 3>(a, r, stream);
    case 2: return launch_grid<E, O, 128, 128, 4>(a, r, stream);
    case 3: return launch_grid<E, O, 128, 192, 3>(a, r, stream);
    case 4: return launch_grid<E, O, 256, 128, 2>(a, r, stream);
    case 5: return launch_grid<E, O, 256, 192, 2>(a, r, stream);
    default: return launch_grid<E, O, 256, 256, 2>(a, r, stream);
  }
}

}  // namespace

void launch_i8_tiles(const I8Args& a, hipStream_t stream) {
  if (a.dt == FM_F16) {
    if (a.c == FM_F32) launch_types<F16, F32>(a, stream);
    else launch_types<F16, F16>(a, stream);
  } else {
    if (a.c == FM_F32) launch_types<BF16, F32>(a, stream);
    else launch_types<BF16, BF16>(a, stream);
  }
}

}  // namespace fm
