// fm_i8.hip -- rows in 8 bits with a scale each, and their products with 8-bit
// weights that have a scale for each output channel.
#include <algorithm>
#include <cstdlib>

#include "fm_act.hpp"
#include "fm_i8_tile.hpp"
#include "fm_layer_norm.hpp"
#include "fm_sched.hpp"

namespace fm {
namespace {

// -- rows to 8 bits ------------------------------------------------------------

constexpr int kQuantLanes = 256;
constexpr int kQuantHeld = 4;   // chunks of eight elements that a lane keeps between its passes

struct QuantArgs {
  const void* x;
  char* q;
  float* scale;
  int64_t M, N;
};

// One row a block: the largest magnitude, then the values, from registers as far as
// they fit and read again beyond.
template <typename E>
__global__ __launch_bounds__(kQuantLanes) void quant_rows(const QuantArgs a) {
  using T = typename Elem<E>::type;
  __shared__ uint32_t s_top[kQuantLanes / 64];
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= a.M) return;
  const T* x = static_cast<const T*>(a.x) + row * a.N;
  f32x4 v[kQuantHeld][2];
  uint32_t top = 0;
  auto join = [&](const f32x4 (&w)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, magnitude(w[h][i]));
  };
#pragma unroll
  for (int c = 0; c < kQuantHeld; ++c) {
    const int64_t e = (int64_t)(c * kQuantLanes + threadIdx.x) * 8;
    if (e < a.N) {
      load8<E>(x + e, v[c]);
      join(v[c]);
    }
  }
  const int64_t rest = (int64_t)(kQuantHeld * kQuantLanes + threadIdx.x) * 8;
  for (int64_t e = rest; e < a.N; e += kQuantLanes * 8) {
    f32x4 w[2];
    load8<E>(x + e, w);
    join(w);
  }
  const RowQuant r = row_quant(row_umax<kQuantLanes>(top, s_top));
  if (threadIdx.x == 0) a.scale[row] = r.scale;
  char* q = a.q + row * a.N;
  auto put = [&](int64_t e, const f32x4 (&w)[2]) {
    *reinterpret_cast<u32x2*>(q + e) = u32x2{quant4(w[0], r), quant4(w[1], r)};
  };
#pragma unroll
  for (int c = 0; c < kQuantHeld; ++c) {
    const int64_t e = (int64_t)(c * kQuantLanes + threadIdx.x) * 8;
    if (e < a.N) put(e, v[c]);
  }
  for (int64_t e = rest; e < a.N; e += kQuantLanes * 8) {
    f32x4 w[2];
    load8<E>(x + e, w);
    put(e, w);
  }
}

fm_status_t check_quant(fm_dtype_t dt, int64_t M, int64_t N) {
  if (dt != FM_F16 && dt != FM_BF16 && dt != FM_F32) return FM_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || N % 8) return FM_ERR_INVALID_ARG;
  if (M >= (1ll << 31) || N >= (1ll << 31)) return FM_ERR_UNSUPPORTED;
  return FM_OK;
}

void launch_quant(fm_dtype_t dt, const QuantArgs& a, hipStream_t stream) {
  const int64_t x = std::min<int64_t>(a.M, 1 << 20);
  const dim3 grid((unsigned)x, (unsigned)cdiv(a.M, x)), lanes(kQuantLanes);
  if (dt == FM_F16) hipLaunchKernelGGL(quant_rows<F16>, grid, lanes, 0, stream, a);
  else if (dt == FM_BF16) hipLaunchKernelGGL(quant_rows<BF16>, grid, lanes, 0, stream, a);
  else hipLaunchKernelGGL(quant_rows<F32>, grid, lanes, 0, stream, a);
}

// -- products --------------------------------------------------------------------

struct I8Args {
  const char *A, *W;                // [M, K], [N, K]
  const float *a_scale, *w_scale;   // [M], [N]
  const void* bias;                 // [N] or NULL
  char* C;                          // [M, N]
  int64_t M, N, K;
  int act;
  int tiles_m, tiles_n, group_m;
};

// Eight results of a row: the sums' scales, bias, activation, rounding.
struct Columns {
  f32x4 scale[2], bias[2];
};

template <typename O>
__device__ __forceinline__ void finish8(const I8Args& a, const Columns& c, const i32x4 (&sum)[2], float sa,
                                        int64_t at) {
  f32x4 v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[h][i] = (float)sum[h][i] * (sa * c.scale[h][i]) + c.bias[h][i];
  activate_all(v, a.act);
  store8<O>(reinterpret_cast<typename Elem<O>::type*>(a.C) + at, v);
}

// A persistent grid of macro-tiles (fm_sched.hpp's order).  The epilogue turns each
// 32-row block of a wave around through its own part of LDS, finished and rounded, so
// that stores cover whole pieces of rows.
template <typename E, typename O, int BM, int BN, int AHEAD>
__global__ __launch_bounds__(256, 1) void gemm_i8_tiles(const I8Args a) {
  using Tile = I8Tile<BM, BN, AHEAD>;
  constexpr int PITCH = Tile::WN * 4 + 16, LPR = Tile::WN / 8;   // staged row, lanes of one
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
#pragma unroll 2
      for (int q = 0; q < 32 * LPR / 64; ++q) {
        const int k = q * 64 + t.lane, y = k / LPR, x = k % LPR * 8;
        const int m = t.wm * Tile::WM + 32 * i + y, n = t.wn * Tile::WN + x;
        if (m < rows && n < cols) {
          const i32x4* p = reinterpret_cast<const i32x4*>(stage + y * PITCH + x * 4);
          const i32x4 sum[2] = {p[0], p[1]};
          Columns c;
          load8<F32>(s_scale + n, c.scale);
          load8<F32>(s_bias + n, c.bias);
          finish8<O>(a, c, sum, s_row[m], (m0 + m) * a.N + n0 + n);
        }
      }
      wave_lds_sync();
    }
    __syncthreads();   // before the next tile's loads land in LDS
  }
}

// A sum of K products of bytes fits 32 bits up to here (127 * 128 * K, and -128 may
// stand in a caller's own codes: 2^14 K < 2^31).
constexpr int64_t kI8MaxK = (1ll << 17) - 16;
constexpr int64_t kI8MaxDim = 1ll << 22;

fm_status_t check_i8(fm_dtype_t dt, fm_dtype_t c, int64_t M, int64_t N, int64_t K, fm_act_t act) {
  if ((dt != FM_F16 && dt != FM_BF16) || (c != dt && c != FM_F32)) return FM_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K < 0 || N % 8 || K % 16) return FM_ERR_INVALID_ARG;
  if ((int)act < FM_ACT_NONE || (int)act > FM_ACT_SILU) return FM_ERR_INVALID_ARG;
  if (M >= kI8MaxDim || N >= kI8MaxDim || K > kI8MaxK) return FM_ERR_UNSUPPORTED;
  return FM_OK;
}

template <typename E, typename O, int BM, int BN, int AHEAD>
void launch_tiles(I8Args a, hipStream_t stream) {
  a.tiles_m = (int)cdiv(a.M, BM);
  a.tiles_n = (int)cdiv(a.N, BN);
  a.group_m = std::min(8, a.tiles_m);
  const int64_t total = (int64_t)a.tiles_m * a.tiles_n;
  hipLaunchKernelGGL((gemm_i8_tiles<E, O, BM, BN, AHEAD>), dim3((unsigned)std::min<int64_t>(total, device_cu_count() * std::min<int>(3, 160 * 1024 / I8Tile<BM, BN, AHEAD>::LDS_BYTES))),
                     dim3(256), 0, stream, a);
}

template <typename E, typename O>
void launch_gemm(const I8Args& a, hipStream_t stream) {
  const char* v = std::getenv("FM_I8");
  const int k = v ? std::atoi(v) : 0;
  if (k == 1) return launch_tiles<E, O, 256, 256, 2>(a, stream);
  if (k == 2) return launch_tiles<E, O, 256, 192, 2>(a, stream);
  if (k == 3) return launch_tiles<E, O, 256, 128, 2>(a, stream);
  if (k == 4) return launch_tiles<E, O, 192, 192, 2>(a, stream);
  if (k == 5) return launch_tiles<E, O, 128, 128, 2>(a, stream);
  if (k == 6) return launch_tiles<E, O, 128, 64, 3>(a, stream);
  if (k == 7) return launch_tiles<E, O, 64, 64, 2>(a, stream);
  if (k == 8) return launch_tiles<E, O, 192, 256, 2>(a, stream);
  if (k == 9) return launch_tiles<E, O, 128, 192, 3>(a, stream);
  if (k == 10) return launch_tiles<E, O, 128, 128, 4>(a, stream);
  if (k == 11) return launch_tiles<E, O, 64, 64, 4>(a, stream);
  if (k == 12) return launch_tiles<E, O, 64, 128, 3>(a, stream);
  return launch_tiles<E, O, 64, 64, 2>(a, stream);
}

void launch_gemm_types(fm_dtype_t dt, fm_dtype_t c, const I8Args& a, hipStream_t stream) {
  if (dt == FM_F16) {
    if (c == FM_F32) launch_gemm<F16, F32>(a, stream);
    else launch_gemm<F16, F16>(a, stream);
  } else {
    if (c == FM_F32) launch_gemm<BF16, F32>(a, stream);
    else launch_gemm<BF16, BF16>(a, stream);
  }
}

int64_t codes_bytes(int64_t M, int64_t K) { return cdiv(M * K, 256) * 256; }

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" fm_status_t fm_quant_i8(fm_dtype_t dt, int64_t M, int64_t N, const void* x, int8_t* q,
                                   float* scale, hipStream_t stream) {
  const fm_status_t st = check_quant(dt, M, N);
  if (st != FM_OK) return st;
  if (M == 0) return FM_OK;
  if (!scale || !aligned4(scale)) return FM_ERR_INVALID_ARG;
  if (N > 0 && (!x || !q)) return FM_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q)) return FM_ERR_INVALID_ARG;
  launch_quant(dt, {x, reinterpret_cast<char*>(q), scale, M, N}, stream);
  return launch_status();
}

extern "C" fm_status_t fm_gemm_i8(fm_dtype_t dt, fm_dtype_t c, int64_t M, int64_t N, int64_t K,
                                  const int8_t* A, const float* a_scale, const int8_t* W,
                                  const float* w_scale, const void* bias, fm_act_t act, void* C,
                                  hipStream_t stream) {
  const fm_status_t st = check_i8(dt, c, M, N, K, act);
  if (st != FM_OK) return st;
  if (M == 0 || N == 0) return FM_OK;
  if (!a_scale || !w_scale || !C || (K > 0 && (!A || !W))) return FM_ERR_INVALID_ARG;
  for (const void* p : {(const void*)A, (const void*)W, (const void*)w_scale, bias, (const void*)C})
    if (!aligned16(p)) return FM_ERR_INVALID_ARG;
  if (!aligned4(a_scale)) return FM_ERR_INVALID_ARG;
  launch_gemm_types(dt, c, {(const char*)A, (const char*)W, a_scale, w_scale, bias, (char*)C, M, N, K, (int)act},
                    stream);
  return launch_status();
}

extern "C" size_t fm_linear_i8_workspace_bytes(int64_t M, int64_t K) {
  if (M < 0 || K < 0 || K % 16 || M >= kI8MaxDim || K > kI8MaxK) return 0;
  return std::max<size_t>((size_t)codes_bytes(M, K) + (size_t)M * 4, 256);
}

extern "C" fm_status_t fm_linear_i8(fm_dtype_t dt, fm_dtype_t c, int64_t M, int64_t N, int64_t K,
                                    const void* X, const int8_t* W, const float* w_scale,
                                    const void* bias, fm_act_t act, void* C, void* ws,
                                    size_t ws_bytes, hipStream_t stream) {
  const fm_status_t st = check_i8(dt, c, M, N, K, act);
  if (st != FM_OK) return st;
  if (M == 0 || N == 0) return FM_OK;
  if (!w_scale || !C || (K > 0 && (!X || !W))) return FM_ERR_INVALID_ARG;
  for (const void* p : {X, (const void*)W, (const void*)w_scale, bias, (const void*)C, (const void*)ws})
    if (!aligned16(p)) return FM_ERR_INVALID_ARG;
  if (!ws || ws_bytes < fm_linear_i8_workspace_bytes(M, K)) return FM_ERR_INVALID_ARG;
  char* codes = static_cast<char*>(ws);
  float* scale = reinterpret_cast<float*>(codes + codes_bytes(M, K));
  launch_quant(dt, {X, codes, scale, M, K}, stream);
  launch_gemm_types(dt, c, {codes, (const char*)W, scale, w_scale, bias, (char*)C, M, N, K, (int)act}, stream);
  return launch_status();
}
