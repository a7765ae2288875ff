// fm_dropout.hip -- dropout of a matrix; forward and backward are the same pass.
//
// A lane takes eight elements, which share one counter.
#include "fm_dropout.hpp"
#include "fm_norm.hpp"

namespace fm {
namespace {

constexpr int64_t kDropGridX = 1 << 20;
constexpr int kDropThreads = 256;
constexpr int kDropUnroll = 2;

struct DropArgs {
  const void* x;
  void* y;
  int64_t chunks;     // M * N / 8
  uint32_t per_row;   // N / 8
  Dropout d;
};

template <typename E>
__global__ __launch_bounds__(kDropThreads) void dropout_rows(const DropArgs a) {
  using T = typename Elem<E>::type;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t first = block * (kDropThreads * kDropUnroll);
  // row and column of the block's first chunk are scalars; a lane's from there in 32 bits
  const int64_t row0 = first / a.per_row;
  const uint32_t col0 = (uint32_t)(first - row0 * a.per_row);
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  f32x4 v[kDropUnroll][2];
#pragma unroll
  for (int u = 0; u < kDropUnroll; ++u) {
    const int64_t at = first + u * kDropThreads + threadIdx.x;
    if (at < a.chunks) {
      v[u][0] = load4<E>(x + at * 8);
      v[u][1] = load4<E>(x + at * 8 + 4);
    }
  }
  Philox p = {};
  if (a.d.rng) p = philox_of(a.d);
#pragma unroll
  for (int u = 0; u < kDropUnroll; ++u) {
    const int64_t at = first + u * kDropThreads + threadIdx.x;
    if (at >= a.chunks) continue;
    if (a.d.rng) {
      const uint32_t c = col0 + u * kDropThreads + threadIdx.x, r = c / a.per_row;
      const u32x4 w = philox(p, a.d.block + (c - r * a.per_row), a.d.row + (uint32_t)row0 + r);
      v[u][0] = drop4(v[u][0], w[0], w[1], a.d);
      v[u][1] = drop4(v[u][1], w[2], w[3], a.d);
    }
    store4<E>(y + at * 8, v[u][0]);
    store4<E>(y + at * 8 + 4, v[u][1]);
  }
}

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" fm_status_t fm_dropout(fm_dtype_t dt, int64_t M, int64_t N, const void* x, float p,
                                  const uint64_t* rng, int64_t draw, int64_t row_begin,
                                  int64_t col_begin, void* y, hipStream_t stream) {
  if (dt != FM_F16 && dt != FM_BF16 && dt != FM_F32) return FM_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || N % 8) return FM_ERR_INVALID_ARG;
  if (M >= (1ll << 31) || N >= (1ll << 31)) return FM_ERR_UNSUPPORTED;
  const fm_status_t st = check_dropout(p, rng, M, row_begin, N, col_begin);
  if (st != FM_OK) return st;
  if (M == 0 || N == 0) return FM_OK;
  if (!x || !y || !aligned16(x) || !aligned16(y)) return FM_ERR_INVALID_ARG;
  DropArgs a = {};
  a.x = x;
  a.y = y;
  a.per_row = (uint32_t)(N / 8);
  a.chunks = M * (N / 8);
  a.d = make_dropout(p, rng, draw, row_begin, col_begin);
  const int64_t blocks = cdiv(a.chunks, kDropThreads * kDropUnroll);
  const int64_t gx = blocks < kDropGridX ? blocks : kDropGridX, gy = cdiv(blocks, gx);
  if (gy > 65535) return FM_ERR_UNSUPPORTED;   // 2^45 elements
  const dim3 grid((unsigned)gx, (unsigned)gy), lanes(kDropThreads);
  if (dt == FM_F16) hipLaunchKernelGGL(dropout_rows<F16>, grid, lanes, 0, stream, a);
  else if (dt == FM_BF16) hipLaunchKernelGGL(dropout_rows<BF16>, grid, lanes, 0, stream, a);
  else hipLaunchKernelGGL(dropout_rows<F32>, grid, lanes, 0, stream, a);
  return launch_status();
}
