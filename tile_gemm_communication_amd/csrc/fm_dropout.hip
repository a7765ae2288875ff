// fm_dropout.hip -- dropout of a matrix; forward and backward are the same pass.
//
// A lane takes eight elements, which share one counter, in one load and one store (two of
// each in 32 bits).  Bound by the bytes: 16384 x 12288 bf16 131 us, 6.1 TB/s (two or four
// chunks a lane: 140, 147); 4096 x 6144 bf16 19.5 us; 61 x 2816 3 to 4 us.
#include "fm_dropout.hpp"
#include "fm_norm.hpp"

namespace fm {
namespace {

constexpr int64_t kDropGridX = 1 << 20;
constexpr int kDropThreads = 256;

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
  const int64_t first = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kDropThreads;
  const int64_t at = first + threadIdx.x;
  if (at >= a.chunks) return;
  f32x4 v[2];
  load8<E>(static_cast<const T*>(a.x) + at * 8, v);
  if (a.d.rng) {
    // row and column of the block's first chunk are scalars; a lane's from there in 32 bits
    const int64_t row0 = a.chunks >> 32 ? first / a.per_row : (int64_t)((uint32_t)first / a.per_row);
    const uint32_t c = (uint32_t)(first - row0 * a.per_row) + threadIdx.x, r = c / a.per_row;
    const u32x4 w = philox(philox_of(a.d), a.d.block + (c - r * a.per_row), a.d.row + (uint32_t)row0 + r);
    v[0] = drop4(v[0], w[0], w[1], a.d);
    v[1] = drop4(v[1], w[2], w[3], a.d);
  }
  store8<E>(static_cast<T*>(a.y) + at * 8, v);
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
  const int64_t blocks = cdiv(a.chunks, kDropThreads);
  const int64_t gx = blocks < kDropGridX ? blocks : kDropGridX, gy = cdiv(blocks, gx);
  if (gy > 65535) return FM_ERR_UNSUPPORTED;   // 2^47 elements
  const dim3 grid((unsigned)gx, (unsigned)gy), lanes(kDropThreads);
  if (dt == FM_F16) hipLaunchKernelGGL(dropout_rows<F16>, grid, lanes, 0, stream, a);
  else if (dt == FM_BF16) hipLaunchKernelGGL(dropout_rows<BF16>, grid, lanes, 0, stream, a);
  else hipLaunchKernelGGL(dropout_rows<F32>, grid, lanes, 0, stream, a);
  return launch_status();
}
