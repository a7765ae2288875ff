// fm_norm.hip -- norm after a block, gate, scale, residual add and the norm
// before the next block, in one pass over the rows (forward).
//
// One row lies in the registers of TH lanes, CH chunks of four elements each, so
// block and residual are read once and out and y written once: the operator is
// bound by those bytes.  The two mean squares are the only exchanges between
// lanes (DPP within a wave, one LDS slot a wave beyond).  16384 x 4096 bf16 with an
// fp32 block: 133 us, 5.0 TB/s; 3 x 4096: 3.8 us, one wait for memory after another.
#include "fm_norm.hpp"

namespace fm {
namespace {

constexpr int64_t kNormGridX = 1 << 20;

// TH lanes hold a row; a block of 256 has 4 rows of 64 lanes, else one row.
template <typename E, typename S, typename B, int TH, int CH>
__global__ __launch_bounds__(TH == 64 ? 256 : TH) void norm_fwd(const NormArgs a) {
  constexpr int RW = TH == 64 ? 4 : 1;
  __shared__ float s_red[2][TH / 64];
  const int t = threadIdx.x % TH, N = a.N;
  const int64_t row =
      ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RW + threadIdx.x / TH;
  if (row >= a.M) return;   // whole waves, and RW > 1 has no barrier
  const float invN = 1.f / (float)N;

  f32x4 z[CH], b[CH];
  typename Raw4<E>::type wq[CH], wp[CH], g[CH];
  const auto* blk = static_cast<const typename Elem<B>::type*>(a.block) + row * N;
  const auto* res = static_cast<const typename Elem<S>::type*>(a.resid) + row * N;
  const auto* gate = static_cast<const typename Elem<E>::type*>(a.gate) +
                     (a.gate ? (int64_t)((uint32_t)row / a.rows_per_gate) * N : 0);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = (c * TH + t) * 4;
    const bool in = e < N;
    b[c] = in && a.block ? load4<B>(blk + e) : f32x4{0.f, 0.f, 0.f, 0.f};
    z[c] = in && a.resid ? load4<S>(res + e) : f32x4{0.f, 0.f, 0.f, 0.f};
    if (in && a.w_post) wq[c] = raw4<E>(a.w_post, e);
    if (in && a.w_pre) wp[c] = raw4<E>(a.w_pre, e);
    if (in && a.gate) g[c] = raw4<E>(gate, e);
  }
  if (a.w_post) {
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) ss += dot4(b[c], b[c]);
    ss = row_sum<TH>(ss, s_red[0]);
    const float r = rstd_of(ss * invN, a.eps);
    if (a.rstd_post && t == 0) a.rstd_post[row] = r;
#pragma unroll
    for (int c = 0; c < CH; ++c) b[c] *= r;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if ((c * TH + t) * 4 < N) b[c] *= widen<E>(wq[c]);
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = (c * TH + t) * 4;
    if (e < N) {
      if (a.gate) b[c] *= widen<E>(g[c]);
      if (a.block) z[c] += b[c] * a.scale;
      if (a.out) store4<S>(static_cast<typename Elem<S>::type*>(a.out) + row * N + e, z[c]);
    }
    ss += dot4(z[c], z[c]);
  }
  if (!a.w_pre) return;
  ss = row_sum<TH>(ss, s_red[1]);
  const float r = rstd_of(ss * invN, a.eps);
  if (a.rstd_pre && t == 0) a.rstd_pre[row] = r;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = (c * TH + t) * 4;
    if (e < N)
      store4<E>(static_cast<typename Elem<E>::type*>(a.y) + row * N + e, z[c] * r * widen<E>(wp[c]));
  }
}

template <typename E, typename S, typename B>
void launch_fwd(const NormArgs& a, hipStream_t stream) {
// Lanes of a row, 16384 rows: N = 256 with 64 lanes 10.4 us, 256 20.3; 512 16.7 and
// 23.9; 1024 either 31; 4096 with 256 lanes 127, 1024 133; 8192 with 1024 238, 256 321.
// Two grid dimensions: one holds fewer than 2^32 lanes.
#define FM_FWD(TH, CH)                                                                       \
  do {                                                                                       \
    const int64_t blocks = cdiv(a.M, TH == 64 ? 4 : 1), x = blocks < kNormGridX ? blocks : kNormGridX; \
    hipLaunchKernelGGL((norm_fwd<E, S, B, TH, CH>), dim3((unsigned)x, (unsigned)cdiv(blocks, x)), \
                       dim3(TH == 64 ? 256 : TH), 0, stream, a);                             \
  } while (0)
  const int N = a.N;
  if (N <= 256) FM_FWD(64, 1);
  else if (N <= 512) FM_FWD(64, 2);
  else if (N <= 1024) FM_FWD(256, 1);
  else if (N <= 2048) FM_FWD(256, 2);
  else if (N <= 4096) FM_FWD(256, 4);
  else if (N <= 8192) FM_FWD(1024, 2);
  else if (N <= 12288) FM_FWD(1024, 3);
  else FM_FWD(1024, 4);
#undef FM_FWD
}

template <typename E>
void launch_types(fm_dtype_t stream_dt, fm_dtype_t block_dt, const NormArgs& a,
                  hipStream_t stream) {
  if (stream_dt == FM_F32) {
    if (block_dt == FM_F32) launch_fwd<E, F32, F32>(a, stream);
    else launch_fwd<E, F32, E>(a, stream);
  } else {
    if (block_dt == FM_F32) launch_fwd<E, E, F32>(a, stream);
    else launch_fwd<E, E, E>(a, stream);
  }
}

}  // namespace

fm_status_t check_norm(fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt, int64_t M,
                       int64_t N, const void* gate, int64_t n_gates) {
  if (dt != FM_F16 && dt != FM_BF16) return FM_ERR_UNSUPPORTED;
  if ((stream_dt != dt && stream_dt != FM_F32) || (block_dt != dt && block_dt != FM_F32))
    return FM_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || N % 8) return FM_ERR_INVALID_ARG;
  if (gate ? (n_gates < 1 || (M > 0 && (n_gates > M || M % n_gates))) : n_gates != 0)
    return FM_ERR_INVALID_ARG;
  if (N > kNormMaxN || M >= (1ll << 31) || (M == 0 && n_gates > kNormGridX))
    return FM_ERR_UNSUPPORTED;
  return FM_OK;
}

}  // namespace fm

using namespace fm;

extern "C" fm_status_t fm_norm_residual(fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt,
                                        int64_t M, int64_t N, const void* block,
                                        const void* resid, const void* w_post, const void* w_pre,
                                        const void* gate, int64_t n_gates, float scale, float eps,
                                        void* out, void* y, float* rstd_post, float* rstd_pre,
                                        hipStream_t stream) {
  const fm_status_t st = check_norm(dt, stream_dt, block_dt, M, N, gate, n_gates);
  if (st != FM_OK) return st;
  if (!(eps >= 0.f)) return FM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return FM_OK;   // an empty batch's tensors have no addresses
  if ((w_pre == nullptr) != (y == nullptr)) return FM_ERR_INVALID_ARG;
  if ((!block && (w_post || gate)) || (rstd_post && !w_post) || (rstd_pre && !w_pre))
    return FM_ERR_INVALID_ARG;
  if ((!block && !resid) || (!out && !y)) return FM_ERR_INVALID_ARG;
  for (const void* p : {block, resid, w_post, w_pre, gate, (const void*)out, (const void*)y})
    if (!aligned16(p)) return FM_ERR_INVALID_ARG;
  if (!aligned4(rstd_post) || !aligned4(rstd_pre)) return FM_ERR_INVALID_ARG;
  NormArgs a = {};
  a.block = block;
  a.resid = resid;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.gate = gate;
  a.out = out;
  a.y = y;
  a.rstd_post = rstd_post;
  a.rstd_pre = rstd_pre;
  a.M = M;
  a.N = (int)N;
  a.rows_per_gate = gate ? (uint32_t)(M / n_gates) : 1u;
  a.scale = scale;
  a.eps = eps;
  if (dt == FM_F16) launch_types<F16>(stream_dt, block_dt, a, stream);
  else launch_types<BF16>(stream_dt, block_dt, a, stream);
  return launch_status();
}
