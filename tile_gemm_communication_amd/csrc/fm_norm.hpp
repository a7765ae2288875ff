// fm_norm.hpp -- what the norm's forward and backward kernels share.
#pragma once

#include "fm_wave.hpp"

namespace fm {

constexpr int kNormMaxN = 16384;

struct NormArgs {
  const void *block, *resid, *w_post, *w_pre, *gate;
  void *out, *y;
  float *rstd_post, *rstd_pre;
  int64_t M;
  int N;
  uint32_t rows_per_gate;
  float scale, eps;
};

fm_status_t check_norm(fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt, int64_t M,
                       int64_t N, const void* gate, int64_t n_gates);

template <typename E>
__device__ __forceinline__ typename Raw4<E>::type raw4(const void* p, int e) {
  return *reinterpret_cast<const typename Raw4<E>::type*>(
      static_cast<const typename Elem<E>::type*>(p) + e);
}

template <typename E>
__device__ __forceinline__ f32x4 load4(const typename Elem<E>::type* p) {
  return widen<E>(*reinterpret_cast<const typename Raw4<E>::type*>(p));
}

template <typename E>
__device__ __forceinline__ void store4(typename Elem<E>::type* p, f32x4 v) {
  *reinterpret_cast<typename Raw4<E>::type*>(p) = narrow<E>(v);
}

__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) {
  return (a[0] * b[0] + a[1] * b[1]) + (a[2] * b[2] + a[3] * b[3]);
}

// 1 / sqrt(mean + eps); v_rsq_f32 is within 1 ulp.
__device__ __forceinline__ float rstd_of(float mean, float eps) {
  return __builtin_amdgcn_rsqf(mean + eps);
}

// Sum over the TH lanes of a row, in all of them; slots: TH / 64 floats of LDS
// that this row does not use again before its next barrier.
template <int TH>
__device__ __forceinline__ float row_sum(float x, float* slots) {
  x = group_sum<64>(x);
  if constexpr (TH > 64) {
    const int t = threadIdx.x % TH;
    if (t % 64 == 0) slots[t / 64] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int w = 0; w < TH / 64; ++w) x += slots[w];
  }
  return x;
}

}  // namespace fm
