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

// Eight consecutive elements, 16 bytes or twice 16, aligned as such, as they are held
// in memory.
template <typename E>
struct Raw8 {
  u32x4 r[sizeof(typename Elem<E>::type) / 2];
};

template <typename E>
__device__ __forceinline__ Raw8<E> raw8(const void* p, int64_t e) {
  const auto* q = static_cast<const typename Elem<E>::type*>(p) + e;
  return *reinterpret_cast<const Raw8<E>*>(q);
}

// Four of them, h = 0 or 1, in 32 bits.
template <typename E>
__device__ __forceinline__ f32x4 half8(const Raw8<E>& v, int h) {
  if constexpr (sizeof(v) == 32) return __builtin_bit_cast(f32x4, v.r[h]);
  else return widen<E>(__builtin_bit_cast(typename Raw4<E>::type, u32x2{v.r[0][2 * h], v.r[0][2 * h + 1]}));
}

template <typename E>
__device__ __forceinline__ void load8(const typename Elem<E>::type* p, f32x4 (&v)[2]) {
  const Raw8<E> r = raw8<E>(p, 0);
  v[0] = half8<E>(r, 0);
  v[1] = half8<E>(r, 1);
}

template <typename E>
__device__ __forceinline__ void store8(typename Elem<E>::type* p, const f32x4 (&v)[2]) {
  if constexpr (sizeof(*p) == 4) {
    store4<E>(p, v[0]);
    store4<E>(p + 4, v[1]);
  } else {
    const u32x2 a = __builtin_bit_cast(u32x2, narrow<E>(v[0]));
    const u32x2 b = __builtin_bit_cast(u32x2, narrow<E>(v[1]));
    *reinterpret_cast<u32x4*>(p) = u32x4{a[0], a[1], b[0], b[1]};
  }
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
