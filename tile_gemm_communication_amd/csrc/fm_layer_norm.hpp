// fm_layer_norm.hpp -- what the layer norm's forward and backward share, and the
// 8-bit form of a row.
#pragma once

#include "fm_dropout.hpp"
#include "fm_norm.hpp"

namespace fm {

fm_status_t check_layer_norm(fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt, int64_t M,
                             int64_t N, float p, const uint64_t* rng, int64_t row_begin);

// Lanes and chunks of eight elements that hold a row of N: F(lanes, chunks).  Forward,
// us: 65536 x 256 with 32 lanes 29, 64 43; 16384 x 4096 with 512 lanes 120, 256 twice 120
// (509 rows: 5.1, 5.9); 8192 x 8192 fp32 with 1024 169, 512 twice 172; 4088 x 12288 with 768
// twice, which fit exactly, 132, 512 three times 137; 4088 x 16384 bf16 with 1024 twice 104,
// 512 four times 131.
#define FM_LN_SIZES(N, F)            \
  do {                               \
    if ((N) <= 128) F(16, 1);        \
    else if ((N) <= 256) F(32, 1);   \
    else if ((N) <= 512) F(64, 1);   \
    else if ((N) <= 1024) F(128, 1); \
    else if ((N) <= 2048) F(256, 1); \
    else if ((N) <= 4096) F(512, 1); \
    else if ((N) <= 8192) F(1024, 1);\
    else if ((N) <= 12288) F(768, 2);\
    else F(1024, 2);                 \
  } while (0)

// The row lane of a thread, where it is one for a whole wave in a scalar register.
template <int TH>
__device__ __forceinline__ int row_lane() {
  const int rw = (int)threadIdx.x / TH;
  return TH < 64 ? rw : __builtin_amdgcn_readfirstlane(rw);
}

// row_sum, also of rows that share a wave.
template <int TH>
__device__ __forceinline__ float ln_sum(float x, float* slots) {
  if constexpr (TH < 64) return group_sum<TH>(x);
  else return row_sum<TH>(x, slots);
}

// Rows in 8 bits: scale = max|x| / 127, q = x * 127 / max|x| rounded to nearest
// even.  A row whose largest magnitude is below 2^-100 is held as zeros with scale
// 0, one with a NaN or with 2^120 and more as zeros with scale NaN.
struct RowQuant {
  float top, inv, scale;
};

// Magnitudes as whole numbers: NaN is the largest.
__device__ __forceinline__ uint32_t magnitude(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}

__device__ __forceinline__ RowQuant row_quant(uint32_t top_bits) {
  const float top = __builtin_bit_cast(float, top_bits);
  if (!(top < 0x1p120f)) return {1.f, 0.f, __builtin_nanf("")};
  if (top < 0x1p-100f) return {1.f, 0.f, 0.f};
  return {top, 1.f / top, top / 127.f};
}

// Four values, a byte each.  t / top is correctly rounded: the remainder of t * inv
// is exact in one fused step (Markstein), and inv is the rounded reciprocal; so a
// half is seen as a half where 127 x is exact, which it is for 16-bit x.
__device__ __forceinline__ uint32_t quant4(f32x4 x, const RowQuant& r) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float t = x[i] * 127.f, q0 = t * r.inv;
    const float q = r.inv == 0.f ? 0.f : fmaf(fmaf(-q0, r.top, t), r.inv, q0);
    w |= ((uint32_t)(int)rintf(q) & 0xffu) << (8 * i);
  }
  return w;
}

// Largest whole number of a row's TH lanes, in all of them (slots as row_sum's).
template <int LANES, int STEP = 1>
__device__ __forceinline__ uint32_t group_umax(uint32_t x) {
  if constexpr (STEP < LANES) {
    const LanePair<int> p = lane_pair<STEP>((int)x);
    const uint32_t a = (uint32_t)p.a, b = (uint32_t)p.b;
    return group_umax<LANES, STEP * 2>(a > b ? a : b);
  } else {
    return x;
  }
}

template <int TH>
__device__ __forceinline__ uint32_t row_umax(uint32_t x, uint32_t* slots) {
  x = group_umax<TH < 64 ? TH : 64>(x);
  if constexpr (TH > 64) {
    const int t = threadIdx.x % TH;
    if (t % 64 == 0) slots[t / 64] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < TH / 64; ++w) x = slots[w] > x ? slots[w] : x;
  }
  return x;
}

}  // namespace fm
