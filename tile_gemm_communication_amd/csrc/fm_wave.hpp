// fm_wave.hpp -- lane exchanges and 16-bit conversions shared by the row-wise
// kernels (router, norms).
#pragma once

#include "fm_common.hpp"

namespace fm {

// x of the lane that a DPP pattern names (every lane has a source).
template <int CTRL>
__device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false);
}

template <typename V>
struct LanePair {
  V a, b;
};

// The two values that an all-reduce step over 2 * STEP lanes joins.  After the
// steps below it, every lane of a STEP-lane group holds the same value, so any
// lane of the other half serves: neighbours and pairs by quad permutes, halves
// of 8 and 16 lanes by mirrors, rows of 16 and halves of 32 by row swaps.
template <int STEP>
__device__ __forceinline__ LanePair<int> lane_pair(int x) {
  if constexpr (STEP == 1) return {x, dpp<0xB1>(x)};
  else if constexpr (STEP == 2) return {x, dpp<0x4E>(x)};
  else if constexpr (STEP == 4) return {x, dpp<0x141>(x)};
  else if constexpr (STEP == 8) return {x, dpp<0x140>(x)};
  else if constexpr (STEP == 16) {
    auto r = __builtin_amdgcn_permlane16_swap((unsigned)x, (unsigned)x, false, false);
    return {(int)r[0], (int)r[1]};
  } else {
    auto r = __builtin_amdgcn_permlane32_swap((unsigned)x, (unsigned)x, false, false);
    return {(int)r[0], (int)r[1]};
  }
}

template <int STEP>
__device__ __forceinline__ LanePair<float> lane_pair(float x) {
  const LanePair<int> p = lane_pair<STEP>(__builtin_bit_cast(int, x));
  return {__builtin_bit_cast(float, p.a), __builtin_bit_cast(float, p.b)};
}

template <int STEP>
__device__ __forceinline__ LanePair<double> lane_pair(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const LanePair<int> lo = lane_pair<STEP>((int)(uint32_t)u);
  const LanePair<int> hi = lane_pair<STEP>((int)(uint32_t)(u >> 32));
  return {__builtin_bit_cast(double, (uint64_t)(uint32_t)lo.a | ((uint64_t)(uint32_t)hi.a << 32)),
          __builtin_bit_cast(double, (uint64_t)(uint32_t)lo.b | ((uint64_t)(uint32_t)hi.b << 32))};
}

// Sum over groups of LANES lanes, in every lane.  Both halves add the same two
// numbers in each step: identical bits in all lanes.
template <int LANES, int STEP = 1, typename V>
__device__ __forceinline__ V group_sum(V x) {
  if constexpr (STEP < LANES) {
    const LanePair<V> p = lane_pair<STEP>(x);
    return group_sum<LANES, STEP * 2>(p.a + p.b);
  } else {
    return x;
  }
}

template <int LANES, int STEP = 1>
__device__ __forceinline__ float group_max(float x) {
  if constexpr (STEP < LANES) {
    const LanePair<float> p = lane_pair<STEP>(x);
    return group_max<LANES, STEP * 2>(fmaxf(p.a, p.b));
  } else {
    return x;
  }
}

// LDS traffic between the lanes of one wave: the wave's LDS operations complete
// in order, so only the compiler has to keep them so.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Element types of a row: F32 beside the 16-bit formats.
struct F32 {
  static constexpr fm_dtype_t id = FM_F32;
};

template <typename E> struct Elem;
template <> struct Elem<F16> { typedef _Float16 type; };
template <> struct Elem<BF16> { typedef __bf16 type; };
template <> struct Elem<F32> { typedef float type; };

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// Four consecutive elements, 8 or 16 bytes, aligned as such.
template <typename E> struct Raw4;
template <> struct Raw4<F16> { typedef f16x4 type; };
template <> struct Raw4<BF16> { typedef bf16x4 type; };
template <> struct Raw4<F32> { typedef f32x4 type; };

template <typename E>
__device__ __forceinline__ f32x4 widen(typename Raw4<E>::type v) {
  return __builtin_convertvector(v, f32x4);
}

template <typename E>
__device__ __forceinline__ typename Raw4<E>::type narrow(f32x4 v) {
  return __builtin_convertvector(v, typename Raw4<E>::type);
}

}  // namespace fm
