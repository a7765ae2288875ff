// fm_dropout.hpp -- the mask of fm_dropout and fm_layer_norm.
//
// Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw: "Parallel Random Numbers:
// As Easy as 1, 2, 3", 2011): four words from a counter and a key by multiplications
// alone, so any element's number can be had anywhere and the mask is never stored.
// A counter serves eight elements of a row, 16 bits each: 20 widening products for
// eight elements, which the row kernels hide behind their loads.
#pragma once

#include <cmath>

#include "fm_common.hpp"

namespace fm {

// What one call draws; rng = NULL: everything is kept as it is.
struct Dropout {
  const uint64_t* rng;    // seed, offset
  int64_t draw;           // added to the offset
  uint32_t row, block;    // first row, and first column / 8
  uint32_t threshold;     // an element is kept if its 16 bits are below it
  float scale;            // of what is kept
};

// p rounded to a multiple of 2^-16, so that threshold and scale agree.
inline Dropout make_dropout(float p, const uint64_t* rng, int64_t draw, int64_t row_begin,
                            int64_t col_begin) {
  const double keep = std::floor((1.0 - (double)p) * 65536.0 + 0.5);
  return {keep < 65536.0 ? rng : nullptr, draw, (uint32_t)row_begin, (uint32_t)(col_begin / 8),
          (uint32_t)keep, keep > 0.0 ? (float)(65536.0 / keep) : 0.f};
}

// The words of a counter that a whole call shares, in scalar registers.
struct Philox {
  uint32_t k0, k1, c2, c3;
};

__device__ __forceinline__ Philox philox_of(const Dropout& d) {
  const uint64_t seed = d.rng[0], at = d.rng[1] + (uint64_t)d.draw;
  auto uniform = [](uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); };
  return {uniform((uint32_t)seed), uniform((uint32_t)(seed >> 32)), uniform((uint32_t)at),
          uniform((uint32_t)(at >> 32))};
}

__device__ __forceinline__ u32x4 philox(const Philox& p, uint32_t c0, uint32_t c1) {
  uint32_t c2 = p.c2, c3 = p.c3, k0 = p.k0, k1 = p.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// Four elements whose numbers are the halves of two words, the low half first.
// What is dropped is 0, whatever it was.
__device__ __forceinline__ f32x4 drop4(f32x4 v, uint32_t lo, uint32_t hi, const Dropout& d) {
  return f32x4{(lo & 0xffffu) < d.threshold ? v[0] * d.scale : 0.f,
               (lo >> 16) < d.threshold ? v[1] * d.scale : 0.f,
               (hi & 0xffffu) < d.threshold ? v[2] * d.scale : 0.f,
               (hi >> 16) < d.threshold ? v[3] * d.scale : 0.f};
}

// What the host checks of p and the mask's place.
inline fm_status_t check_dropout(float p, const uint64_t* rng, int64_t M, int64_t row_begin,
                                 int64_t N, int64_t col_begin) {
  if (!(p >= 0.f && p <= 1.f) || (p > 0.f && !rng) || (reinterpret_cast<uintptr_t>(rng) & 7u))
    return FM_ERR_INVALID_ARG;
  if (row_begin < 0 || col_begin < 0 || col_begin % 8) return FM_ERR_INVALID_ARG;
  if (row_begin > (1ll << 32) - M || col_begin > (1ll << 34) - N) return FM_ERR_UNSUPPORTED;
  return FM_OK;
}

}  // namespace fm
