// fm_act.hpp -- activations of a product's epilogue (fm_act_t).
#pragma once

#include "fm_common.hpp"

namespace fm {

__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case FM_ACT_RELU: return x > 0.f ? x : 0.f;
    case FM_ACT_GELU_TANH: {
      // x/2 (1 + tanh u) = x / (1 + exp(-2u))
      const float u = 0.7978845608028654f * (x + 0.044715f * x * x * x);
      return x / (1.f + __expf(-2.f * u));
    }
    case FM_ACT_SILU: return x / (1.f + __expf(-x));
    default: return x;
  }
}

// The activations of N values, one branch for all: x / (1 + exp(-z)) as x times the
// hardware's reciprocal (1 ulp) of 1 + 2^(-z log2 e), z's factors folded into two
// constants.  A large tile's results are all finished at once with the matrix cores idle,
// so its instructions count: GELU takes 7 vector instructions a value, 19 with a division
// (4096 x 12288 x 6144 with its rows quantised: 283 us, so 305).
// Where z overflows the limits hold: x or -0.
template <int N>
__device__ __forceinline__ void activate_all(f32x4 (&v)[N], int act) {
  auto each = [&](auto f) {
#pragma unroll
    for (int h = 0; h < N; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[h][i] = f(v[h][i]);
  };
  auto gated = [](float x, float e) {
    return x * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(e));
  };
  constexpr float kLog2e = 1.4426950408889634f, kGelu = -2.f * 0.7978845608028654f * kLog2e;
  switch (act) {
    case FM_ACT_RELU:   // a NaN stays one, in one instruction
      return each([](float x) { return __builtin_elementwise_maximum(x, 0.f); });
    case FM_ACT_GELU_TANH:
      return each([&](float x) { return gated(x, x * fmaf(kGelu * 0.044715f, x * x, kGelu)); });
    case FM_ACT_SILU: return each([&](float x) { return gated(x, x * -kLog2e); });
    default: return;
  }
}

}  // namespace fm
