// fm_act.hpp -- activations of a product's epilogue (fm_act_t).
#pragma once

#include <type_traits>

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

// The same of N values, one branch for all.
template <int N>
__device__ __forceinline__ void activate_all(f32x4 (&v)[N], int act) {
  auto each = [&](auto code) {
#pragma unroll
    for (int h = 0; h < N; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[h][i] = activate(v[h][i], decltype(code)::value);
  };
  switch (act) {
    case FM_ACT_RELU: return each(std::integral_constant<int, FM_ACT_RELU>{});
    case FM_ACT_GELU_TANH: return each(std::integral_constant<int, FM_ACT_GELU_TANH>{});
    case FM_ACT_SILU: return each(std::integral_constant<int, FM_ACT_SILU>{});
    default: return;
  }
}

}  // namespace fm
