// fm_i8.hpp -- what the kernels of 8-bit products share.
#pragma once

#include "fm_act.hpp"
#include "fm_layer_norm.hpp"

namespace fm {

struct I8Args {
  const char *A, *W;                // [M, K], [N, K]
  const float *a_scale, *w_scale;   // [M], [N]
  const void* bias;                 // [N] or NULL
  char* C;                          // [M, N]
  int64_t M, N, K;
  int act;
  fm_dtype_t dt, c;                 // bias; C
};

// Products of at most kI8FewRows rows (fm_i8_few.hip).
constexpr int kI8FewRows = 64;
void launch_i8_few(const I8Args& a, hipStream_t stream);

// The same of rows in 16 bits (A, in dt), quantised by each block for itself.
bool i8_few_quantises(int64_t M, int64_t K);
void launch_i8_few_quant(const I8Args& a, hipStream_t stream);

// Products of many rows (fm_i8_tiles.hip).
void launch_i8_tiles(const I8Args& a, hipStream_t stream);

}  // namespace fm
