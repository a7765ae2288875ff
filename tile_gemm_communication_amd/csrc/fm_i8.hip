// fm_i8.hip -- rows in 8 bits with a scale each, and the C interface of their products
// with 8-bit weights (fm_i8_few.hip, fm_i8_tiles.hip).
//
// Quantisation reads a row once: a lane keeps its part between the largest magnitude and
// the values.  Bound by the bytes: 4096 x 12288 bf16 31 us, 4.9 TB/s.
#include <algorithm>

#include "fm_i8.hpp"

namespace fm {
namespace {

// -- rows to 8 bits ------------------------------------------------------------

constexpr int kQuantHeld = 4;   // chunks of eight elements that a lane keeps between its passes

struct QuantArgs {
  const void* x;
  char* q;
  float* scale;
  int64_t M, N;
};

// A row of TH lanes (a block has at least 256): the largest magnitude, then the values, from
// registers as far as they fit and read again beyond.
template <typename E, int TH>
__global__ __launch_bounds__(TH < 256 ? 256 : TH) void quant_rows(const QuantArgs a) {
  using T = typename Elem<E>::type;
  constexpr int RW = TH < 256 ? 256 / TH : 1;
  __shared__ uint32_t s_top[TH / 64];   // (one wave a row needs none)
  const int t = threadIdx.x % TH;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RW + row_lane<TH>();
  if (row >= a.M) return;   // whole waves, and RW > 1 has no barrier
  const T* x = static_cast<const T*>(a.x) + row * a.N;
  Raw8<E> v[kQuantHeld];
  uint32_t top = 0;
  auto join = [&](const Raw8<E>& r) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4 w = half8<E>(r, h);
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, magnitude(w[i]));
    }
  };
#pragma unroll
  for (int c = 0; c < kQuantHeld; ++c) {
    const int64_t e = (int64_t)(c * TH + t) * 8;
    v[c] = {};
    if (e < a.N) v[c] = raw8<E>(x, e);
  }
#pragma unroll
  for (int c = 0; c < kQuantHeld; ++c) join(v[c]);
  const int64_t rest = (int64_t)(kQuantHeld * TH + t) * 8;
  for (int64_t e = rest; e < a.N; e += TH * 8) join(raw8<E>(x, e));
  const RowQuant r = row_quant(row_umax<TH>(top, s_top));
  if (t == 0) a.scale[row] = r.scale;
  char* q = a.q + row * a.N;
  auto put = [&](int64_t e, const Raw8<E>& w) {
    *reinterpret_cast<u32x2*>(q + e) = u32x2{quant4(half8<E>(w, 0), r), quant4(half8<E>(w, 1), r)};
  };
#pragma unroll
  for (int c = 0; c < kQuantHeld; ++c) {
    const int64_t e = (int64_t)(c * TH + t) * 8;
    if (e < a.N) put(e, v[c]);
  }
  for (int64_t e = rest; e < a.N; e += TH * 8) put(e, raw8<E>(x, e));
}

fm_status_t check_quant(fm_dtype_t dt, int64_t M, int64_t N) {
  if (dt != FM_F16 && dt != FM_BF16 && dt != FM_F32) return FM_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || N % 8) return FM_ERR_INVALID_ARG;
  if (M >= (1ll << 31) || N >= (1ll << 31)) return FM_ERR_UNSUPPORTED;
  return FM_OK;
}

template <typename E>
void launch_quant_rows(const QuantArgs& a, hipStream_t stream) {
#define FM_QUANT(TH)                                                                        \
  do {                                                                                      \
    const int64_t blocks = cdiv(a.M, TH < 256 ? 256 / TH : 1), x = std::min<int64_t>(blocks, 1 << 20); \
    hipLaunchKernelGGL((quant_rows<E, TH>), dim3((unsigned)x, (unsigned)cdiv(blocks, x)),   \
                       dim3(TH < 256 ? 256 : TH), 0, stream, a);                            \
  } while (0)
  // 65536 x 512 with 64 lanes a row 24 us, 256 58; 16384 x 2048 22 and 24; 16384 x 4096 with
  // 256 lanes 38, 64 47, 1024 66; 16384 x 6144 57, 78, 77; 4096 x 12288 with 1024 31, 256 35
  if (a.N <= 2048) FM_QUANT(64);
  else if (a.N <= 8192) FM_QUANT(256);
  else FM_QUANT(1024);
#undef FM_QUANT
}

void launch_quant(fm_dtype_t dt, const QuantArgs& a, hipStream_t stream) {
  if (dt == FM_F16) launch_quant_rows<F16>(a, stream);
  else if (dt == FM_BF16) launch_quant_rows<BF16>(a, stream);
  else launch_quant_rows<F32>(a, stream);
}

// A sum of K products of bytes fits 32 bits up to here (127 * 128 * K, and -128 may
// stand in a caller's own codes: 2^14 K < 2^31).
constexpr int64_t kI8MaxK = (1ll << 17) - 16;
constexpr int64_t kI8MaxDim = 1ll << 22;

fm_status_t check_i8(fm_dtype_t dt, fm_dtype_t c, int64_t M, int64_t N, int64_t K, fm_act_t act) {
  if ((dt != FM_F16 && dt != FM_BF16) || (c != dt && c != FM_F32)) return FM_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K < 0 || N % 8 || K % 16) return FM_ERR_INVALID_ARG;
  if ((int)act < FM_ACT_NONE || (int)act > FM_ACT_SILU) return FM_ERR_INVALID_ARG;
  if (M >= kI8MaxDim || N >= kI8MaxDim || M * N >= (1ll << 42) || K > kI8MaxK) return FM_ERR_UNSUPPORTED;
  return FM_OK;
}

// Few rows share k among a block's waves, tiles walk all of it: few columns and a long k cost a
// step at the border (64 x 1024 x 12288 11.2 us, 65 rows 21.3; of 512 x 4096 4.9 and 9.2).
void launch_product(const I8Args& a, hipStream_t stream) {
  if (a.M <= kI8FewRows) launch_i8_few(a, stream);
  else launch_i8_tiles(a, stream);
}

int64_t codes_bytes(int64_t M, int64_t K) { return cdiv(M * K, 256) * 256; }

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" fm_status_t fm_quant_i8(fm_dtype_t dt, int64_t M, int64_t N, const void* x, int8_t* q,
                                   float* scale, hipStream_t stream) {
  const fm_status_t st = check_quant(dt, M, N);
  if (st != FM_OK) return st;
  if (M == 0) return FM_OK;
  if (!scale || !aligned4(scale)) return FM_ERR_INVALID_ARG;
  if (N > 0 && (!x || !q)) return FM_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q)) return FM_ERR_INVALID_ARG;
  launch_quant(dt, {x, reinterpret_cast<char*>(q), scale, M, N}, stream);
  return launch_status();
}

extern "C" fm_status_t fm_gemm_i8(fm_dtype_t dt, fm_dtype_t c, int64_t M, int64_t N, int64_t K,
                                  const int8_t* A, const float* a_scale, const int8_t* W,
                                  const float* w_scale, const void* bias, fm_act_t act, void* C,
                                  hipStream_t stream) {
  const fm_status_t st = check_i8(dt, c, M, N, K, act);
  if (st != FM_OK) return st;
  if (M == 0 || N == 0) return FM_OK;
  if (!a_scale || !w_scale || !C || (K > 0 && (!A || !W))) return FM_ERR_INVALID_ARG;
  for (const void* p : {(const void*)A, (const void*)W, (const void*)w_scale, bias, (const void*)C})
    if (!aligned16(p)) return FM_ERR_INVALID_ARG;
  if (!aligned4(a_scale)) return FM_ERR_INVALID_ARG;
  launch_product({(const char*)A, (const char*)W, a_scale, w_scale, bias, (char*)C, M, N, K, (int)act, dt, c},
                 stream);
  return launch_status();
}

extern "C" size_t fm_linear_i8_workspace_bytes(int64_t M, int64_t K) {
  if (M < 0 || K < 0 || K % 16 || M >= kI8MaxDim || K > kI8MaxK) return 0;
  return std::max<size_t>((size_t)codes_bytes(M, K) + (size_t)M * 4, 256);
}

extern "C" fm_status_t fm_linear_i8(fm_dtype_t dt, fm_dtype_t c, int64_t M, int64_t N, int64_t K,
                                    const void* X, const int8_t* W, const float* w_scale,
                                    const void* bias, fm_act_t act, void* C, void* ws,
                                    size_t ws_bytes, hipStream_t stream) {
  const fm_status_t st = check_i8(dt, c, M, N, K, act);
  if (st != FM_OK) return st;
  if (M == 0 || N == 0) return FM_OK;
  if (!w_scale || !C || (K > 0 && (!X || !W))) return FM_ERR_INVALID_ARG;
  for (const void* p : {X, (const void*)W, (const void*)w_scale, bias, (const void*)C, (const void*)ws})
    if (!aligned16(p)) return FM_ERR_INVALID_ARG;
  if (!ws || ws_bytes < fm_linear_i8_workspace_bytes(M, K)) return FM_ERR_INVALID_ARG;
  I8Args a = {(const char*)X, (const char*)W, nullptr, w_scale, bias, (char*)C, M, N, K, (int)act, dt, c};
  if (i8_few_quantises(M, K)) {
    launch_i8_few_quant(a, stream);
    return launch_status();
  }
  char* codes = static_cast<char*>(ws);
  float* scale = reinterpret_cast<float*>(codes + codes_bytes(M, K));
  launch_quant(dt, {X, codes, scale, M, K}, stream);
  a.A = codes;
  a.a_scale = scale;
  launch_product(a, stream);
  return launch_status();
}
