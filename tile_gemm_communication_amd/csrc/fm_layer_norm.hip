// fm_layer_norm.hip -- bias, dropout, residual add and layer norm in one pass over
// the rows (forward).
//
// One row lies in the registers of TH lanes, CH chunks of eight elements each, so
// block and residual are read once and out and y written once: the operator is
// bound by those bytes.  Mean, centred mean square and, for y in 8 bits, the largest
// magnitude are the only exchanges between lanes.  16384 x 4096 bf16 with an fp32 block
// 120 us, 5.6 TB/s (116 without dropout; to 8 bits 113); 4088 x 12288 fp32 133 us; 1 x 4096
// 4 us, the call.  A lane's loads follow one another, each operand's under its own branch: many
// rows cover that, some hundred do not (509 x 4096 5.2 us, 3.2 TB/s).
#include "fm_layer_norm.hpp"

namespace fm {
namespace {

constexpr int64_t kLnGridX = 1 << 20;

struct LnArgs {
  const void *block, *resid, *bias, *w, *b;
  void *out, *y;
  float *y_scale, *mean, *rstd;
  int64_t M;
  int N;
  float eps;
  Dropout d;
};

// TH lanes hold a row; a block has at least 256 lanes.
template <typename E, typename S, typename B, int TH, int CH>
__global__ __launch_bounds__(TH < 256 ? 256 : TH) void layer_norm_fwd(const LnArgs a) {
  constexpr int RW = TH < 256 ? 256 / TH : 1;
  __shared__ float s_red[2][RW][(TH + 63) / 64];
  __shared__ uint32_t s_top[RW][(TH + 63) / 64];
  const int t = threadIdx.x % TH, N = a.N;
  const int rw = row_lane<TH>();
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RW + rw;
  if (TH == 64 && row >= a.M) return;   // whole waves, and no barrier follows
  const bool live = row < a.M;
  const int64_t at = row * N;
  const float invN = 1.f / (float)N;

  f32x4 z[CH][2], b[CH][2];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = (c * TH + t) * 8;
    const bool in = live && e < N;
    b[c][0] = b[c][1] = z[c][0] = z[c][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (in && a.block) load8<B>(static_cast<const typename Elem<B>::type*>(a.block) + at + e, b[c]);
    if (in && a.resid) load8<S>(static_cast<const typename Elem<S>::type*>(a.resid) + at + e, z[c]);
    if (in && a.bias) {
      f32x4 v[2];
      load8<E>(static_cast<const typename Elem<E>::type*>(a.bias) + e, v);
      b[c][0] += v[0];
      b[c][1] += v[1];
    }
  }
  if (a.d.rng) {
    const Philox p = philox_of(a.d);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const u32x4 w = philox(p, (uint32_t)(c * TH + t), a.d.row + (uint32_t)row);
      b[c][0] = drop4(b[c][0], w[0], w[1], a.d);
      b[c][1] = drop4(b[c][1], w[2], w[3], a.d);
    }
  }
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = (c * TH + t) * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      z[c][h] += b[c][h];
      s += (z[c][h][0] + z[c][h][1]) + (z[c][h][2] + z[c][h][3]);
    }
    if (a.out && live && e < N)
      store8<S>(static_cast<typename Elem<S>::type*>(a.out) + at + e, z[c]);
  }
  if (!a.w) return;
  const float mean = ln_sum<TH>(s, s_red[0][rw]) * invN;
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if ((c * TH + t) * 8 < N) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        z[c][h] -= mean;
        ss += dot4(z[c][h], z[c][h]);
      }
    }
  }
  const float r = rstd_of(ln_sum<TH>(ss, s_red[1][rw]) * invN, a.eps);
  if (live && t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = r;
  }
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = (c * TH + t) * 8;
    if (e < N) {
      f32x4 v[2];
      load8<E>(static_cast<const typename Elem<E>::type*>(a.w) + e, v);
#pragma unroll
      for (int h = 0; h < 2; ++h) z[c][h] *= v[h] * r;
      if (a.b) {
        load8<E>(static_cast<const typename Elem<E>::type*>(a.b) + e, v);
#pragma unroll
        for (int h = 0; h < 2; ++h) z[c][h] += v[h];
      }
      if (!a.y_scale) {
        if (live) store8<E>(static_cast<typename Elem<E>::type*>(a.y) + at + e, z[c]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = max(top, magnitude(z[c][h][i]));
      }
    }
  }
  if (!a.y_scale) return;
  const RowQuant q = row_quant(row_umax<TH>(top, s_top[rw]));
  if (live && t == 0) a.y_scale[row] = q.scale;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = (c * TH + t) * 8;
    if (live && e < N)
      *reinterpret_cast<u32x2*>(static_cast<char*>(a.y) + at + e) =
          u32x2{quant4(z[c][0], q), quant4(z[c][1], q)};
  }
}

template <typename E, typename S, typename B>
void launch_fwd(const LnArgs& a, hipStream_t stream) {
#define FM_LN_FWD(TH, CH)                                                                    \
  do {                                                                                       \
    const int64_t blocks = cdiv(a.M, TH < 256 ? 256 / TH : 1);                               \
    const int64_t x = blocks < kLnGridX ? blocks : kLnGridX;                                 \
    hipLaunchKernelGGL((layer_norm_fwd<E, S, B, TH, CH>),                                    \
                       dim3((unsigned)x, (unsigned)cdiv(blocks, x)),                         \
                       dim3(TH < 256 ? 256 : TH), 0, stream, a);                             \
  } while (0)
  FM_LN_SIZES(a.N, FM_LN_FWD);
#undef FM_LN_FWD
}

template <typename E>
void launch_types(fm_dtype_t stream_dt, fm_dtype_t block_dt, const LnArgs& a, hipStream_t stream) {
  if (stream_dt == FM_F32) {
    if (block_dt == FM_F32) launch_fwd<E, F32, F32>(a, stream);
    else launch_fwd<E, F32, E>(a, stream);
  } else {
    if (block_dt == FM_F32) launch_fwd<E, E, F32>(a, stream);
    else launch_fwd<E, E, E>(a, stream);
  }
}

}  // namespace

fm_status_t check_layer_norm(fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt, int64_t M,
                             int64_t N, float p, const uint64_t* rng, int64_t row_begin) {
  const fm_status_t st = check_norm(dt, stream_dt, block_dt, M, N, nullptr, 0);
  return st != FM_OK ? st : check_dropout(p, rng, M, row_begin, N, 0);
}

}  // namespace fm

using namespace fm;

extern "C" fm_status_t fm_layer_norm(fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt,
                                     int64_t M, int64_t N, const void* block, const void* resid,
                                     const void* bias, const void* w, const void* b, float p,
                                     const uint64_t* rng, int64_t draw, int64_t row_begin,
                                     float eps, void* out, void* y, float* y_scale, float* mean,
                                     float* rstd, hipStream_t stream) {
  const fm_status_t st = check_layer_norm(dt, stream_dt, block_dt, M, N, p, rng, row_begin);
  if (st != FM_OK) return st;
  if (!(eps >= 0.f)) return FM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return FM_OK;   // an empty batch's tensors have no addresses
  if ((w == nullptr) != (y == nullptr) || (!w && (b || y_scale || mean || rstd)))
    return FM_ERR_INVALID_ARG;
  if ((!block && (bias || p > 0.f)) || (!block && !resid) || (!out && !y))
    return FM_ERR_INVALID_ARG;
  for (const void* v : {block, resid, bias, w, b, (const void*)out, (const void*)y})
    if (!aligned16(v)) return FM_ERR_INVALID_ARG;
  if (!aligned4(y_scale) || !aligned4(mean) || !aligned4(rstd)) return FM_ERR_INVALID_ARG;
  LnArgs a = {};
  a.block = block;
  a.resid = resid;
  a.bias = bias;
  a.w = w;
  a.b = b;
  a.out = out;
  a.y = y;
  a.y_scale = y_scale;
  a.mean = mean;
  a.rstd = rstd;
  a.M = M;
  a.N = (int)N;
  a.eps = eps;
  a.d = make_dropout(p, rng, draw, row_begin, 0);
  if (dt == FM_F16) launch_types<F16>(stream_dt, block_dt, a, stream);
  else launch_types<BF16>(stream_dt, block_dt, a, stream);
  return launch_status();
}
