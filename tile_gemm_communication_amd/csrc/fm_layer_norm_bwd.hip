// fm_layer_norm_bwd.hip -- gradients of fm_layer_norm.
//
// One pass over the rows gives d_resid and d_block and, in registers, each lane's
// share of the three column sums (bias and both norm weights).  A block holds RW rows
// of TH lanes at a time, the row lanes of all blocks taking rows in turn; at its end
// the block writes one partial row a sum, and a second launch joins the partial
// rows in order (no atomics: the same bits on every call).  Bound by the bytes of the
// [M, N] arrays: 16384 x 4096 bf16 130 us, 5.2 TB/s, 4 of it the join; 4088 x 12288 fp32
// 192 us, 4.7 TB/s, 8 of it the join; 61 x 2816 8.8 us, two launches.
#include <algorithm>

#include "fm_layer_norm.hpp"

namespace fm {
namespace {

constexpr int kLnBwdBlocks = 256;   // one a compute unit

struct LnBwdArgs {
  const void *d_y, *d_out, *out, *w;
  const float *mean, *rstd;
  void *d_resid, *d_block;
  float *part_bias, *part_w, *part_b;   // [blocks, N], NULL if not wanted
  int64_t M;
  int N;
  Dropout d;
};

// The registers' values as far as the compiler knows: what was made of them before
// is not kept beside them.
template <typename E>
__device__ __forceinline__ void hold(Raw8<E>& v) {
  for (u32x4& r : v.r) asm("" : "+v"(r));
}

template <int TH>
constexpr int ln_rows() { return TH == 768 ? 1 : 1024 / TH; }

template <typename E, typename S, typename B, int TH, int CH>
__global__ __launch_bounds__(TH == 768 ? 768 : 1024) void layer_norm_bwd(const LnBwdArgs a) {
  constexpr int RW = ln_rows<TH>();
  constexpr f32x4 kZero = {0.f, 0.f, 0.f, 0.f};
  __shared__ f32x2 s_red[2][RW][(TH + 63) / 64];
  // Rows from 8200 elements on keep their sums in LDS, each lane's in places of its own; the
  // registers hold the next row instead, which is on its way while this one is worked on
  // (the wait for it, at the row's end, is also one for this row's stores).
  // 1024 lanes have 128 registers each: the longest rows (from 12296 on) do without that,
  // and read d_out behind the barrier; of their sums LDS holds two.
  constexpr bool kRoom = CH == 1, kAhead = TH * CH < 2048, kBiasRoom = kRoom || !kAhead;
  // joins the row lanes' sums, or holds the lanes' own
  __shared__ f32x4 s_acc[!kRoom ? (kBiasRoom ? 2 : 3) * TH * CH * 2 : RW > 1 ? RW * TH * CH * 2 : 1];
  const int t = threadIdx.x % TH, N = a.N;
  const int rw = row_lane<TH>();
  const int64_t parts = (int64_t)gridDim.x * RW, part = (int64_t)blockIdx.x * RW + rw;
  // row lanes take rows in turn, so that the rows in work lie side by side (each walking its
  // own stretch, equally far apart in memory: 16384 x 4096 145 us, so 131); all take part in the
  // barriers of the longest
  const int64_t count = (a.M + parts - 1) / parts;
  const float invN = 1.f / (float)N;
  const bool has_d = a.d_block || a.part_bias;
  Philox p = {};
  if (a.d.rng) p = philox_of(a.d);
  f32x4 acc_w[CH][2], acc_b[CH][2], acc_bias[CH][2];
  Raw8<E> w[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      acc_w[c][h] = acc_b[c][h] = acc_bias[c][h] = kZero;
      if (!kRoom) s_acc[(c * 2 + h) * TH + t] = s_acc[((CH + c) * 2 + h) * TH + t] = kZero;
      if (!kBiasRoom) s_acc[((2 * CH + c) * 2 + h) * TH + t] = kZero;
    }
    w[c] = {};
    if (a.w && (c * TH + t) * 8 < N) w[c] = raw8<E>(a.w, (c * TH + t) * 8);
  }

  // rows are held as they came and widened in both passes: half the registers
  struct Row {
    Raw8<E> d_y[CH];
    Raw8<S> out[CH], d_out[CH];
    float mean, rstd;
  };
  auto load = [&](int64_t i) {
    Row v = {};
    const int64_t row = part + i * parts, at = row * N;
    const bool live = row < a.M;
    if (live && a.w) {
      v.mean = a.mean[row];
      v.rstd = a.rstd[row];
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = (c * TH + t) * 8;
      if (!live || e >= N) continue;
      if (a.w) {
        v.d_y[c] = raw8<E>(a.d_y, at + e);
        v.out[c] = raw8<S>(a.out, at + e);
      }
      if (kAhead && a.d_out) v.d_out[c] = raw8<S>(a.d_out, at + e);
    }
    return v;
  };

  Row next = load(0);
  for (int64_t i = 0; i < count; ++i) {
    const int64_t row = part + i * parts;
    const bool live = row < a.M;
    const int64_t at = row * N;
    Row v = next;
    if (kAhead) next = load(i + 1);
    const float r = v.rstd, mean = v.mean;
    // dz = r * (t - mean(t) - hat * mean(t hat)) + d_out, t = d_y w
    float s1 = 0.f, s2 = 0.f;
    if (a.w) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if ((c * TH + t) * 8 >= N) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 dy = half8<E>(v.d_y[c], h), hat = (half8<S>(v.out[c], h) - mean) * r;
          const f32x4 q = dy * half8<E>(w[c], h);
          if (kRoom) {
            acc_b[c][h] += dy;
            acc_w[c][h] += dy * hat;
          } else {
            s_acc[(c * 2 + h) * TH + t] += dy;
            s_acc[((CH + c) * 2 + h) * TH + t] += dy * hat;
          }
          s1 += (q[0] + q[1]) + (q[2] + q[3]);
          s2 += dot4(q, hat);
        }
      }
      s1 = group_sum<TH < 64 ? TH : 64>(s1);
      s2 = group_sum<TH < 64 ? TH : 64>(s2);
      if constexpr (TH > 64) {
        // the other slot is written before the next barrier: one barrier a row
        f32x2* slots = s_red[i & 1][rw];
        if (t % 64 == 0) slots[t / 64] = f32x2{s1, s2};
        __syncthreads();
        s1 = s2 = 0.f;
#pragma unroll
        for (int k = 0; k < TH / 64; ++k) {
          s1 += slots[k][0];
          s2 += slots[k][1];
        }
      }
      s1 *= invN;
      s2 *= invN;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = (c * TH + t) * 8;
      if (!live || e >= N) continue;
      if (!kAhead && a.d_out) v.d_out[c] = raw8<S>(a.d_out, at + e);
      hold(v.d_y[c]);
      hold(v.out[c]);
      f32x4 dz[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        dz[h] = half8<S>(v.d_out[c], h);
        if (a.w) {
          const f32x4 hat = (half8<S>(v.out[c], h) - mean) * r;
          dz[h] += (half8<E>(v.d_y[c], h) * half8<E>(w[c], h) - s1 - hat * s2) * r;
        }
      }
      if (a.d_resid) store8<S>(static_cast<typename Elem<S>::type*>(a.d_resid) + at + e, dz);
      if (has_d) {
        if (a.d.rng) {
          const u32x4 k = philox(p, (uint32_t)(c * TH + t), a.d.row + (uint32_t)row);
          dz[0] = drop4(dz[0], k[0], k[1], a.d);
          dz[1] = drop4(dz[1], k[2], k[3], a.d);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (kBiasRoom) acc_bias[c][h] += dz[h];
          else s_acc[((2 * CH + c) * 2 + h) * TH + t] += dz[h];
        }
        if (a.d_block) store8<B>(static_cast<typename Elem<B>::type*>(a.d_block) + at + e, dz);
      }
    }
    if (!kAhead) next = load(i + 1);
  }
  auto flush = [&](f32x4 (&acc)[CH][2], float* to) {
    if (!to) return;
    if constexpr (RW > 1) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) s_acc[((rw * CH + c) * 2 + h) * TH + t] = acc[c][h];
      __syncthreads();
      if (rw == 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll 4
            for (int o = 1; o < RW; ++o) acc[c][h] += s_acc[((o * CH + c) * 2 + h) * TH + t];
      }
    }
    if (rw == 0) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int e = (c * TH + t) * 8;
        if (e < N) store8<F32>(to + (int64_t)blockIdx.x * N + e, acc[c]);
      }
    }
  };
  if constexpr (!kRoom) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        acc_b[c][h] = s_acc[(c * 2 + h) * TH + t];
        acc_w[c][h] = s_acc[((CH + c) * 2 + h) * TH + t];
        if (!kBiasRoom) acc_bias[c][h] = s_acc[((2 * CH + c) * 2 + h) * TH + t];
      }
  }
  flush(acc_bias, a.part_bias);
  flush(acc_w, a.part_w);
  flush(acc_b, a.part_b);
}

struct LnJoinArgs {
  const float* part[3];   // [rows, N] each
  float* to[3];
  int rows, N;
};

// Column sums of the partial rows, blockIdx.x which: 64 columns (16 lanes of four) and 16
// slices of the rows a block, joined in order.
__global__ __launch_bounds__(256) void layer_norm_join(const LnJoinArgs a) {
  __shared__ f32x4 s[16][16];
  const int col = (int)threadIdx.x % 16, slice = threadIdx.x / 16, e = blockIdx.y * 64 + col * 4;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if (e < a.N) {
    const float* p = a.part[blockIdx.x] + e;
#pragma unroll 8
    for (int r = slice; r < a.rows; r += 16) sum += *reinterpret_cast<const f32x4*>(p + (int64_t)r * a.N);
  }
  s[slice][col] = sum;
  __syncthreads();
  if (slice == 0 && e < a.N) {
#pragma unroll
    for (int i = 1; i < 16; ++i) sum += s[i][col];
    *reinterpret_cast<f32x4*>(a.to[blockIdx.x] + e) = sum;
  }
}

int64_t rows_of_block(int64_t N) {
  int64_t rows = 1;
#define FM_LN_ROWS(TH, CH) rows = ln_rows<TH>()
  FM_LN_SIZES(N, FM_LN_ROWS);
#undef FM_LN_ROWS
  return rows;
}

int64_t blocks_of(int64_t M, int64_t N) {
  return std::min<int64_t>(cdiv(M, rows_of_block(N)), kLnBwdBlocks);
}

size_t ln_ws(int64_t M, int64_t N) { return (size_t)blocks_of(M, N) * N * 4 * 3; }

template <typename E, typename S, typename B>
void launch_bwd(const LnBwdArgs& a, int64_t blocks, hipStream_t stream) {
#define FM_LN_BWD(TH, CH)                                                     \
  hipLaunchKernelGGL((layer_norm_bwd<E, S, B, TH, CH>), dim3((unsigned)blocks), \
                     dim3(TH == 768 ? 768 : 1024), 0, stream, a)
  FM_LN_SIZES(a.N, FM_LN_BWD);
#undef FM_LN_BWD
}

template <typename E>
void launch_types(fm_dtype_t stream_dt, fm_dtype_t block_dt, const LnBwdArgs& a, int64_t blocks,
                  hipStream_t stream) {
  if (stream_dt == FM_F32) {
    if (block_dt == FM_F32) launch_bwd<E, F32, F32>(a, blocks, stream);
    else launch_bwd<E, F32, E>(a, blocks, stream);
  } else {
    if (block_dt == FM_F32) launch_bwd<E, E, F32>(a, blocks, stream);
    else launch_bwd<E, E, E>(a, blocks, stream);
  }
}

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" size_t fm_layer_norm_workspace_bytes(int64_t M, int64_t N) {
  if (M < 0 || N < 0 || N % 8 || N > kNormMaxN || M >= (1ll << 31)) return 0;
  return std::max<size_t>(ln_ws(M, N), 256);
}

extern "C" fm_status_t fm_layer_norm_bwd(fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt,
                                         int64_t M, int64_t N, const void* d_y, const void* d_out,
                                         const void* out, const float* mean, const float* rstd,
                                         const void* w, float p, const uint64_t* rng,
                                         int64_t draw, int64_t row_begin, void* d_resid,
                                         void* d_block, float* d_bias, float* d_w, float* d_b,
                                         void* ws, size_t ws_bytes, hipStream_t stream) {
  const fm_status_t st = check_layer_norm(dt, stream_dt, block_dt, M, N, p, rng, row_begin);
  if (st != FM_OK) return st;
  for (const void* v : {d_y, d_out, out, w, (const void*)d_resid, (const void*)d_block,
                        (const void*)d_bias, (const void*)d_w, (const void*)d_b, (const void*)ws})
    if (!aligned16(v)) return FM_ERR_INVALID_ARG;
  if (!aligned4(mean) || !aligned4(rstd)) return FM_ERR_INVALID_ARG;
  const bool sums = d_bias || d_w || d_b;
  if (N > 0 && sums && (!ws || ws_bytes < ln_ws(M, N))) return FM_ERR_INVALID_ARG;
  if (N == 0) return FM_OK;
  LnBwdArgs a = {};
  const int64_t blocks = blocks_of(M, N);
  if (M > 0) {   // (an empty batch's tensors have no addresses)
    if (!d_resid && !d_block && !sums) return FM_ERR_INVALID_ARG;
    if ((w == nullptr) != (d_y == nullptr) || (w && (!out || !mean || !rstd)) ||
        (!w && (!d_out || d_w || d_b)))
      return FM_ERR_INVALID_ARG;
    a.d_y = d_y;
    a.d_out = d_out;
    a.out = out;
    a.w = w;
    a.mean = mean;
    a.rstd = rstd;
    a.d_resid = d_resid;
    a.d_block = d_block;
    a.M = M;
    a.N = (int)N;
    a.d = make_dropout(p, rng, draw, row_begin, 0);
  }
  float* part = static_cast<float*>(ws);
  LnJoinArgs j = {};
  j.rows = (int)blocks;
  j.N = (int)N;
  int n = 0;
  auto want = [&](float* to, float*& slot) {
    if (!to) return;
    slot = part;
    j.part[n] = part;
    j.to[n++] = to;
    part += blocks * N;
  };
  want(d_bias, a.part_bias);
  want(d_w, a.part_w);
  want(d_b, a.part_b);
  if (M == 0 && n == 0) return FM_OK;
  if (M > 0) {
    if (dt == FM_F16) launch_types<F16>(stream_dt, block_dt, a, blocks, stream);
    else launch_types<BF16>(stream_dt, block_dt, a, blocks, stream);
  }
  if (n > 0) hipLaunchKernelGGL(layer_norm_join, dim3(n, (unsigned)cdiv(N, 64)), dim3(256), 0, stream, j);
  return launch_status();
}
