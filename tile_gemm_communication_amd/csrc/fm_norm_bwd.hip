// fm_norm_bwd.hip -- gradients of fm_norm_residual.
//
// One pass over the rows gives d_resid and d_block and, in registers, each
// lane's share of the three column sums (both norm weights, the gate).  A block
// keeps 1024 lanes: RW rows of TH lanes at a time, each row lane walking its own
// contiguous rows; at its end the block writes one partial row a sum, and a
// second launch joins the partial rows in order (no atomics: the same bits on
// every call).  Bound by the bytes of the four to six [M, N] arrays: 4088 x 12288
// fp16 with fp32 stream and block 241 us, 4.6 TB/s, and 10 us for the join.
#include <algorithm>

#include "fm_norm.hpp"

namespace fm {
namespace {

constexpr int kBwdThreads = 1024;
constexpr int kBwdBlocks = 256;   // one a compute unit

struct NormBwdArgs {
  const void *d_y, *d_out, *out, *block, *w_post, *w_pre, *gate;
  const float *rstd_post, *rstd_pre;
  void *d_resid, *d_block;
  float* d_gate;                              // written here where whole groups are walked
  float *part_post, *part_pre, *part_gate;    // [blocks, N], NULL if not wanted
  int64_t M;
  int N;
  int64_t rows_per_gate, n_gates;
  int split;                                  // blocks of one gate group; 0: whole groups
  float scale;
};

// Rows [first, last) of row lane rw of block bid: the blocks of a group share its
// rows, or (split = 0) all row lanes share the groups.
struct RowRange {
  int64_t first, last;
};

__host__ __device__ inline RowRange rows_of(const NormBwdArgs& a, int64_t blocks, int64_t bid,
                                            int rw, int RW) {
  if (a.split) {
    const int64_t g = bid / a.split, j = (bid % a.split) * RW + rw, parts = (int64_t)a.split * RW;
    return {g * a.rows_per_gate + j * a.rows_per_gate / parts,
            g * a.rows_per_gate + (j + 1) * a.rows_per_gate / parts};
  }
  const int64_t i = bid * RW + rw, parts = blocks * RW;
  return {i * a.n_gates / parts * a.rows_per_gate, (i + 1) * a.n_gates / parts * a.rows_per_gate};
}

template <typename E, typename S, typename B, int TH, int CH>
__global__ __launch_bounds__(kBwdThreads) void norm_bwd(const NormBwdArgs a) {
  constexpr int RW = kBwdThreads / TH;
  constexpr f32x4 kZero = {0.f, 0.f, 0.f, 0.f};
  // 1024 lanes have 128 registers each.  The longest rows keep one of the sums in
  // LDS and read block only behind the first exchange.
  constexpr bool kEarly = CH < 4;
  __shared__ float s_red[2][RW][TH / 64];
  // joins the row lanes' sums; for the longest rows it holds the lanes' sums of
  // d_w_pre, each in a place of its own
  __shared__ f32x4 s_acc[RW > 1 || !kEarly ? RW * TH * CH : 1];
  const int t = threadIdx.x % TH, rw = threadIdx.x / TH, N = a.N;
  const RowRange rr = rows_of(a, gridDim.x, blockIdx.x, rw, RW);
  const float invN = 1.f / (float)N;
  // every row lane takes part in the barriers of the longest
  int64_t count = rr.last - rr.first;
  if constexpr (TH > 64) {
    for (int i = 0; i < RW; ++i) {
      const RowRange o = rows_of(a, gridDim.x, blockIdx.x, i, RW);
      count = max(count, o.last - o.first);
    }
  }
  const bool has_block = a.d_block || a.part_post || a.part_gate || a.d_gate;
  f32x4 acc_pre[CH], acc_post[CH], acc_gate[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    acc_pre[c] = acc_post[c] = acc_gate[c] = kZero;
    if (!kEarly) s_acc[c * TH + t] = kZero;
  }

  for (int64_t i = 0; i < count; ++i) {
    const int64_t row = rr.first + i;
    const bool live = row < rr.last;
    const int64_t at = row * N;
    f32x4 dz[CH], hat[CH], b[CH];
    const float rp = live && a.w_pre ? a.rstd_pre[row] : 0.f;
    const float rb = live && a.w_post ? a.rstd_post[row] : 1.f;
    float s1 = 0.f;
    // the norm before: dz = rp * (t - hat * mean(t hat)) + d_out, t = d_y w_pre
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = (c * TH + t) * 4;
      const bool in = live && e < N;
      dz[c] = hat[c] = b[c] = kZero;
      if (kEarly && in && a.block)
        b[c] = load4<B>(static_cast<const typename Elem<B>::type*>(a.block) + at + e);
      if (in && a.w_pre) {
        const f32x4 dy = load4<E>(static_cast<const typename Elem<E>::type*>(a.d_y) + at + e);
        hat[c] = load4<S>(static_cast<const typename Elem<S>::type*>(a.out) + at + e) * rp;
        if (kEarly) acc_pre[c] += dy * hat[c];
        else s_acc[c * TH + t] += dy * hat[c];
        dz[c] = dy * widen<E>(raw4<E>(a.w_pre, e));
        s1 += dot4(dz[c], hat[c]);
      }
    }
    if (a.w_pre) {
      s1 = row_sum<TH>(s1, s_red[0][rw]) * invN;
#pragma unroll
      for (int c = 0; c < CH; ++c) dz[c] = (dz[c] - hat[c] * s1) * rp;
    }
    const uint32_t rpg = (uint32_t)a.rows_per_gate;
    const int64_t grp = a.gate && live ? (uint32_t)row / rpg : 0;
    float s2 = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = (c * TH + t) * 4;
      const bool in = live && e < N;
      if (in && a.d_out)
        dz[c] += load4<S>(static_cast<const typename Elem<S>::type*>(a.d_out) + at + e);
      if (in && a.d_resid) store4<S>(static_cast<typename Elem<S>::type*>(a.d_resid) + at + e, dz[c]);
      if (!kEarly && in && a.block)
        b[c] = load4<B>(static_cast<const typename Elem<B>::type*>(a.block) + at + e);
      if (in && has_block) {
        const f32x4 wq = a.w_post ? widen<E>(raw4<E>(a.w_post, e)) : f32x4{1.f, 1.f, 1.f, 1.f};
        b[c] *= rb;
        f32x4 d = dz[c] * a.scale;
        acc_gate[c] += d * (b[c] * wq);
        if (a.gate)
          d *= widen<E>(raw4<E>(static_cast<const typename Elem<E>::type*>(a.gate) + grp * N, e));
        acc_post[c] += d * b[c];
        dz[c] = d * wq;
        s2 += dot4(dz[c], b[c]);
      }
    }
    if (a.w_post && has_block) {
      s2 = row_sum<TH>(s2, s_red[1][rw]) * invN;
#pragma unroll
      for (int c = 0; c < CH; ++c) dz[c] = (dz[c] - b[c] * s2) * rb;
    }
    if (a.d_block) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int e = (c * TH + t) * 4;
        if (live && e < N)
          store4<B>(static_cast<typename Elem<B>::type*>(a.d_block) + at + e, dz[c]);
      }
    }
    if (a.d_gate && !a.split && live && ((uint32_t)row + 1) % rpg == 0) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int e = (c * TH + t) * 4;
        if (e < N) *reinterpret_cast<f32x4*>(a.d_gate + grp * N + e) = acc_gate[c];
        acc_gate[c] = kZero;
      }
    }
    // a slot is written again only behind the other norm's barrier
    if (TH > 64 && (a.w_pre != nullptr) != (a.w_post && has_block)) __syncthreads();
  }
  auto flush = [&](f32x4 (&acc)[CH], float* part) {
    if (!part) return;
    if constexpr (RW > 1) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < CH; ++c) s_acc[(rw * CH + c) * TH + t] = acc[c];
      __syncthreads();
      if (rw == 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
          for (int o = 1; o < RW; ++o) acc[c] += s_acc[(o * CH + c) * TH + t];
      }
    }
    if (rw == 0) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int e = (c * TH + t) * 4;
        if (e < N) *reinterpret_cast<f32x4*>(part + (int64_t)blockIdx.x * N + e) = acc[c];
      }
    }
  };
  if constexpr (!kEarly) {
#pragma unroll
    for (int c = 0; c < CH; ++c) acc_pre[c] = s_acc[c * TH + t];
  }
  flush(acc_post, a.part_post);
  flush(acc_pre, a.part_pre);
  flush(acc_gate, a.part_gate);
}

struct JoinArgs {
  const float* part[3];
  float* to[3];
  int64_t rows[3];   // partial rows of one result row
  int64_t N;
  int first[3];      // first blockIdx.x of each
};

// Column sums of the partial rows: a block takes 64 columns (16 lanes of four)
// and 64 slices of the rows, joined in order.
__global__ __launch_bounds__(1024) void norm_join(const JoinArgs a) {
  __shared__ f32x4 s[64][16];
  int w = 0;
  for (int i = 1; i < 3; ++i)
    if ((int)blockIdx.x >= a.first[i]) w = i;
  const int64_t g = (int)blockIdx.x - a.first[w];
  const int col = (int)threadIdx.x % 16, slice = threadIdx.x / 16;
  const int64_t e = (int64_t)blockIdx.y * 64 + col * 4;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if (e < a.N) {
    const float* p = a.part[w] + g * a.rows[w] * a.N + e;
#pragma unroll 4
    for (int64_t r = slice; r < a.rows[w]; r += 64)
      sum += *reinterpret_cast<const f32x4*>(p + r * a.N);
  }
  s[slice][col] = sum;
  __syncthreads();
  if (slice == 0 && e < a.N) {
    for (int i = 1; i < 64; ++i) sum += s[i][col];
    *reinterpret_cast<f32x4*>(a.to[w] + g * a.N + e) = sum;
  }
}

// Lanes of a row, 16384 rows: N = 256 with 64 lanes 20.8 us, 256 44; 512 34.6 and 45.6;
// 1024 with 256 lanes 65, 64 98; 4096 with 1024 lanes 254, 256 309.
int lanes_of(int64_t N) { return N <= 512 ? 64 : N <= 2048 ? 256 : 1024; }

struct Split {
  int64_t blocks;
  int split;   // blocks of a gate group, 0: every row lane walks whole groups
};

// Few groups are each shared by several blocks, whose partial gate rows are
// joined; from as many groups as row lanes on, each lane walks whole groups.  The blocks
// are whole numbers a group: 32768 rows of 4096 take 530 to 540 us with 128 or 256 groups,
// but 976 with 129 (as many blocks as groups on 256 units) and 947 with 257 (one block
// walks two).
Split split_of(int64_t M, int64_t N, int64_t n_gates) {
  const int64_t RW = kBwdThreads / lanes_of(N), G = std::max<int64_t>(n_gates, 1);
  if (G >= kBwdBlocks * RW || G == M) return {std::min<int64_t>(cdiv(G, RW), kBwdBlocks), 0};
  const int64_t per = std::max<int64_t>(1, kBwdBlocks / G);
  const int64_t s = std::min(per, cdiv(M / G, RW));
  return {G * s, (int)s};
}

size_t norm_ws(int64_t M, int64_t N, int64_t n_gates) {
  if (M == 0) return 0;
  return (size_t)split_of(M, N, n_gates).blocks * N * 4 * 3;
}

template <typename E, typename S, typename B>
void launch_bwd(const NormBwdArgs& a, int64_t blocks, hipStream_t stream) {
#define FM_BWD(TH, CH) \
  hipLaunchKernelGGL((norm_bwd<E, S, B, TH, CH>), dim3(blocks), dim3(kBwdThreads), 0, stream, a)
  const int N = a.N;
  if (N <= 256) FM_BWD(64, 1);
  else if (N <= 512) FM_BWD(64, 2);
  else if (N <= 1024) FM_BWD(256, 1);
  else if (N <= 2048) FM_BWD(256, 2);
  else if (N <= 4096) FM_BWD(1024, 1);
  else if (N <= 8192) FM_BWD(1024, 2);
  else if (N <= 12288) FM_BWD(1024, 3);
  else FM_BWD(1024, 4);
#undef FM_BWD
}

template <typename E>
void launch_types(fm_dtype_t stream_dt, fm_dtype_t block_dt, const NormBwdArgs& a, int64_t blocks,
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

extern "C" size_t fm_norm_residual_workspace_bytes(int64_t M, int64_t N, int64_t n_gates) {
  if (M < 0 || N < 0 || N % 8 || N > kNormMaxN || M >= (1ll << 31) || n_gates < 0 ||
      (M > 0 && n_gates > 0 && (n_gates > M || M % n_gates)))
    return 0;
  return std::max<size_t>(norm_ws(M, N, n_gates), 256);
}

extern "C" fm_status_t fm_norm_residual_bwd(
    fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt, int64_t M, int64_t N,
    const void* d_y, const void* d_out, const void* out, const void* block, const void* w_post,
    const void* w_pre, const void* gate, int64_t n_gates, float scale, const float* rstd_post,
    const float* rstd_pre, void* d_resid, void* d_block, float* d_w_post, float* d_w_pre,
    float* d_gate, void* ws, size_t ws_bytes, hipStream_t stream) {
  const fm_status_t st = check_norm(dt, stream_dt, block_dt, M, N, gate, n_gates);
  if (st != FM_OK) return st;
  if ((d_w_post && !w_post) || (d_w_pre && !w_pre) || (d_gate && !gate)) return FM_ERR_INVALID_ARG;
  if (M > 0 && N > 0 && !d_resid && !d_block && !d_w_post && !d_w_pre && !d_gate)
    return FM_ERR_INVALID_ARG;   // (an empty batch's tensors have no addresses)
  for (const void* p : {d_y, d_out, out, block, w_post, w_pre, gate, (const void*)d_resid,
                        (const void*)d_block, (const void*)d_w_post, (const void*)d_w_pre,
                        (const void*)d_gate, (const void*)ws})
    if (!aligned16(p)) return FM_ERR_INVALID_ARG;
  if (!aligned4(rstd_post) || !aligned4(rstd_pre)) return FM_ERR_INVALID_ARG;
  const bool sums = d_w_post || d_w_pre || d_gate;
  if (N > 0 && sums && (!ws || ws_bytes < norm_ws(M, N, n_gates))) return FM_ERR_INVALID_ARG;
  if (N == 0) return FM_OK;
  NormBwdArgs a = {};
  Split sp = {0, 0};
  if (M > 0) {
    if ((w_pre == nullptr) != (d_y == nullptr) || (w_pre && (!out || !rstd_pre)) ||
        (!w_pre && !d_out))
      return FM_ERR_INVALID_ARG;
    const bool need_b = d_gate || (w_post && (d_block || d_w_post));
    if ((need_b && !block) || (w_post && need_b && !rstd_post)) return FM_ERR_INVALID_ARG;
    sp = split_of(M, N, n_gates);
    a.d_y = d_y;
    a.d_out = d_out;
    a.out = out;
    // without them block, w_post and rstd_post have no part in what is wanted
    a.block = need_b ? block : nullptr;
    a.w_post = need_b ? w_post : nullptr;
    a.w_pre = w_pre;
    a.gate = gate;
    a.rstd_post = rstd_post;
    a.rstd_pre = rstd_pre;
    a.d_resid = d_resid;
    a.d_block = d_block;
    a.d_gate = d_gate;
    a.M = M;
    a.N = (int)N;
    a.n_gates = std::max<int64_t>(n_gates, 1);
    a.rows_per_gate = M / a.n_gates;
    a.split = sp.split;
    a.scale = scale;
  }
  // d_w_post [blocks, N], d_w_pre, d_gate, one after another
  float* part = static_cast<float*>(ws);
  JoinArgs j = {};
  int n = 0, y = 0;
  auto want = [&](float* to, float*& slot, int64_t groups, int64_t rows) {
    if (!to) return;
    slot = part;
    j.part[n] = part;
    j.to[n] = to;
    j.rows[n] = rows;
    j.first[n++] = y;
    part += sp.blocks * N;
    y += (int)groups;
  };
  want(d_w_post, a.part_post, 1, sp.blocks);
  want(d_w_pre, a.part_pre, 1, sp.blocks);
  if (d_gate && (M == 0 || sp.split)) want(d_gate, a.part_gate, n_gates, sp.split);
  for (int i = n; i < 3; ++i) j.first[i] = 0x7fffffff;
  j.N = N;
  if (M == 0 && n == 0) return FM_OK;
  if (M > 0) {
    if (dt == FM_F16) launch_types<F16>(stream_dt, block_dt, a, sp.blocks, stream);
    else launch_types<BF16>(stream_dt, block_dt, a, sp.blocks, stream);
  }
  if (n > 0)
    hipLaunchKernelGGL(norm_join, dim3(y, cdiv(N, 64)), dim3(1024), 0, stream, j);
  return launch_status();
}
