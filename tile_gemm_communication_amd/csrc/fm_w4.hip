// fm_w4.hip -- products with 4-bit weights and group scales for few rows: the
// dense shard, and the two matrices of each local expert of a MoE layer.
//
// With a handful of rows the weights are all there is to read, so the kernel is
// built to stream them: a block owns 16 columns, its waves share K, and every
// lane's 16-byte load is the B operand of four 16x16x32 matrix instructions.
// A code c enters the matrix core exactly, without a conversion, as the 16-bit
// number base + c, whose bit pattern is the code shifted into a constant's
// mantissa (bf16: base 16, fp16: base 64).  With t = sum x (base + c) and
// S = sum x over one group of K (a matrix product with ones),
//   sum x (c - zero) scale = scale * (t - (base + zero) * S),
// so that scale and zero cost two fused multiply-adds a group and output.
#include <algorithm>

#include "fm_wave.hpp"

namespace fm {
namespace {

constexpr int kW4Waves = 8;
constexpr int kW4Threads = 64 * kW4Waves;
constexpr int kW4MaxExperts = 64;

__device__ __forceinline__ f32x4 mfma16(F16, u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(BF16, u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight codes of a word as base + code, pair i holding nibbles i and i + 4.
__device__ __forceinline__ u32x4 codes8(BF16, uint32_t w) {
  constexpr uint32_t mask = 0x00780078u, base = 0x41804180u;   // 16, ulp 1/8
  return {((w << 3) & mask) | base, ((w >> 1) & mask) | base, ((w >> 5) & mask) | base,
          ((w >> 9) & mask) | base};
}
__device__ __forceinline__ u32x4 codes8(F16, uint32_t w) {
  constexpr uint32_t mask = 0x00F000F0u, base = 0x54005400u;   // 64, ulp 1/16
  return {((w << 4) & mask) | base, (w & mask) | base, ((w >> 4) & mask) | base,
          ((w >> 8) & mask) | base};
}
__device__ constexpr float code_base(BF16) { return 16.f; }
__device__ constexpr float code_base(F16) { return 64.f; }
__device__ constexpr uint32_t ones2(BF16) { return 0x3F803F80u; }
__device__ constexpr uint32_t ones2(F16) { return 0x3C003C00u; }

enum W4Mode { kDense16, kDense32, kGather, kScatter };

struct W4Args {
  const void* x;
  const uint8_t* packed;
  const void* scales;
  const uint8_t* zeros;
  void* out;
  const int32_t* pairs;
  const int32_t* offsets;
  const float* weights;
  int64_t M;
  int N, K;
  int blocks;    // 128-wide blocks of K
  int groups;
  int topk, act;
};

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

// What one step of 128 k reads: the lane's 32 codes, its rows' x, and the scale
// and zero of its column's groups.
template <typename E, int GB, int MT>
struct W4Step {
  u32x4 w;
  u32x4 x[MT][4];
  typename Elem<E>::type s[4 / GB];
  uint8_t z[4 / GB];
};

// GB: 32-wide matrix instructions of a group.  A chunk of rows is MT * R * 4:
// logical row (mt R + r) 4 + q is operand row 4 q + r, so that with few rows
// only accumulator r < R of every lane is in use.  PF steps are in flight.
template <typename E, int GB, int MT, int R, int PF, W4Mode MODE>
__global__ __launch_bounds__(kW4Threads) void w4_product(const W4Args a) {
  typedef typename Elem<E>::type L;
  constexpr int GP = 4 / GB;
  constexpr int ROWS = MT * R * 4;
  __shared__ float s_part[kW4Waves][MT * R][64];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int i16 = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int n = min(n0 + i16, a.N - 1);
  const int e = MODE == kGather || MODE == kScatter ? blockIdx.y : 0;
  int64_t first = 0, rows = a.M;
  if (MODE == kGather || MODE == kScatter) {
    first = a.offsets[e];
    rows = a.offsets[e + 1] - first;
    if (rows <= 0) return;
  }
  const uint8_t* wp = a.packed + ((int64_t)e * a.N + n) * a.blocks * 64 + q * 16;
  const int64_t sbase = (int64_t)e * a.groups * a.N + n;
  const L* sp = static_cast<const L*>(a.scales) + sbase;
  const uint8_t* zp = a.zeros ? a.zeros + sbase : nullptr;
  const int per = (a.blocks + kW4Waves - 1) / kW4Waves;
  const int s0 = wave * per, s1 = min(a.blocks, s0 + per);
  constexpr uint32_t one = ones2(E());
  const u32x4 ones = {one, one, one, one};

  for (int64_t m0 = MODE <= kDense32 ? (int64_t)blockIdx.z * ROWS : 0; m0 < rows;
       m0 += MODE <= kDense32 ? (int64_t)gridDim.z * ROWS : ROWS) {
    const L* xp[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int64_t m = m0 + (mt * R + (i16 & 3)) * 4 + (i16 >> 2);
      xp[mt] = nullptr;
      if ((i16 & 3) < R && m < rows) {
        int64_t row = first + m;
        if (MODE == kGather) row = a.pairs[row] / a.topk;
        xp[mt] = static_cast<const L*>(a.x) + row * a.K + q * 8;
      }
    }
    auto load = [&](W4Step<E, GB, MT>& f, int s) {
      f.w = *reinterpret_cast<const u32x4*>(wp + (int64_t)s * 64);
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        const int64_t at = (int64_t)min(s * GP + g, a.groups - 1) * a.N;
        f.s[g] = sp[at];
        f.z[g] = zp ? zp[at] : 8;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = s * 128 + j * 32;
          f.x[mt][j] = u32x4{0, 0, 0, 0};
          if (xp[mt] && k + q * 8 < a.K)
            f.x[mt][j] = *reinterpret_cast<const u32x4*>(xp[mt] + k);
        }
    };
    f32x4 acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto use = [&](const W4Step<E, GB, MT>& f) {
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        f32x4 tt[MT], xs[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) tt[mt] = xs[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < GB; ++b) {
          const int j = g * GB + b;
          const u32x4 c = codes8(E(), f.w[j]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            tt[mt] = mfma16(E(), f.x[mt][j], c, tt[mt]);
            xs[mt] = mfma16(E(), f.x[mt][j], ones, xs[mt]);
          }
        }
        const float scale = (float)f.s[g], off = -(code_base(E()) + (float)f.z[g]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < R; ++r)
            acc[mt][r] = fmaf(scale, fmaf(off, xs[mt][r], tt[mt][r]), acc[mt][r]);
      }
    };
    W4Step<E, GB, MT> ring[PF];
#pragma unroll
    for (int p = 0; p < PF; ++p)
      if (s0 + p < s1) load(ring[p], s0 + p);
    for (int s = s0; s < s1; s += PF) {
#pragma unroll
      for (int p = 0; p < PF; ++p)
        if (s + p < s1) {
          use(ring[p]);
          if (s + p + PF < s1) load(ring[p], s + p + PF);
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < R; ++r) s_part[wave][mt * R + r][lane] = acc[mt][r];
    __syncthreads();
    for (int o = t; o < MT * R * 64; o += kW4Threads) {
      const int l = o & 63, tile = o >> 6;
      const int64_t m = m0 + tile * 4 + (l >> 4);
      const int col = n0 + (l & 15);
      if (m < rows && col < a.N) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kW4Waves; ++w) v += s_part[w][tile][l];
        if (MODE == kScatter) {
          const int64_t p = a.pairs[first + m];
          static_cast<float*>(a.out)[p * a.N + col] = v * a.weights[p];
        } else if (MODE == kDense32) {
          static_cast<float*>(a.out)[m * a.N + col] = v;
        } else {
          if (MODE == kGather) v = activate(v, a.act);
          static_cast<L*>(a.out)[(first + m) * a.N + col] = (L)v;
        }
      }
    }
    __syncthreads();
  }
}

// out[t] = add[t] + sum of the weighted rows of t's local pairs, in the order of k.
__global__ __launch_bounds__(256) void w4_join(int64_t T, int n4, int topk, int e0, int n_local,
                                               const int32_t* __restrict__ ids,
                                               const f32x4* __restrict__ rows, const f32x4* add,
                                               f32x4* out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < T * n4;
       i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / n4;
    const int c = (int)(i - t * n4);
    f32x4 v = add ? add[i] : f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < topk; ++k) {
      const int64_t p = t * topk + k;
      const int e = ids[p] - e0;
      if (e >= 0 && e < n_local) v += rows[p * n4 + c];
    }
    out[i] = v;
  }
}

// One thread a packed word; neighbours take neighbouring columns.
__global__ __launch_bounds__(256) void w4_pack(int64_t n_matrices, int64_t K, int64_t N,
                                               int64_t blocks, const uint8_t* __restrict__ codes,
                                               uint32_t* __restrict__ packed) {
  const int64_t words = blocks * 16, total = n_matrices * words * N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t n = i % N, w = i / N % words, mat = i / N / words;
    const int64_t k0 = w / 16 * 128 + w % 4 * 32 + w % 16 / 4 * 8;
    uint32_t v = 0;
    for (int p = 0; p < 8; ++p) {
      const int64_t k = k0 + (p < 4 ? 2 * p : 2 * p - 7);
      if (k < K) v |= (uint32_t)(codes[(mat * K + k) * N + n] & 15) << (4 * p);
    }
    packed[(mat * N + n) * words + w] = v;
  }
}

template <typename E, int GB, W4Mode MODE>
void launch_rows(const W4Args& a, int64_t most, dim3 grid, hipStream_t stream) {
#define FM_W4(MT, R, PF)                                                                    \
  do {                                                                                      \
    if (MODE <= kDense32)                                                                   \
      grid.z = (unsigned)std::min<int64_t>(cdiv(a.M, MT * R * 4), 65535);                   \
    hipLaunchKernelGGL((w4_product<E, GB, MT, R, PF, MODE>), grid, dim3(kW4Threads), 0, stream, \
                       a);                                                                  \
  } while (0)
  if (most <= 4) FM_W4(1, 1, 3);
  else if (most <= 16) FM_W4(1, 4, 3);
  else FM_W4(2, 4, 2);
#undef FM_W4
}

// most: the rows that a chunk is chosen for.
template <W4Mode MODE>
void launch_w4(fm_dtype_t dt, int group, const W4Args& a, int64_t most, int n_local,
               hipStream_t stream) {
  const dim3 grid((unsigned)cdiv(a.N, 16), (unsigned)n_local, 1);
  if (dt == FM_F16) {
    if (group == 32) launch_rows<F16, 1, MODE>(a, most, grid, stream);
    else if (group == 64) launch_rows<F16, 2, MODE>(a, most, grid, stream);
    else launch_rows<F16, 4, MODE>(a, most, grid, stream);
  } else {
    if (group == 32) launch_rows<BF16, 1, MODE>(a, most, grid, stream);
    else if (group == 64) launch_rows<BF16, 2, MODE>(a, most, grid, stream);
    else launch_rows<BF16, 4, MODE>(a, most, grid, stream);
  }
}

int64_t row_bytes(int64_t K) { return cdiv(K, 128) * 64; }

fm_status_t check_w4(fm_dtype_t dt, int64_t N, int64_t K, int group, const void* x,
                     const void* packed, const void* scales, bool work) {
  if (dt != FM_F16 && dt != FM_BF16) return FM_ERR_UNSUPPORTED;
  if (N < 0 || K < 0 || N % 8 || K % 8) return FM_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return FM_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(packed) || !aligned16(scales)) return FM_ERR_INVALID_ARG;
  if (work && K > 0 && (!x || !packed || !scales)) return FM_ERR_INVALID_ARG;
  if (N >= (1ll << 22) || K >= (1ll << 22)) return FM_ERR_UNSUPPORTED;
  return FM_OK;
}

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" size_t fm_w4_row_bytes(int64_t K) { return K < 0 ? 0 : (size_t)row_bytes(K); }

extern "C" fm_status_t fm_w4_pack(int64_t n_matrices, int64_t K, int64_t N, const uint8_t* codes,
                                  void* packed, hipStream_t stream) {
  if (n_matrices < 0 || K < 0 || N < 0 || K % 8 || N % 8) return FM_ERR_INVALID_ARG;
  if (n_matrices >= (1ll << 20) || K >= (1ll << 22) || N >= (1ll << 22)) return FM_ERR_UNSUPPORTED;
  if (n_matrices == 0 || K == 0 || N == 0) return FM_OK;
  if (!codes || !packed || !aligned16(packed)) return FM_ERR_INVALID_ARG;
  const int64_t total = n_matrices * (row_bytes(K) / 4) * N;
  hipLaunchKernelGGL(w4_pack, dim3((unsigned)std::min<int64_t>(cdiv(total, 256), 65536)), dim3(256),
                     0, stream, n_matrices, K, N, cdiv(K, 128), codes,
                     static_cast<uint32_t*>(packed));
  return launch_status();
}

extern "C" fm_status_t fm_gemm_w4(fm_dtype_t ab, fm_dtype_t c, int64_t M, int64_t N, int64_t K,
                                  int32_t group, const void* A, const void* packed,
                                  const void* scales, const uint8_t* zeros, void* C,
                                  hipStream_t stream) {
  if (c != ab && c != FM_F32) return FM_ERR_UNSUPPORTED;
  const fm_status_t st = check_w4(ab, N, K, group, A, packed, scales, M > 0 && N > 0);
  if (st != FM_OK) return st;
  if (M < 0 || !aligned16(C)) return FM_ERR_INVALID_ARG;
  if (M >= (1ll << 31)) return FM_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return FM_OK;
  if (!C) return FM_ERR_INVALID_ARG;
  W4Args a = {};
  a.x = A;
  a.packed = static_cast<const uint8_t*>(packed);
  a.scales = scales;
  a.zeros = zeros;
  a.out = C;
  a.M = M;
  a.N = (int)N;
  a.K = (int)K;
  a.blocks = (int)cdiv(K, 128);
  a.groups = (int)cdiv(K, group);
  if (c == FM_F32) launch_w4<kDense32>(ab, group, a, M, 1, stream);
  else launch_w4<kDense16>(ab, group, a, M, 1, stream);
  return launch_status();
}

extern "C" fm_status_t fm_moe_gather_gemm_w4(
    fm_dtype_t dt, int64_t T, int64_t hidden, int64_t ffn, int32_t topk, int32_t expert_begin,
    int32_t n_local, int32_t group, const void* X, const int32_t* topk_ids, const void* packed,
    const void* scales, const uint8_t* zeros, void* H, int32_t* sorted_pairs,
    int32_t* expert_offsets, fm_act_t act, void* ws, size_t ws_bytes, hipStream_t stream) {
  if ((int)act < FM_ACT_NONE || (int)act > FM_ACT_SILU) return FM_ERR_INVALID_ARG;
  fm_status_t st = check_w4(dt, ffn, hidden, group, X, packed, scales, T > 0 && ffn > 0);
  if (st != FM_OK) return st;
  if (T > 0 && ffn > 0 && (!H || !aligned16(H))) return FM_ERR_INVALID_ARG;
  st = fm_moe_route(T, topk, expert_begin, n_local, topk_ids, sorted_pairs, expert_offsets, ws,
                    ws_bytes, stream);
  if (st != FM_OK || T == 0 || ffn == 0) return st;
  W4Args a = {};
  a.x = X;
  a.packed = static_cast<const uint8_t*>(packed);
  a.scales = scales;
  a.zeros = zeros;
  a.out = H;
  a.pairs = sorted_pairs;
  a.offsets = expert_offsets;
  a.N = (int)ffn;
  a.K = (int)hidden;
  a.blocks = (int)cdiv(hidden, 128);
  a.groups = (int)cdiv(hidden, group);
  a.topk = topk;
  a.act = act;
  launch_w4<kGather>(dt, group, a, cdiv(2 * T * topk, n_local), n_local, stream);
  return launch_status();
}

extern "C" size_t fm_moe_w4_workspace_bytes(int64_t T, int32_t topk, int64_t hidden) {
  if (T < 0 || topk < 1 || hidden < 0 || hidden % 8) return 0;
  return (size_t)std::max<int64_t>(T * topk * hidden * 4, 256);
}

extern "C" fm_status_t fm_moe_gemm_scatter_w4(
    fm_dtype_t dt, int64_t T, int64_t hidden, int64_t ffn, int32_t topk, int32_t expert_begin,
    int32_t n_local, int32_t group, const void* H, const void* packed, const void* scales,
    const uint8_t* zeros, const int32_t* topk_ids, const int32_t* sorted_pairs,
    const int32_t* expert_offsets, const float* topk_weights, const float* add, float* out,
    void* ws, size_t ws_bytes, hipStream_t stream) {
  const fm_status_t st = check_w4(dt, hidden, ffn, group, H, packed, scales, T > 0 && hidden > 0);
  if (st != FM_OK) return st;
  if (T < 0 || topk < 1 || n_local < 1 || n_local > kW4MaxExperts) return FM_ERR_INVALID_ARG;
  if (T * topk >= (1ll << 31)) return FM_ERR_UNSUPPORTED;
  if (T == 0 || hidden == 0) return FM_OK;
  if (!topk_ids || !sorted_pairs || !expert_offsets || !topk_weights || !out || !aligned16(out) ||
      !aligned16(add) || !ws || !aligned16(ws) ||
      ws_bytes < fm_moe_w4_workspace_bytes(T, topk, hidden))
    return FM_ERR_INVALID_ARG;
  W4Args a = {};
  a.x = H;
  a.packed = static_cast<const uint8_t*>(packed);
  a.scales = scales;
  a.zeros = zeros;
  a.out = ws;
  a.pairs = sorted_pairs;
  a.offsets = expert_offsets;
  a.weights = topk_weights;
  a.N = (int)hidden;
  a.K = (int)ffn;
  a.blocks = (int)cdiv(ffn, 128);
  a.groups = (int)cdiv(ffn, group);
  a.topk = topk;
  launch_w4<kScatter>(dt, group, a, cdiv(2 * T * topk, n_local), n_local, stream);
  const int n4 = (int)(hidden / 4);
  hipLaunchKernelGGL(w4_join, dim3((unsigned)std::min<int64_t>(cdiv(T * n4, 256), 65536)), dim3(256),
                     0, stream, T, n4, (int)topk, (int)expert_begin, (int)n_local, topk_ids,
                     static_cast<const f32x4*>(ws), reinterpret_cast<const f32x4*>(add),
                     reinterpret_cast<f32x4*>(out));
  return launch_status();
}
