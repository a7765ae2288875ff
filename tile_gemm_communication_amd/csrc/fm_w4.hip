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
constexpr int64_t kFewRows = 16;   // mean rows of an expert up to which x goes through LDS

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
  int64_t M;     // rows of x
  int N, K;
  int blocks;    // 128-wide blocks of K
  int groups;
  int topk, act;
  int n_local;
  // a route inside the product: at most kW4Threads pairs
  const int32_t* ids;
  int32_t *pairs_out, *offsets_out;
  int n_pairs, e0;
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

// The column tile of a block: each XCD (blocks go to them in turn) takes
// neighbouring tiles, whose scales share cache lines.
__device__ __forceinline__ int column_tile() {
  const int b = blockIdx.x, n = gridDim.x, x = b & 7;
  return x * (n >> 3) + min(x, n & 7) + (b >> 3);
}

// Loads go through buffer resources: the lane's 32-bit offset stays as it is and
// the step's is a scalar, so that a load costs no address registers.  An offset
// past the resource reads 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)(uint32_t)bytes,
                                           kBufRsrcWord3);
}

// The weights of the columns from n0 of matrix e (up to 16 * NT of them), and the
// scales and zeros of the matrix.
struct W4Source {
  __amdgpu_buffer_rsrc_t w, s, z;
};

template <bool Z>
__device__ __forceinline__ W4Source source_of(const W4Args& a, int e, int n0, int columns) {
  const int64_t row = (int64_t)a.blocks * 64, scales = (int64_t)a.groups * a.N;
  const uint8_t* w = a.packed + ((int64_t)e * a.N + n0) * row;
  return {resource(w, min(columns, a.N - n0) * row),
          resource(static_cast<const char*>(a.scales) + e * scales * 2, scales * 2),
          resource(Z ? a.zeros + e * scales : nullptr, Z ? scales : 0)};
}

__device__ __forceinline__ u32x4 load_codes(const W4Source& src, uint32_t lane_offset, int step) {
  return __builtin_bit_cast(u32x4,
                            __builtin_amdgcn_raw_buffer_load_b128(src.w, lane_offset, step * 64, 0));
}

// A loaded value where it is first used.  Without this the optimizer moves what
// the loop's body and its remainder both compute from a load up to the load
// itself, where it waits for the data and holds the wider result.
__device__ __forceinline__ void loaded(u32x4& v) { asm volatile("" : "+v"(v)); }

// Scales and zeros of one 16-column tile and step of 128 k.
template <typename E, int GB, bool Z>
struct W4Scales {
  uint32_t s[4 / GB];            // the 16 bits of each scale
  uint32_t z[Z ? 4 / GB : 1];
  __device__ __forceinline__ void loaded() {
#pragma unroll
    for (int g = 0; g < 4 / GB; ++g) {
      asm volatile("" : "+v"(s[g]));
      if constexpr (Z) asm volatile("" : "+v"(z[g]));
    }
  }
  __device__ __forceinline__ float scale(int g) const {
    return (float)__builtin_bit_cast(typename Elem<E>::type, (uint16_t)s[g]);
  }
  // -(base + zero)
  __device__ __forceinline__ float offset(int g) const {
    return Z ? -code_base(E()) - (float)z[Z ? g : 0] : -code_base(E()) - 8.f;
  }
};

// n: the lane's column.  Groups past the last repeat it; x is 0 there.
template <typename E, int GB, bool Z>
__device__ __forceinline__ void load_scales(W4Scales<E, GB, Z>& f, const W4Args& a,
                                            const W4Source& src, uint32_t n, int step) {
#pragma unroll
  for (int g = 0; g < 4 / GB; ++g) {
    const int row = min(step * (4 / GB) + g, a.groups - 1) * a.N;
    f.s[g] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(src.s, n * 2, row * 2, 0);
    if constexpr (Z) f.z[g] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(src.z, n, row, 0);
  }
}

// A block of an expert product: blockIdx.y-th expert that has rows, those rows'
// places [first, first + rows), or rows = 0 past the last such expert.  Experts
// without rows get no blocks: a decode step leaves most of them empty.
struct W4Expert {
  int e, first, rows;
};

// From expert_offsets, by every wave on its own: lane l looks at expert l.
__device__ __forceinline__ W4Expert find_expert(const W4Args& a) {
  const int lane = threadIdx.x & 63;
  int first = 0, rows = 0;
  if (lane < a.n_local) {
    first = a.offsets[lane];
    rows = a.offsets[lane + 1] - first;
  }
  const uint64_t has = __ballot(rows > 0);
  const uint64_t mine = __ballot(rows > 0 && __popcll(has & ((1ull << lane) - 1)) == (int)blockIdx.y);
  if (!mine) return {0, 0, 0};
  const int e = __ffsll((unsigned long long)mine) - 1;
  return {e, __builtin_amdgcn_readlane(first, e), __builtin_amdgcn_readlane(rows, e)};
}

// From topk_ids, for at most one pair a thread: the stable counting sort that
// fm_moe_route does over its workgroups, of which each block needs one expert.
// The rows' pairs go to s_rows; the blocks of column tile 0 write sorted_pairs
// and expert_offsets.
__device__ __forceinline__ W4Expert route_here(const W4Args& a, int* s_rows, int* s_count,
                                               int* s_wave) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int mine = -1;
  if (t < a.n_pairs) {
    const int e = a.ids[t] - a.e0;
    if (e >= 0 && e < a.n_local) mine = e;
  }
  if (t < kW4MaxExperts) s_count[t] = 0;
  __syncthreads();
  if (mine >= 0) atomicAdd(&s_count[mine], 1);
  __syncthreads();
  const int rows_l = s_count[lane];
  const uint64_t has = __ballot(rows_l > 0);
  const uint64_t hit = __ballot(rows_l > 0 && __popcll(has & ((1ull << lane) - 1)) == (int)blockIdx.y);
  W4Expert x = {0, 0, 0};
  if (hit) {
    x.e = __ffsll((unsigned long long)hit) - 1;
    x.first = __builtin_amdgcn_readfirstlane(group_sum<64>(lane < x.e ? rows_l : 0));
    x.rows = __builtin_amdgcn_readlane(rows_l, x.e);
  }
  const bool in = hit && mine == x.e;
  const uint64_t match = __ballot(in);
  if (lane == 0) s_wave[wave] = __popcll(match);
  __syncthreads();
  if (in) {
    int rank = __popcll(match & ((1ull << lane) - 1));
    for (int w = 0; w < wave; ++w) rank += s_wave[w];
    s_rows[rank] = t;
    if (blockIdx.x == 0) a.pairs_out[x.first + rank] = t;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && t <= a.n_local) {
    int sum = 0;
    for (int e = 0; e < t; ++e) sum += s_count[e];
    a.offsets_out[t] = sum;
  }
  __syncthreads();
  return x;
}

template <W4Mode MODE>
__device__ __forceinline__ int64_t x_row(const W4Args& a, int64_t first, int64_t m) {
  return MODE == kGather ? a.pairs[first + m] / a.topk : first + m;
}

// Stores output (row m of the expert's, col) = v.
template <typename E, W4Mode MODE>
__device__ __forceinline__ void store_out(const W4Args& a, int64_t first, int64_t m, int col,
                                          float v) {
  typedef typename Elem<E>::type L;
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

// Few rows (chunks of 4 R): a block owns 16 columns and its 8 waves share K in
// contiguous parts.  x lies in LDS, so that the loads in flight are weights and
// scales alone (memory loads complete in order: an x load behind them would
// wait for them).  Logical row 4 r + i of a chunk is operand row 4 i + r, so that
// only accumulators r < R of a lane are in use; operand rows without a logical
// row repeat others, and what they give is not looked at.
constexpr int kFewAhead = 4;    // steps of 128 k in flight
constexpr int kTinyAhead = 6;

template <typename E, int GB, bool Z, int R, W4Mode MODE, bool ROUTE>
__global__ __launch_bounds__(kW4Threads) __attribute__((amdgpu_waves_per_eu(4))) void w4_few(
    const W4Args a) {
  typedef typename Elem<E>::type L;
  constexpr int ROWS = 4 * R, GP = 4 / GB, PF = kFewAhead;
  __shared__ float s_part[kW4Waves][R][64];
  __shared__ int s_rows[ROUTE ? kW4Threads : 1];   // the expert's pairs
  extern __shared__ char s_x[];                    // rows of stride bytes
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int i16 = lane & 15, q = lane >> 4;
  const int n0 = column_tile() * 16;
  const int n = min(n0 + i16, a.N - 1);
  int e = 0;
  int64_t first = 0, rows = a.M;
  if (MODE == kGather || MODE == kScatter) {
    W4Expert x;
    if constexpr (ROUTE) {
      __shared__ int s_count[kW4MaxExperts], s_wave[kW4Waves];
      x = route_here(a, s_rows, s_count, s_wave);
    } else {
      x = find_expert(a);
    }
    if (x.rows <= 0) return;
    e = x.e;
    first = x.first;
    rows = x.rows;
  }
  const int stride = a.blocks * 256 + 16;   // rows start 16 bytes apart in the banks
  const W4Source src = source_of<Z>(a, e, n0, 16);
  const uint32_t wo = (uint32_t)i16 * a.blocks * 64 + q * 16;   // columns past N read 0
  const int per = (a.blocks + kW4Waves - 1) / kW4Waves;
  const int s0 = min(a.blocks, wave * per), s1 = min(a.blocks, s0 + per);
  constexpr uint32_t one = ones2(E());
  const u32x4 ones = {one, one, one, one};

  for (int64_t m0 = MODE <= kDense32 ? (int64_t)blockIdx.z * ROWS : 0; m0 < rows;
       m0 += MODE <= kDense32 ? (int64_t)gridDim.z * ROWS : ROWS) {
    const int count = (int)min((int64_t)ROWS, rows - m0);
    u32x4 w[PF];
    W4Scales<E, GB, Z> sc[PF];
    // steps past the wave's last repeat it: no branch stands between the loads
    auto load = [&](u32x4& wr, W4Scales<E, GB, Z>& sr, int s) {
      s = min(s, s1 - 1);
      wr = load_codes(src, wo, s);
      load_scales<E, GB, Z>(sr, a, src, n, s);
    };
    if (s0 < s1) {
#pragma unroll
      for (int p = 0; p < PF; ++p) load(w[p], sc[p], s0 + p);
    }
    // x rows, zeros past K (the codes there may be anything)
    for (int m = 0; m < count; ++m) {
      const int64_t from = ROUTE ? s_rows[m0 + m] / a.topk : x_row<MODE>(a, first, m0 + m);
      const L* xr = static_cast<const L*>(a.x) + from * a.K;
      for (int k = t * 8; k < a.blocks * 128; k += kW4Threads * 8) {
        u32x4 v = {0, 0, 0, 0};
        if (k < a.K) v = *reinterpret_cast<const u32x4*>(xr + k);
        *reinterpret_cast<u32x4*>(s_x + m * stride + k * 2) = v;
      }
    }
    __syncthreads();
    int row = (i16 & 3) % R * 4 + (i16 >> 2);
    row = row < count ? row : 0;
    const char* xp = s_x + row * stride + q * 16;
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0.f;
    auto use = [&](u32x4& wr, W4Scales<E, GB, Z>& sr, int s) {
      loaded(wr);
      sr.loaded();
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        f32x4 tt = {0.f, 0.f, 0.f, 0.f}, xs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < GB; ++b) {
          const int j = g * GB + b;
          const u32x4 x = *reinterpret_cast<const u32x4*>(xp + s * 256 + j * 64);
          tt = mfma16(E(), x, codes8(E(), wr[j]), tt);
          xs = mfma16(E(), x, ones, xs);
        }
        const float scale = sr.scale(g), off = sr.offset(g);
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = fmaf(scale, fmaf(off, xs[r], tt[r]), acc[r]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    int s = s0;
    for (; s + PF <= s1; s += PF) {
#pragma unroll
      for (int p = 0; p < PF; ++p) {
        use(w[p], sc[p], s + p);
        __builtin_amdgcn_sched_barrier(0);   // a load kept behind the use needs no other registers
        load(w[p], sc[p], s + p + PF);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int p = 0; p < PF; ++p)
      if (s + p < s1) use(w[p], sc[p], s + p);
#pragma unroll
    for (int r = 0; r < R; ++r) s_part[wave][r][lane] = acc[r];
    __syncthreads();
    for (int o = t; o < R * 64; o += kW4Threads) {
      const int l = o & 63, m = (o >> 6) * 4 + (l >> 4), col = n0 + (l & 15);
      if (m < count && col < a.N) {
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < kW4Waves; ++u) v += s_part[u][o >> 6][l];
        store_out<E, MODE>(a, first, m0 + m, col, v);
      }
    }
    __syncthreads();
  }
}

constexpr uint32_t kNoX = 0xFE000000u;   // with any k * 2 added, past every x (below kNoX bytes)

// More rows: a wave keeps MT x NT tiles of 16 rows and 16 columns over its part of
// K, so that each x it reads (from L2) serves 16 NT columns.
template <typename E, int GB, bool Z, int MT, int NT, W4Mode MODE>
__global__ __launch_bounds__(kW4Threads) void w4_many(const W4Args a) {
  constexpr int ROWS = 16 * MT, GP = 4 / GB, PF = 2;
  __shared__ float s_part[kW4Waves][MT][4][64];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int i16 = lane & 15, q = lane >> 4;
  const int n0 = column_tile() * 16 * NT;
  int e = 0;
  int64_t first = 0, rows = a.M;
  if (MODE == kGather || MODE == kScatter) {
    const W4Expert x = find_expert(a);
    if (x.rows <= 0) return;
    e = x.e;
    first = x.first;
    rows = x.rows;
  }
  const W4Source src = source_of<Z>(a, e, n0, 16 * NT);
  uint32_t n[NT], wo[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    n[nt] = min(n0 + nt * 16 + i16, a.N - 1);
    wo[nt] = (uint32_t)(nt * 16 + i16) * a.blocks * 64 + q * 16;
  }
  const int per = (a.blocks + kW4Waves - 1) / kW4Waves;
  const int s0 = min(a.blocks, wave * per), s1 = min(a.blocks, s0 + per);
  constexpr uint32_t one = ones2(E());
  const u32x4 ones = {one, one, one, one};

  for (int64_t m0 = MODE <= kDense32 ? (int64_t)blockIdx.z * ROWS : 0; m0 < rows;
       m0 += MODE <= kDense32 ? (int64_t)gridDim.z * ROWS : ROWS) {
    // byte offsets from the chunk's first row, or from the first token: below 2^32
    const int64_t from = MODE == kGather ? 0 : first + m0;
    const __amdgpu_buffer_rsrc_t xr =
        resource(static_cast<const char*>(a.x) + from * a.K * 2,
                 (MODE == kGather ? a.M : min((int64_t)ROWS, rows - m0)) * a.K * 2);
    uint32_t xo[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)   // rows past the last repeat it
      xo[mt] = (uint32_t)(x_row<MODE>(a, first, min(m0 + mt * 16 + i16, rows - 1)) - from) * a.K * 2 +
               q * 16;
    u32x4 w[PF][NT], x[PF][MT][4];
    W4Scales<E, GB, Z> sc[PF][NT];
    auto load = [&](int p, int s) {
      s = min(s, s1 - 1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        w[p][nt] = load_codes(src, wo[nt], s);
        load_scales<E, GB, Z>(sc[p][nt], a, src, n[nt], s);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = s * 128 + j * 32;   // past K: an offset past the resource
          x[p][mt][j] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, k + q * 8 < a.K ? xo[mt] : kNoX, k * 2, 0));
        }
    };
    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto use = [&](int p) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        loaded(w[p][nt]);
        sc[p][nt].loaded();
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) loaded(x[p][mt][j]);
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        f32x4 xs[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          xs[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < GB; ++b) xs[mt] = mfma16(E(), x[p][mt][g * GB + b], ones, xs[mt]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          f32x4 tt[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) tt[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < GB; ++b) {
            const u32x4 c = codes8(E(), w[p][nt][g * GB + b]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) tt[mt] = mfma16(E(), x[p][mt][g * GB + b], c, tt[mt]);
          }
          const float scale = sc[p][nt].scale(g), off = sc[p][nt].offset(g);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[mt][nt][r] = fmaf(scale, fmaf(off, xs[mt][r], tt[mt][r]), acc[mt][nt][r]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    if (s0 < s1) {
#pragma unroll
      for (int p = 0; p < PF; ++p) load(p, s0 + p);
    }
    int s = s0;
    for (; s + PF <= s1; s += PF) {
#pragma unroll
      for (int p = 0; p < PF; ++p) {
        use(p);
        __builtin_amdgcn_sched_barrier(0);
        load(p, s + p + PF);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int p = 0; p < PF; ++p)
      if (s + p < s1) use(p);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) s_part[wave][mt][r][lane] = acc[mt][nt][r];
      __syncthreads();
      for (int o = t; o < MT * 256; o += kW4Threads) {
        const int l = o & 63, r = (o >> 6) & 3, mt = o >> 8;
        const int64_t m = m0 + mt * 16 + (l >> 4) * 4 + r;
        const int col = n0 + nt * 16 + (l & 15);
        if (m < rows && col < a.N) {
          float v = 0.f;
#pragma unroll
          for (int u = 0; u < kW4Waves; ++u) v += s_part[u][mt][r][l];
          store_out<E, MODE>(a, first, m, col, v);
        }
      }
      __syncthreads();
    }
  }
}

// The second layer of a single token's few pairs (at most kTinyPairs): a block
// owns 16 columns of out and walks every local pair, its waves sharing K, so that
// the weighted sum needs neither a second launch nor memory between.
constexpr int kTinyPairs = 8;

struct W4TinyArgs {
  W4Args w;             // pairs, offsets: sorted_pairs, expert_offsets; ids, e0, n_pairs
  const float* add;
  float* out;
  int T;
};

template <typename E, int GB, bool Z>
__global__ __launch_bounds__(kW4Threads) void w4_scatter_tiny(const W4TinyArgs args) {
  typedef typename Elem<E>::type L;
  constexpr int GP = 4 / GB, PF = kTinyAhead;
  const W4Args& a = args.w;
  __shared__ float s_part[kW4Waves][kTinyPairs][16];
  extern __shared__ char s_x[];   // one row of x a pair
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int i16 = lane & 15, q = lane >> 4;
  const int n0 = column_tile() * 16;
  const int n = min(n0 + i16, a.N - 1);
  const int stride = a.blocks * 256 + 16;
  // lane p: pair p's expert (-1: not here) and its row of x
  int ex = -1, row = -1, at_l = -1;
  const int places = a.offsets[a.n_local];
  if (lane < a.n_pairs) {
    ex = a.ids[lane] - a.e0;
    if (lane < places) at_l = a.pairs[lane];
  }
  for (int p = 0; p < a.n_pairs; ++p) {
    const int at = __builtin_amdgcn_readlane(at_l, p);   // place p holds pair `at`
    if (lane == at) row = p;
  }
  if (ex < 0 || ex >= a.n_local || row < 0) ex = -1;
  const uint64_t has = __ballot(ex >= 0);
  const int units = __popcll(has);
  // the u-th local pair's lane
  auto pair_of = [&](int u) {
    uint64_t m = has;
    for (int i = 0; i < u; ++i) m &= m - 1;
    return __ffsll((unsigned long long)m) - 1;
  };
  const int per = (a.blocks + kW4Waves - 1) / kW4Waves;
  const int s0 = min(a.blocks, wave * per), s1 = min(a.blocks, s0 + per);
  const int steps = s1 - s0, total = steps * units;
  u32x4 w[PF];
  W4Scales<E, GB, Z> sc[PF];
  int lu = 0, li = 0, lp = units ? pair_of(0) : 0;   // next to load: unit, step, pair
  W4Source src = source_of<Z>(a, units ? __builtin_amdgcn_readlane(ex, lp) : 0, n0, 16);
  const uint32_t wo = (uint32_t)i16 * a.blocks * 64 + q * 16;
  auto load = [&](u32x4& wr, W4Scales<E, GB, Z>& sr) {
    wr = load_codes(src, wo, s0 + li);
    load_scales<E, GB, Z>(sr, a, src, n, s0 + li);
    if (++li == steps && lu + 1 < units) {   // past the last step: that one again
      li = 0;
      lp = pair_of(++lu);
      src = source_of<Z>(a, __builtin_amdgcn_readlane(ex, lp), n0, 16);
    }
    li = min(li, steps - 1);
  };
  if (total > 0) {
#pragma unroll
    for (int p = 0; p < PF; ++p) load(w[p], sc[p]);
  }
  for (int u = 0; u < units; ++u) {
    const int64_t from = __builtin_amdgcn_readlane(row, pair_of(u));
    const L* xr = static_cast<const L*>(a.x) + from * a.K;
    for (int k = t * 8; k < a.blocks * 128; k += kW4Threads * 8) {
      u32x4 v = {0, 0, 0, 0};
      if (k < a.K) v = *reinterpret_cast<const u32x4*>(xr + k);
      *reinterpret_cast<u32x4*>(s_x + u * stride + k * 2) = v;
    }
  }
  __syncthreads();
  constexpr uint32_t one = ones2(E());
  const u32x4 ones = {one, one, one, one};
  float acc = 0.f;
  int cu = 0, ci = 0;   // next to use
  auto use = [&](u32x4& wr, W4Scales<E, GB, Z>& sr) {
    loaded(wr);
    sr.loaded();
    const char* xp = s_x + cu * stride + q * 16 + (s0 + ci) * 256;   // every operand row the same
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      f32x4 tt = {0.f, 0.f, 0.f, 0.f}, xs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < GB; ++b) {
        const int j = g * GB + b;
        const u32x4 x = *reinterpret_cast<const u32x4*>(xp + j * 64);
        tt = mfma16(E(), x, codes8(E(), wr[j]), tt);
        xs = mfma16(E(), x, ones, xs);
      }
      acc = fmaf(sr.scale(g), fmaf(sr.offset(g), xs[0], tt[0]), acc);
    }
    if (++ci == steps) {
      if (lane < 16) s_part[wave][cu][lane] = acc;
      acc = 0.f;
      ci = 0;
      ++cu;
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  int i = 0;
  for (; i + PF <= total; i += PF) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      use(w[p], sc[p]);
      load(w[p], sc[p]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int p = 0; p < PF; ++p)
    if (i + p < total) use(w[p], sc[p]);
  if (steps <= 0 && lane < 16)
    for (int u = 0; u < units; ++u) s_part[wave][u][lane] = 0.f;
  __syncthreads();
  const int col = n0 + (t & 15);
  if (t < args.T * 16 && col < a.N) {
    const int token = t >> 4;
    float v = args.add ? args.add[(int64_t)token * a.N + col] : 0.f;
    for (int k = 0; k < a.topk; ++k) {
      const int p = token * a.topk + k;
      if (!(has >> p & 1)) continue;
      const int u = __popcll(has & ((1ull << p) - 1));
      float y = 0.f;
      for (int x = 0; x < kW4Waves; ++x) y += s_part[x][u][t & 15];
      v += y * a.weights[p];
    }
    args.out[(int64_t)token * a.N + col] = v;
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

constexpr int64_t kFewLds = 128 << 10;   // most LDS that x may take

template <typename E, int GB, bool Z, W4Mode MODE>
void launch_rows(const W4Args& a, int64_t most, dim3 grid, hipStream_t stream) {
  const int64_t stride = (int64_t)a.blocks * 256 + 16;
#define FM_FEW(R, ROUTE)                                                                     \
  do {                                                                                       \
    if (MODE <= kDense32) grid.z = (unsigned)std::min<int64_t>(cdiv(a.M, 4 * R), 65535);     \
    const int64_t rows = std::min<int64_t>(most, 4 * R);                                     \
    hipLaunchKernelGGL((w4_few<E, GB, Z, R, MODE, ROUTE>), grid, dim3(kW4Threads),           \
                       rows* stride, stream, a);                                             \
  } while (0)
#define FM_MANY(MT, NT)                                                                      \
  do {                                                                                       \
    if (MODE <= kDense32) grid.z = (unsigned)std::min<int64_t>(cdiv(a.M, 16 * MT), 65535);   \
    grid.x = (unsigned)cdiv(a.N, 16 * NT);                                                   \
    hipLaunchKernelGGL((w4_many<E, GB, Z, MT, NT, MODE>), grid, dim3(kW4Threads), 0, stream, a); \
  } while (0)
  if constexpr (MODE == kGather) {
    if (a.n_pairs > 0) {
      if (most <= 4) FM_FEW(1, true);
      else FM_FEW(2, true);
      return;
    }
  }
  if (most <= 4 && std::min<int64_t>(most, 4) * stride <= kFewLds) FM_FEW(1, false);
  else if (most <= 8 && 8 * stride <= kFewLds) FM_FEW(2, false);
  else if (most <= 16) FM_MANY(1, 2);
  else if (most <= 32) FM_MANY(2, 2);
  else FM_MANY(3, 2);
#undef FM_FEW
#undef FM_MANY
}

#define FM_W4_ZERO(CALL, E, GB)     \
  do {                              \
    if (zeros) CALL(E, GB, true);   \
    else CALL(E, GB, false);        \
  } while (0)
#define FM_W4_GROUP(CALL, E)                      \
  do {                                            \
    if (group == 32) FM_W4_ZERO(CALL, E, 1);      \
    else if (group == 64) FM_W4_ZERO(CALL, E, 2); \
    else FM_W4_ZERO(CALL, E, 4);                  \
  } while (0)

// most: the rows (of an expert) that a chunk is chosen for.
template <W4Mode MODE>
void launch_w4(fm_dtype_t dt, int group, const W4Args& a, int64_t most, int64_t experts,
               hipStream_t stream) {
  const dim3 grid((unsigned)cdiv(a.N, 16), (unsigned)experts, 1);
  const uint8_t* zeros = a.zeros;
#define FM_W4_CALL(E, GB, Z) launch_rows<E, GB, Z, MODE>(a, most, grid, stream)
  if (dt == FM_F16) FM_W4_GROUP(FM_W4_CALL, F16);
  else FM_W4_GROUP(FM_W4_CALL, BF16);
#undef FM_W4_CALL
}

void launch_tiny(fm_dtype_t dt, int group, const W4TinyArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)cdiv(a.w.N, 16));
  const uint8_t* zeros = a.w.zeros;
  const size_t lds = (size_t)a.w.n_pairs * ((size_t)a.w.blocks * 256 + 16);
#define FM_W4_CALL(E, GB, Z) \
  hipLaunchKernelGGL((w4_scatter_tiny<E, GB, Z>), grid, dim3(kW4Threads), lds, stream, a)
  if (dt == FM_F16) FM_W4_GROUP(FM_W4_CALL, F16);
  else FM_W4_GROUP(FM_W4_CALL, BF16);
#undef FM_W4_CALL
}
#undef FM_W4_GROUP
#undef FM_W4_ZERO

// Rows that an expert product is chosen for: no expert can have more than the
// pairs, and few have more than twice the mean.
int64_t expert_rows(int64_t pairs, int n_local) {
  return std::min(pairs, cdiv(2 * pairs, n_local));
}

int64_t row_bytes(int64_t K) { return cdiv(K, 128) * 64; }

fm_status_t check_w4(fm_dtype_t dt, int64_t N, int64_t K, int group, const void* x,
                     const void* packed, const void* scales, bool work) {
  if (dt != FM_F16 && dt != FM_BF16) return FM_ERR_UNSUPPORTED;
  if (N < 0 || K < 0 || N % 8 || K % 8) return FM_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return FM_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(packed) || !aligned16(scales)) return FM_ERR_INVALID_ARG;
  if (work && K > 0 && (!x || !packed || !scales)) return FM_ERR_INVALID_ARG;
  if (N >= (1ll << 22) || K >= (1ll << 22) || cdiv(K, group) * N >= (1ll << 30))
    return FM_ERR_UNSUPPORTED;   // 32-bit offsets into one matrix's scales
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
  if (T > 0 && T * hidden * 2 >= kNoX) return FM_ERR_UNSUPPORTED;   // 32-bit row offsets
  // A decode step's pairs are sorted by the product's own blocks (one launch); more
  // pairs, or rows too long for LDS, by the route's.
  const int64_t pairs = T * topk;
  const bool here = T > 0 && ffn > 0 && topk > 0 && T <= kW4Threads && pairs <= kW4Threads &&
                    n_local >= 1 && n_local <= kW4MaxExperts && pairs / n_local <= kFewRows &&
                    8 * (cdiv(hidden, 128) * 256 + 16) <= kFewLds;
  if (here) {
    st = check_route(T, topk, n_local, topk_ids, sorted_pairs, expert_offsets, ws, ws_bytes);
  } else {
    st = fm_moe_route(T, topk, expert_begin, n_local, topk_ids, sorted_pairs, expert_offsets, ws,
                      ws_bytes, stream);
  }
  if (st != FM_OK || T == 0 || ffn == 0) return st;
  W4Args a = {};
  a.x = X;
  a.packed = static_cast<const uint8_t*>(packed);
  a.scales = scales;
  a.zeros = zeros;
  a.out = H;
  a.pairs = sorted_pairs;
  a.offsets = expert_offsets;
  a.M = T;
  a.N = (int)ffn;
  a.K = (int)hidden;
  a.blocks = (int)cdiv(hidden, 128);
  a.groups = (int)cdiv(hidden, group);
  a.topk = topk;
  a.act = act;
  a.n_local = n_local;
  if (here) {
    a.ids = topk_ids;
    a.pairs_out = sorted_pairs;
    a.offsets_out = expert_offsets;
    a.n_pairs = (int)pairs;
    a.e0 = expert_begin;
  }
  launch_w4<kGather>(dt, group, a, here ? pairs : expert_rows(pairs, n_local),
                     std::min<int64_t>(n_local, pairs), stream);
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
  a.n_local = n_local;
  const int64_t pairs = T * topk;
  if (pairs <= kTinyPairs && pairs * (a.blocks * 256 + 16) <= kFewLds) {
    a.ids = topk_ids;
    a.e0 = expert_begin;
    a.n_pairs = (int)pairs;
    const W4TinyArgs tiny = {a, add, out, (int)T};
    launch_tiny(dt, group, tiny, stream);
    return launch_status();
  }
  launch_w4<kScatter>(dt, group, a, expert_rows(pairs, n_local),
                      std::min<int64_t>(n_local, pairs), stream);
  const int n4 = (int)(hidden / 4);
  hipLaunchKernelGGL(w4_join, dim3((unsigned)std::min<int64_t>(cdiv(T * n4, 256), 65536)), dim3(256),
                     0, stream, T, n4, (int)topk, (int)expert_begin, (int)n_local, topk_ids,
                     static_cast<const f32x4*>(ws), reinterpret_cast<const f32x4*>(add),
                     reinterpret_cast<f32x4*>(out));
  return launch_status();
}
