// fm_w4.hip -- products with 4-bit weights and group scales for few rows: the
// dense shard, and the two matrices of each local expert of a MoE layer.
//
// With few rows the weights are all there is to read, so the kernels are built to
// stream them in whole cache lines, two steps of 128 k ahead.  Three shapes:
//   w4_one    one row (few_rows): 4x4x4 products whose diagonal is what is wanted
//   few_rows  one row so, or up to 4 (experts) with 16x16x32 products: x in LDS, the
//             waves share the tiles of a block and K
//   many_rows 16, 32 or 48 rows at a time: 16x16x32 products, K over the waves
// A code c enters the matrix core exactly, without a conversion, as the 16-bit
// number 16 + c, whose bit pattern is the code shifted to the top of a constant's
// mantissa.  With t = sum x (16 + c) and S = sum x over one group of K (a matrix
// product with ones),
//   sum x (c - zero) scale = scale * (t - (16 + zero) * S),
// so that scale and zero cost two fused multiply-adds a group and output.  16 is the
// smallest base whose sums have one exponent: what t loses to rounding grows with it
// (fp16 has bits for a base of 64 at one shift less in eight codes; with x of one
// sign that lost two more bits of the result).
//
// Measured (kernel alone, three matrices in turn, which the Infinity Cache holds where
// one is below 80 MB; the bytes of codes, scales and zeros over that time): 1 x 6144 x
// 12288 fp16 9.5 to 10 us (4 TB/s; a call with the weights from HBM 13.4), 61 tokens
// over 8 of 64 experts of 4096 x 2816 14.1 us (3.0 TB/s), over all 64 80 to 83 us (4.0
// TB/s): waves wait for memory half of their time or more.  45 x 12288 x 6144 bf16 25
// to 26 us (1.9 TB/s): 256 blocks, whose LDS leaves room for one a compute unit, with
// two waves a SIMD that issue vector instructions in 48% of the cycles (group 32: eight
// fused multiply-adds a product), use LDS in 38% and the matrix core in 16%.
#include <algorithm>

#include "fm_act.hpp"
#include "fm_w4_index.hpp"
#include "fm_wave.hpp"

namespace fm {
namespace {

constexpr int kW4Waves = 8;          // few rows
constexpr int kW4Threads = 64 * kW4Waves;
constexpr int kManyWaves = 8;            // more rows
constexpr int kManyThreads = 64 * kManyWaves;
constexpr int kW4MaxExperts = 64;
// Rows of an expert up to which they all lie in LDS (61 and 240 tokens over 64
// experts, 4096 x 2816: 4 rows 79 and 115 us, 8 rows 82 and 127).
constexpr int kFewRows = 4;
// Mean rows of an expert up to which w4_mixed runs, with the route in its own blocks
// for the first layer (8 experts, 4096 x 2816: 61 tokens 22.6 us, as two launches of
// route and w4_many 31.5).  The mean is the host's bound, tokens x topk over the local
// experts: on one rank of eight it is eight times too high, and 68 tokens on 8 of 64
// experts already take the other form (32 us, 61 tokens 16).
constexpr int64_t kMixedRows = 16;

__device__ __forceinline__ f32x4 mfma16(F16, u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(BF16, u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// 16 independent 4x4x4 products: lanes 4 b + i hold row i of A and column i of B of
// product b (four k each), and get column i of D, its rows in the four registers.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ f32x4 mfma4(F16, u32x2 a, u32x2 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, a),
                                            __builtin_bit_cast(f16x4, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma4(BF16, u32x2 a, u32x2 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, a),
                                                __builtin_bit_cast(s16x4, b), c, 0, 0, 0);
}

// Constants that stay in registers: as literals they would keep (x & mask) | base
// from being one instruction (v_and_or_b32 takes no literal).
template <typename E>
struct W4Consts {
  uint32_t mask, base;
  u32x4 ones;
  __device__ __forceinline__ W4Consts() {
    constexpr bool half = E::id == FM_F16;
    mask = half ? 0x03C003C0u : 0x00780078u;
    base = half ? 0x4C004C00u : 0x41804180u;   // 16; the mask is where 1 + 2 + 4 + 8 lie
    const uint32_t one = half ? 0x3C003C00u : 0x3F803F80u;
    ones = u32x4{one, one, one, one};
    asm volatile("" : "+s"(mask));
    asm volatile("" : "+v"(base));
    asm volatile("" : "+v"(ones));
  }
};

// Eight codes of a word as 16 + code, pair i holding nibbles i and i + 4.
__device__ __forceinline__ u32x4 codes8(const W4Consts<BF16>& k, uint32_t w) {
  return {((w << 3) & k.mask) | k.base, ((w >> 1) & k.mask) | k.base,
          ((w >> 5) & k.mask) | k.base, ((w >> 9) & k.mask) | k.base};
}
__device__ __forceinline__ u32x4 codes8(const W4Consts<F16>& k, uint32_t w) {
  return {((w << 6) & k.mask) | k.base, ((w << 2) & k.mask) | k.base,
          ((w >> 2) & k.mask) | k.base, ((w >> 6) & k.mask) | k.base};
}
constexpr float kCodeBase = 16.f;

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
  int some;      // 1, or 0 with K = 0: then every resource is empty and offset 0
  int topk, act;
  int n_local;
  int tiles;     // column tiles of a block (few rows)
  // a route inside the product: at most kW4Threads pairs
  const int32_t* ids;
  int32_t *pairs_out, *offsets_out;
  int n_pairs, e0;
};

// The column tile of a block: each XCD (blocks go to them in turn) takes
// neighbouring tiles, whose scales share cache lines.
__device__ __forceinline__ int column_tile() {
  const int b = blockIdx.x, n = gridDim.x, x = b & 7;
  return x * (n >> 3) + min(x, n & 7) + (b >> 3);
}

// An offset past every x (those have fewer bytes), also with any row's and step's
// added to it.
constexpr uint32_t kNoX = 0xFE000000u;

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

__device__ __forceinline__ u32x4 load_codes(const W4Source& src, uint32_t lane_offset, int offset) {
  return __builtin_bit_cast(u32x4,
                            __builtin_amdgcn_raw_buffer_load_b128(src.w, lane_offset, offset, 0));
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
  // -(16 + zero)
  __device__ __forceinline__ float offset(int g) const {
    return Z ? -kCodeBase - (float)z[Z ? g : 0] : -kCodeBase - 8.f;
  }
};

// i16: the lane's column in the tile.  Groups past the last read another (x is 0
// there), and columns past N what follows, or 0.
template <typename E, int GB, bool Z>
__device__ __forceinline__ void load_scales(W4Scales<E, GB, Z>& f, const W4Source& src,
                                            uint32_t i16, int s, int s_group, int s_last) {
#pragma unroll
  for (int g = 0; g < 4 / GB; ++g) {
    const int at = min(s + g * s_group, s_last);
    f.s[g] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(src.s, i16 * 2, at, 0);
    if constexpr (Z) f.z[g] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(src.z, i16, at >> 1, 0);
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

// What a block works on: the columns from n0 of one matrix, and the rows that it
// multiplies, which s_rows lists where the block routed them itself.
struct W4Work {
  int n0, e;
  int64_t first, rows;
  const int* s_rows;
};

template <W4Mode MODE, bool ROUTE>
__device__ __forceinline__ int64_t x_row(const W4Args& a, const W4Work& b, int64_t m) {
  if (MODE != kGather) return b.first + m;
  return (ROUTE ? b.s_rows[m] : a.pairs[b.first + m]) / a.topk;
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

// x in LDS: rows of 16-bit values, 16 bytes apart in the banks, behind them fp32
// sums of x, and places of each lane for what it has not to keep.  For one row the
// sums are those of octets (8 values), ordered [step of 128 k][q][j] so that a
// lane's four lie together; for several rows those of 32 values, in order.
struct W4Stage {
  char* base;
  int stride, sums, sum_stride, dump;   // bytes: of a row, start, of a row, start
};

__host__ __device__ inline int64_t stage_bytes(int blocks, int64_t rows) {
  return rows * (blocks * 320 + 16) + 64 * 20;
}

__device__ __forceinline__ W4Stage stage_at(char* base, int blocks, int rows) {
  return {base, blocks * 256 + 16, rows * (blocks * 256 + 16), blocks * 64,
          rows * (blocks * 320 + 16)};
}

// Octet `at` (bytes / 16 of the row) of row m, if `keep`.  No branch: the compiler
// would move the load of v into it, behind loads that are to be waited for later.
template <typename E, bool ONE>
__device__ __forceinline__ void stage_octet(const W4Stage& st, int m, uint32_t octet,
                                            const u32x4& v, bool keep) {
  typedef typename Raw4<E>::type L4;
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t to = keep ? m * st.stride + octet * 16 : st.dump + lane * 16;
  const uint32_t in_row = ONE ? (octet >> 4) * 64 + (octet & 3) * 16 + (octet >> 2 & 3) * 4
                              : (octet >> 2) * 4;
  const uint32_t sum_to = keep && (ONE || (octet & 3) == 0) ? st.sums + m * st.sum_stride + in_row
                                                            : st.dump + 64 * 16 + lane * 4;
  *reinterpret_cast<u32x4*>(st.base + to) = v;
  const f32x4 lo = widen<E>(__builtin_bit_cast(L4, u32x2{v[0], v[1]}));
  const f32x4 hi = widen<E>(__builtin_bit_cast(L4, u32x2{v[2], v[3]}));
  const f32x4 s = lo + hi;
  float sum = (s[0] + s[1]) + (s[2] + s[3]);
  if (!ONE) sum = group_sum<4>(sum);
  *reinterpret_cast<float*>(st.base + sum_to) = sum;
}

// A tile's weights are loaded with lane 4 c + q on the 16 bytes of column c that
// hold the octets 8 q + 32 j: four neighbours share a 64-byte line.  (In the order
// of a 16x16x32 instruction's operand, l = 16 q + c, a load touched 64 lines, and the
// cache's one lookup a clock was what bounded the kernel.)

// One row, one step of 128 k: in a 4x4x4 instruction the four lanes of a column are
// the columns of one product; its A rows are x at the four lanes' own k, so that the
// diagonal, row q of lane q's column, is the lane's part, whatever the others are.
template <typename E, int GB, bool Z>
__device__ __forceinline__ float one_row_step(const W4Consts<E>& k, u32x4& w,
                                              W4Scales<E, GB, Z>& sc, const W4Stage& st,
                                              int step) {
  const int q = threadIdx.x & 3;
  loaded(w);
  sc.loaded();
  const char* x = st.base + step * 256 + q * 16;
  const f32x4 xs = *reinterpret_cast<const f32x4*>(st.base + st.sums + step * 64 + q * 16);
  float acc = 0.f;
#pragma unroll
  for (int g = 0; g < 4 / GB; ++g) {
    f32x4 t = {0.f, 0.f, 0.f, 0.f};
    float sum = xs[g * GB];
#pragma unroll
    for (int b = 1; b < GB; ++b) sum += xs[g * GB + b];
#pragma unroll
    for (int b = 0; b < GB; ++b) {
      const int j = g * GB + b;
      const u32x4 c = codes8(k, w[j]);
      const u32x4 xv = *reinterpret_cast<const u32x4*>(x + j * 64);
      t = mfma4(E(), u32x2{xv[0], xv[1]}, u32x2{c[0], c[1]}, t);
      t = mfma4(E(), u32x2{xv[2], xv[3]}, u32x2{c[2], c[3]}, t);
    }
    const float mine = q & 2 ? (q & 1 ? t[3] : t[2]) : (q & 1 ? t[1] : t[0]);
    acc = fmaf(sc.scale(g), fmaf(sc.offset(g), sum, mine), acc);
  }
  __builtin_amdgcn_sched_barrier(0);
  return acc;
}

// From the order of the load into the operand's, through 1 KiB of LDS of the wave's
// own.  Slot 4 c + (q + c / 4) % 4 keeps both sides free of bank conflicts.
__device__ __forceinline__ u32x4 to_operand(const u32x4& w, char* own) {
  const int l = threadIdx.x & 63, c = l >> 2, q = l & 3, n = l & 15, k = l >> 4;
  *reinterpret_cast<u32x4*>(own + (4 * c + ((q + (c >> 2)) & 3)) * 16) = w;
  wave_lds_sync();
  const u32x4 v = *reinterpret_cast<const u32x4*>(own + (4 * n + ((k + (n >> 2)) & 3)) * 16);
  wave_lds_sync();
  return v;
}

// Up to four rows, one step: logical row i is operand row 4 i, so that only
// accumulator 0 of a lane, row lane / 16, is in use; the other operand rows repeat
// these, and what they give is not looked at.
template <typename E, int GB, bool Z>
__device__ __forceinline__ float four_row_step(const W4Consts<E>& k, u32x4& w,
                                               W4Scales<E, GB, Z>& sc, const W4Stage& st, int step,
                                               int x_row, int sum_row, char* own) {
  loaded(w);
  const u32x4 v = to_operand(w, own);
  sc.loaded();
  const char* x = st.base + x_row * st.stride + step * 256 + (threadIdx.x >> 4 & 3) * 16;
  const f32x4 xs =
      *reinterpret_cast<const f32x4*>(st.base + st.sums + sum_row * st.sum_stride + step * 16);
  float acc = 0.f;
#pragma unroll
  for (int g = 0; g < 4 / GB; ++g) {
    f32x4 t = {0.f, 0.f, 0.f, 0.f};
    float sum = xs[g * GB];
#pragma unroll
    for (int b = 1; b < GB; ++b) sum += xs[g * GB + b];
#pragma unroll
    for (int b = 0; b < GB; ++b) {
      const int j = g * GB + b;
      t = mfma16(E(), *reinterpret_cast<const u32x4*>(x + j * 64), codes8(k, v[j]), t);
    }
    acc = fmaf(sc.scale(g), fmaf(sc.offset(g), sum, t[0]), acc);
  }
  __builtin_amdgcn_sched_barrier(0);
  return acc;
}

// A block owns a.tiles tiles of 16 columns (1, 2, 4 or 8); its 8 waves share the
// tiles, and K in contiguous parts where they outnumber them (with all 8 waves on
// one tile after another, 61 tokens over 64 experts of 4096 x 2816 took 87 us for 80).  x lies in LDS, so that the loads in flight are
// weights and scales alone (memory loads complete in order: an x load behind them
// would wait for them).
constexpr int kAhead = 2;   // steps of 128 k in flight; 3 and 4 measured no better, 6 worse

// LDS: x, then the waves' own memory and their sums.
__host__ __device__ constexpr int few_own(int R) { return R > 1 ? kW4Waves * 1024 : 0; }
__host__ __device__ inline int64_t few_lds(int blocks, int R) {
  return stage_bytes(blocks, R) + few_own(R) + kW4Waves * R * 64;
}

template <typename E, int GB, bool Z, int R, W4Mode MODE, bool ROUTE>
__device__ __forceinline__ void few_rows(const W4Args& a, const W4Work& b, char* lds) {
  constexpr int PF = kAhead, XB = 3, GP = 4 / GB;
  const W4Stage st = stage_at(lds, a.blocks, R);
  char* s_own = lds + stage_bytes(a.blocks, R);
  float* s_part = reinterpret_cast<float*>(s_own + few_own(R));   // [waves][R * 16]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = threadIdx.x >> 2 & 15, q = threadIdx.x & 3;
  const int sc16 = R > 1 ? threadIdx.x & 15 : c16;   // the column whose sums the lane takes
  const int n0 = b.n0, e = b.e;
  const int64_t first = b.first, rows = b.rows;
  const W4Source src = source_of<Z>(a, e, n0, 16 * a.tiles);
  const uint32_t wo = (uint32_t)c16 * a.blocks * 64 + q * 16;   // columns past N read 0
  // Tiles and the parts of K are powers of two.
  const int shift = 3 - __builtin_ctz(a.tiles), parts = 1 << shift;
  const int tile = wave >> shift;
  const bool busy = n0 + tile * 16 < a.N;
  const int per = (a.blocks + parts - 1) >> shift;
  const int s0 = busy ? min(a.blocks, (wave & parts - 1) * per) : 0;
  const int steps = busy ? min(a.blocks, s0 + per) - s0 : 0;
  const W4Consts<E> consts;

  for (int64_t m0 = 0; m0 < rows; m0 += R) {
    const int count = (int)min((int64_t)R, rows - m0);
    // x rows into LDS in pieces of 16 bytes a lane, zeros past K (the codes there
    // may be anything).  The first pieces are asked for ahead of the weights.
    const int64_t from = MODE == kGather ? 0 : first + m0;
    const __amdgpu_buffer_rsrc_t xr =
        resource(static_cast<const char*>(a.x) + from * a.K * 2,
                 (MODE == kGather ? a.M : (int64_t)count) * a.K * 2);
    const uint32_t lane_x = threadIdx.x * 16;
    struct Piece {
      int m, c;   // row, and 16 * kW4Threads-byte part of it
    };
    auto next = [&](Piece& p) {
      const bool wrap = (p.c + 1) * (kW4Threads * 16) >= a.blocks * 256;
      p.c = wrap ? 0 : p.c + 1;
      p.m += wrap ? 1 : 0;
    };
    auto fetch = [&](const Piece& p) {
      int row = min(p.m, count - 1);   // rows past the last repeat it
      if (MODE == kGather)
        row = __builtin_amdgcn_readfirstlane((int)x_row<MODE, ROUTE>(a, b, m0 + row));
      const bool in = lane_x + p.c * (kW4Threads * 16) < (uint32_t)a.K * 2;
      return __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                     xr, in ? lane_x : kNoX,
                     (uint32_t)row * a.K * 2 + p.c * (kW4Threads * 16), 0));
    };
    auto place = [&](const Piece& p, const u32x4& v) {
      const uint32_t at = lane_x + p.c * (kW4Threads * 16);
      stage_octet<E, R == 1>(st, p.m, at >> 4, v, p.m < count && at < (uint32_t)a.blocks * 256);
    };
    u32x4 xv[XB];
    Piece ask = {0, 0}, put = {0, 0};
#pragma unroll
    for (int i = 0; i < XB; ++i) {
      xv[i] = fetch(ask);
      next(ask);
    }

    u32x4 w[PF];
    W4Scales<E, GB, Z> sc[PF];
    // Where the wave's next step lies in the resources (bytes, scalar); past the last
    // step, that one again.
    const int n_tile = tile_column(n0, tile * 16, a.N), at0 = n_tile - n0;
    const int w_last = (at0 * a.blocks + max(s0 + steps - 1, 0)) * 64;
    const int s_last = scale_offset(a.groups, a.groups, n_tile, a.N, a.some);
    const int s_step = a.N * (2 * GP);
    int lw = min((at0 * a.blocks + s0) * 64, w_last);
    int ls = scale_offset(s0 * GP, a.groups, n_tile, a.N, a.some);
    auto load = [&](u32x4& wr, W4Scales<E, GB, Z>& sr) {
      wr = load_codes(src, wo, lw);
      load_scales<E, GB, Z>(sr, src, sc16, ls, a.N * 2, s_last);
      lw = min(lw + 64, w_last);
      ls = min(ls + s_step, s_last);
    };
    // Every load up to here is issued by all waves on one path, needed or not (none
    // leaves its resource): behind a branch the compiler would wait for them early.
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      load(w[p], sc[p]);
      __builtin_amdgcn_sched_barrier(0);   // in the loop's order, which the waits count by
    }
#pragma unroll
    for (int i = 0; i < XB; ++i) {
      place(put, xv[i]);
      next(put);
    }
    for (; put.m < count; next(put)) place(put, fetch(put));
    __syncthreads();
    static_assert(R == 1 || R == 4, "one row, or four");
    float acc = 0.f;
    int step = s0;
    const int i4 = threadIdx.x >> 2 & 3, k4 = threadIdx.x >> 4 & 3;
    const int x_row = i4 < count ? i4 : 0, sum_row = k4 < count ? k4 : 0;
    auto use = [&](u32x4& wr, W4Scales<E, GB, Z>& sr) {
      if constexpr (R == 1)
        acc += one_row_step<E, GB, Z>(consts, wr, sr, st, step);
      else
        acc += four_row_step<E, GB, Z>(consts, wr, sr, st, step, x_row, sum_row,
                                       s_own + wave * 1024);
      ++step;
      __builtin_amdgcn_sched_barrier(0);   // a load kept behind the use needs no other registers
    };
    // No copy of the body for the last steps: the first pass over the code waits for
    // its instructions too.
#pragma clang loop unroll(disable)
    for (int i = 0; i < steps; i += PF) {
#pragma unroll
      for (int p = 0; p < PF; ++p) {
        if (i + p < steps) use(w[p], sc[p]);
        load(w[p], sc[p]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (R == 1) acc = group_sum<4>(acc);
    if (R > 1 || q == 0) s_part[wave * R * 16 + (R > 1 ? threadIdx.x & 63 : c16)] = acc;
    __syncthreads();
    for (int o = threadIdx.x; o < a.tiles * R * 16; o += kW4Threads) {
      const int t = o / (R * 16), m = (o >> 4) % R, col = n0 + t * 16 + (o & 15);
      if (m < count && col < a.N) {
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < kW4Waves; ++u) {
          const float p = s_part[((t << shift) + u & kW4Waves - 1) * R * 16 + o % (R * 16)];
          v += u < parts ? p : 0.f;
        }
        store_out<E, MODE>(a, first, m0 + m, col, v);
      }
    }
    __syncthreads();
  }
}

// More rows: a wave keeps MT x NT tiles of 16 rows and 16 columns over its part of
// K, so that each x it reads serves 16 NT columns.  Both operands are loaded in whole
// lines and take the operands' order through LDS of the wave's own; the next step's
// loads are in flight meanwhile.
constexpr int kManyRow = 256 + 16;   // bytes of a row of x in LDS: 16 apart in the banks

constexpr int many_lds(int MT, int NT) {
  return kManyWaves * (MT * 16 * kManyRow + NT * 1024);
}

template <typename E, int GB, bool Z, int MT, int NT, W4Mode MODE, bool ROUTE>
__device__ __forceinline__ void many_rows(const W4Args& a, const W4Work& b, char* s_dyn) {
  constexpr int ROWS = 16 * MT, GP = 4 / GB, XL = MT * 4;   // loads of 4 rows
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, q = lane >> 4;
  const int n0 = b.n0, e = b.e;
  const int64_t first = b.first, rows = b.rows;
  char* own_x = s_dyn + wave * (MT * 16 * kManyRow + NT * 1024);
  char* own_w = own_x + MT * 16 * kManyRow;
  const W4Source src = source_of<Z>(a, e, n0, 16 * NT);
  uint32_t wo[NT];   // columns past N read 0
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    wo[nt] = (uint32_t)(nt * 16 + (lane >> 2)) * a.blocks * 64 + (lane & 3) * 16;
  const int per = (a.blocks + kManyWaves - 1) / kManyWaves;
  const int s0 = min(a.blocks, wave * per), s1 = min(a.blocks, s0 + per);
  const W4Consts<E> consts;

  for (int64_t m0 = MODE <= kDense32 ? (int64_t)blockIdx.z * ROWS : 0; m0 < rows;
       m0 += MODE <= kDense32 ? (int64_t)gridDim.z * ROWS : ROWS) {
    // byte offsets from the chunk's first row, or from the first token: below 2^32
    const int64_t from = MODE == kGather ? 0 : first + m0;
    const __amdgpu_buffer_rsrc_t xr =
        resource(static_cast<const char*>(a.x) + from * a.K * 2,
                 (MODE == kGather ? a.M : min((int64_t)ROWS, rows - m0)) * a.K * 2);
    uint32_t xo[XL];   // lane: row lane / 16 of four, 16 bytes lane % 16 of a step's 256
#pragma unroll
    for (int i = 0; i < XL; ++i)   // rows past the last repeat it
      xo[i] = (uint32_t)(x_row<MODE, ROUTE>(a, b, min(m0 + i * 4 + q, rows - 1)) - from) * a.K * 2 +
              i16 * 16;
    u32x4 w[NT], x[XL];
    W4Scales<E, GB, Z> sc[NT], now[NT];
    auto load = [&](int s) {
      s = max(min(s, s1 - 1), 0);
      const int k = s * 128;   // lanes past K: an offset past the resource
#pragma unroll
      for (int i = 0; i < XL; ++i)
        x[i] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, k + i16 * 8 < a.K ? xo[i] : kNoX,
                                                         min(k, max(a.K - 8, 0)) * 2, 0));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        w[nt] = load_codes(src, wo[nt], s * 64);
        const int column = tile_column(n0, nt * 16, a.N);
        load_scales<E, GB, Z>(sc[nt], src, i16, scale_offset(s * GP, a.groups, column, a.N, a.some),
                              a.N * 2, scale_offset(a.groups, a.groups, column, a.N, a.some));
      }
    };
    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    load(s0);
#pragma clang loop unroll(disable)
    for (int s = s0; s < s1; ++s) {
#pragma unroll
      for (int i = 0; i < XL; ++i)
        *reinterpret_cast<u32x4*>(own_x + (i * 4 + q) * kManyRow + i16 * 16) = x[i];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int c = lane >> 2;
        *reinterpret_cast<u32x4*>(own_w + nt * 1024 +
                                  (4 * c + (((lane & 3) + (c >> 2)) & 3)) * 16) = w[nt];
        sc[nt].loaded();
        now[nt] = sc[nt];
      }
      wave_lds_sync();
      __builtin_amdgcn_sched_barrier(0);
      load(s + 1);
      __builtin_amdgcn_sched_barrier(0);
      u32x4 v[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        v[nt] = *reinterpret_cast<const u32x4*>(own_w + nt * 1024 +
                                                (4 * i16 + ((q + (i16 >> 2)) & 3)) * 16);
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        u32x4 xv[MT][GB];
        f32x4 xs[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          xs[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < GB; ++b) {
            xv[mt][b] = *reinterpret_cast<const u32x4*>(own_x + (mt * 16 + i16) * kManyRow +
                                                        (g * GB + b) * 64 + q * 16);
            xs[mt] = mfma16(E(), xv[mt][b], consts.ones, xs[mt]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          f32x4 tt[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) tt[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < GB; ++b) {
            const u32x4 c = codes8(consts, v[nt][g * GB + b]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) tt[mt] = mfma16(E(), xv[mt][b], c, tt[mt]);
          }
          const float scale = now[nt].scale(g), off = now[nt].offset(g);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[mt][nt][r] = fmaf(scale, fmaf(off, xs[mt][r], tt[mt][r]), acc[mt][nt][r]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      wave_lds_sync();
    }
    // the waves' sums, through the same memory
    static_assert(many_lds(MT, NT) >= kManyWaves * MT * 1024, "room for a tile's sums");
    float* s_part = reinterpret_cast<float*>(s_dyn);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      __syncthreads();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) s_part[((wave * MT + mt) * 4 + r) * 64 + lane] = acc[mt][nt][r];
      __syncthreads();
      for (int o = threadIdx.x; o < MT * 256; o += kManyThreads) {
        const int l = o & 63, r = (o >> 6) & 3, mt = o >> 8;
        const int64_t m = m0 + mt * 16 + (l >> 4) * 4 + r;
        const int col = n0 + nt * 16 + (l & 15);
        if (m < rows && col < a.N) {
          float v = 0.f;
#pragma unroll
          for (int u = 0; u < kManyWaves; ++u) v += s_part[((u * MT + mt) * 4 + r) * 64 + l];
          store_out<E, MODE>(a, first, m, col, v);
        }
      }
    }
    __syncthreads();
  }
}

// The rows of this block's expert, or of a dense product; false past the last expert.
template <W4Mode MODE, bool ROUTE>
__device__ __forceinline__ bool find_work(const W4Args& a, int columns, W4Work& b) {
  b = {column_tile() * columns, 0, 0, a.M, nullptr};
  if (MODE == kGather || MODE == kScatter) {
    W4Expert x;
    if constexpr (ROUTE) {
      __shared__ int s_rows[kW4Threads];   // the expert's pairs
      __shared__ int s_count[kW4MaxExperts], s_wave[kW4Waves];
      x = route_here(a, s_rows, s_count, s_wave);
      b.s_rows = s_rows;
    } else {
      x = find_expert(a);
    }
    b.e = x.e;
    b.first = x.first;
    b.rows = x.rows;
  }
  return b.rows > 0;
}

// One row (6144 x 12288, weights from HBM: 12.7 us a call, few_rows with 4 rows 16.7,
// many_rows 14.3).
template <typename E, int GB, bool Z, W4Mode MODE, bool ROUTE>
__global__ __launch_bounds__(kW4Threads) __attribute__((amdgpu_waves_per_eu(4))) void w4_one(
    const W4Args a) {
  extern __shared__ __align__(16) char s_dyn[];
  W4Work b;
  if (find_work<MODE, ROUTE>(a, 16 * a.tiles, b))
    few_rows<E, GB, Z, 1, MODE, ROUTE>(a, b, s_dyn);
}

// Experts of few rows, as each block finds them: the host knows a bound of the mean,
// which on one rank of many is far above it.
template <typename E, int GB, bool Z, W4Mode MODE, bool ROUTE>
__global__ __launch_bounds__(kW4Threads) __attribute__((amdgpu_waves_per_eu(4))) void w4_mixed(
    const W4Args a) {
  extern __shared__ __align__(16) char s_dyn[];
  W4Work b;
  if (!find_work<MODE, ROUTE>(a, 16 * a.tiles, b)) return;
  if (b.rows <= kFewRows || a.tiles < 2) {
    few_rows<E, GB, Z, 4, MODE, ROUTE>(a, b, s_dyn);
  } else {
    for (const int end = min(b.n0 + 16 * a.tiles, a.N); b.n0 < end; b.n0 += 32)
      many_rows<E, GB, Z, 1, 2, MODE, ROUTE>(a, b, s_dyn);
  }
}

template <typename E, int GB, bool Z, int MT, int NT, W4Mode MODE>
__global__ __launch_bounds__(kManyThreads) void w4_many(const W4Args a) {
  extern __shared__ __align__(16) char s_dyn[];
  W4Work b;
  if (find_work<MODE, false>(a, 16 * NT, b)) many_rows<E, GB, Z, MT, NT, MODE, false>(a, b, s_dyn);
}

// The second layer of a single token's few pairs (at most kTinyPairs): a block
// owns 16 columns of out and walks every local pair, its waves sharing K, so that
// the weighted sum needs neither a second launch nor memory between.  4096 x 2816,
// this kernel and the two launches: 2 pairs 7.2 and 8.8 us, 4 pairs 11.1 and 10.3,
// 8 pairs 20.3 and 14.4.
constexpr int kTinyPairs = 3;

struct W4TinyArgs {
  W4Args w;             // pairs, offsets: sorted_pairs, expert_offsets; ids, e0, n_pairs
  const float* add;
  float* out;
  int T;
};

template <typename E, int GB, bool Z>
__global__ __launch_bounds__(kW4Threads) void w4_scatter_tiny(const W4TinyArgs args) {
  typedef typename Elem<E>::type L;
  constexpr int PF = kAhead, GP = 4 / GB;
  const W4Args& a = args.w;
  __shared__ float s_part[kW4Waves][kTinyPairs][16];
  extern __shared__ __align__(16) char s_dyn[];   // one row of x a pair
  const W4Stage st = stage_at(s_dyn, a.blocks, a.n_pairs);
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int c16 = lane >> 2, q = lane & 3;
  const int n0 = column_tile() * 16;
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
  int lu = 0;   // the pair that is loaded
  W4Source src =
      source_of<Z>(a, units ? __builtin_amdgcn_readlane(ex, pair_of(0)) : 0, n0, 16);
  const uint32_t wo = (uint32_t)c16 * a.blocks * 64 + q * 16;
  const int last = scale_offset(a.groups, a.groups, n0, a.N, a.some);
  const int first_s = scale_offset(s0 * GP, a.groups, n0, a.N, a.some);
  const int w_last = max(s0 + steps - 1, 0) * 64;
  int lw = min(s0 * 64, w_last), ls = first_s, li = 0;
  auto load = [&](u32x4& wr, W4Scales<E, GB, Z>& sr) {
    wr = load_codes(src, wo, lw);
    load_scales<E, GB, Z>(sr, src, c16, ls, a.N * 2, last);
    const bool turn = ++li == steps;
    lw = turn ? s0 * 64 : min(lw + 64, w_last);
    ls = turn ? first_s : min(ls + a.N * (2 * GP), last);
    li = turn ? 0 : li;
    lu += turn ? 1 : 0;   // past the last pair: that one again
    const int at = pair_of(min(lu, max(units - 1, 0)));
    src = source_of<Z>(a, units ? __builtin_amdgcn_readlane(ex, at) : 0, n0, 16);
  };
#pragma unroll
  for (int p = 0; p < PF; ++p) {   // on one path and in the loop's order, as in few_rows
    load(w[p], sc[p]);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int u = 0; u < units; ++u) {
    const int64_t from = __builtin_amdgcn_readlane(row, pair_of(u));
    const L* xr = static_cast<const L*>(a.x) + from * a.K;
    for (int k = t * 8; k < a.blocks * 128; k += kW4Threads * 8) {
      u32x4 v = {0, 0, 0, 0};
      if (k < a.K) v = *reinterpret_cast<const u32x4*>(xr + k);
      stage_octet<E, true>(st, u, k >> 3, v, true);
    }
  }
  __syncthreads();
  const W4Consts<E> consts;
  float acc = 0.f;
  int cu = 0, ci = 0;   // next to use
  auto use = [&](u32x4& wr, W4Scales<E, GB, Z>& sr) {
    W4Stage row = st;
    row.base += cu * st.stride;
    row.sums += cu * (st.sum_stride - st.stride);
    acc += one_row_step<E, GB, Z>(consts, wr, sr, row, s0 + ci);
    if (++ci == steps) {
      const float v = group_sum<4>(acc);
      if (q == 0) s_part[wave][cu][c16] = v;
      acc = 0.f;
      ci = 0;
      ++cu;
    }
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma clang loop unroll(disable)
  for (int i = 0; i < total; i += PF) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      if (i + p < total) use(w[p], sc[p]);
      load(w[p], sc[p]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
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

// Column tiles of a block: one until there are blocks enough to fill the chip twice
// over, then up to 8, which spread a block's fixed costs (4096 x 2816, 61 tokens: 8
// experts, 1 tile 16.3 us, 2 14.0, 4 15.7; 64 experts, 2 tiles 89 us, 4 83, 8 80).
constexpr int64_t kFewBlocks = 512;
int few_tiles(int64_t blocks) {
  int t = 1;
  while (t < 8 && blocks / (2 * t) >= kFewBlocks) t *= 2;
  return t;
}

template <typename E, int GB, bool Z, W4Mode MODE>
void launch_rows(W4Args a, int64_t most, dim3 grid, hipStream_t stream) {
#define FM_MANY(MT, NT)                                                                      \
  do {                                                                                       \
    if (MODE <= kDense32) grid.z = (unsigned)std::min<int64_t>(cdiv(a.M, 16 * MT), 65535);   \
    grid.x = (unsigned)cdiv(a.N, 16 * NT);                                                   \
    hipLaunchKernelGGL((w4_many<E, GB, Z, MT, NT, MODE>), grid, dim3(kManyThreads),          \
                       many_lds(MT, NT), stream, a);                                         \
  } while (0)
  constexpr bool ROUTE = MODE == kGather;   // there, only where the blocks route
  a.tiles = few_tiles((int64_t)grid.x * grid.y);
  const dim3 few((unsigned)cdiv(a.N, 16 * a.tiles), grid.y);
  if constexpr (MODE != kScatter) {
    if ((ROUTE ? a.n_pairs : a.M) == 1 && stage_bytes(a.blocks, 1) <= kFewLds) {
      hipLaunchKernelGGL((w4_one<E, GB, Z, MODE, ROUTE>), few, dim3(kW4Threads),
                         few_lds(a.blocks, 1), stream, a);
      return;
    }
  }
  if constexpr (MODE == kGather || MODE == kScatter) {
    if (ROUTE ? a.n_pairs > 0
              : most <= 2 * kMixedRows && stage_bytes(a.blocks, 4) <= kFewLds) {
      if (most > 2 * kFewRows) a.tiles = std::max(a.tiles, 2);
      hipLaunchKernelGGL((w4_mixed<E, GB, Z, MODE, ROUTE>),
                         dim3((unsigned)cdiv(a.N, 16 * a.tiles), grid.y), dim3(kW4Threads),
                         std::max<int64_t>(few_lds(a.blocks, 4), many_lds(1, 2)), stream, a);
      return;
    }
  }
  // Dense 6144 x 12288: 16 rows 16.7 us, with 32-row chunks 18.7; 32 rows 22.2 us,
  // 16-row chunks 25.1, 48-row ones 28.6; 48 rows 31.1, 32-row chunks 32.9.
  if (most <= 16) FM_MANY(1, 2);
  else if (most <= 32) FM_MANY(2, 2);
  else FM_MANY(3, 3);
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
  const size_t lds = stage_bytes(a.w.blocks, a.w.n_pairs);
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
  if (N >= (1ll << 22) || K >= (1ll << 22) || cdiv(K, group) * N >= (1ll << 29))
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
  a.some = K > 0;
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
  if (T >= (1ll << 31) || (T > 0 && T * hidden * 2 >= kNoX))
    return FM_ERR_UNSUPPORTED;   // 32-bit row offsets
  // A decode step's pairs are sorted by the product's own blocks (one launch); more
  // pairs, or rows too long for LDS, by the route's.
  const int64_t pairs = T * topk;
  const bool here = T > 0 && ffn > 0 && topk > 0 && T <= kW4Threads && pairs <= kW4Threads &&
                    n_local >= 1 && n_local <= kW4MaxExperts && pairs / n_local <= kMixedRows &&
                    hidden <= 4 * kFewLds && stage_bytes((int)cdiv(hidden, 128), 4) <= kFewLds;
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
  a.some = hidden > 0;
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
  if (T >= (1ll << 31) || T * topk >= (1ll << 31) || hidden >= (1ll << 22)) return 0;
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
  if (T >= (1ll << 31) || T * topk >= (1ll << 31)) return FM_ERR_UNSUPPORTED;
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
  a.some = ffn > 0;
  a.topk = topk;
  a.n_local = n_local;
  const int64_t pairs = T * topk;
  if (pairs <= kTinyPairs && stage_bytes(a.blocks, pairs) <= kFewLds) {
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
