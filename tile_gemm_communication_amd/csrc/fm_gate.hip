// fm_gate.hip -- the router of an MoE layer: logits -> experts and weights of
// each token, expert counts and balance loss, and their gradient.
//
// A row of E logits lies in the registers of a group of LPR lanes, V a lane, so
// one load of the row serves the choice, the softmax and the balance sums (the
// operator moves little more than the logits).  Softmax statistics and weights
// are fp32; the keys of a biased choice are fp64, because a rounded score next
// to another one would change which experts are taken.
//
// Measured: 16384 x 64 bf16, top 2, with statistics 4.9 us (the steps of the choice one
// after another, not the 2.4 MB: two waves a SIMD, which wait 60% of their time) and 4.9
// for the join; one token 2.3.  65536 x 256, top 8, 72 us: 62% of the cycles issue the
// choice's vector instructions.  Backward of 65521 x 256 fp32, top 8, 39 us: 3.5 TB/s,
// vector instructions in 64% of the cycles and LDS exchanges in 31%.
#include <algorithm>

#include "fm_wave.hpp"

namespace fm {
namespace {

constexpr int kGateThreads = 512;       // forward: few blocks, whose partial sums one block joins
constexpr int kGateWaves = kGateThreads / 64;
constexpr int kGateBwdThreads = 256;
constexpr int kGateBwdWaves = kGateBwdThreads / 64;
// Four blocks a compute unit, each with several passes whose loads run one pass
// ahead (65521 x 256: 39.3 us; 2048 blocks 43.6, 4096 48.9).
constexpr int64_t kGateBwdBlocks = 1024;
constexpr int kGateMaxExperts = 1024;
constexpr int kGateMaxTopk = 16;
// Blocks whose partial sums one block joins (65536 x 256: 256 blocks 72 us, 512 63, 1024
// 78; 16384 x 256: 29, 34 and 34).
constexpr int kGateMaxBlocks = 256;
constexpr int kGateBatch = 18;          // loads in flight of the join: 256 blocks of 64 experts at once
constexpr int kGateFinishThreads = 1024;
constexpr float kNegInf = -__builtin_inff();

// exp(x) for x <= 0 (or NaN): 1 ulp of exp2 plus the argument's rounding.
__device__ __forceinline__ float exp_neg(float x) { return __expf(x); }
// 1 / x within 1 ulp.
__device__ __forceinline__ float recip(float x) { return __builtin_amdgcn_rcpf(x); }

// sigmoid(x) * exp(-m) with m <= 0: for shares and renormalised weights, which
// do not change with m; m near the largest min(x, 0) keeps them from vanishing.
__device__ __forceinline__ float sigmoid_num(float x, float m) {
  return exp_neg(fminf(x, 0.f) - m) * recip(1.f + exp_neg(-fabsf(x)));
}

// The numerators of a row's shares, given m (the largest x, for a sigmoid at most
// 0), and for a sigmoid dsig = sigmoid(-x).  Unless a row's m is far below 0,
// e = exp(-|x|) gives all of a sigmoid's terms.
template <int V>
__device__ __forceinline__ void share_nums(const float (&x)[V], bool sigmoid, float m, float (&p)[V],
                                           float (&dsig)[V]) {
  if (!sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = exp_neg(x[v] - m);
  } else {
    if (__any(m < -60.f)) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        p[v] = sigmoid_num(x[v], m);
        dsig[v] = sigmoid_num(-x[v], 0.f);
      }
    } else {
      const float scale = recip(exp_neg(m));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float e = exp_neg(-fabsf(x[v])), r = recip(1.f + e), er = e * r;
        p[v] = (x[v] > 0.f ? r : er) * scale;
        dsig[v] = x[v] > 0.f ? er : r;
      }
    }
  }
}

// Sum over the groups of LPR lanes of a wave, lane by lane, right in group 0.
template <int LPR>
__device__ __forceinline__ float sum_over_groups(float x) {
  auto rotated = [](float v, auto ctrl) {
    return __builtin_bit_cast(float, dpp<decltype(ctrl)::value>(__builtin_bit_cast(int, v)));
  };
  if constexpr (LPR <= 8) x += rotated(x, std::integral_constant<int, 0x128>());   // row_ror:8
  if constexpr (LPR <= 4) x += rotated(x, std::integral_constant<int, 0x124>());   // row_ror:4
  if constexpr (LPR <= 16) {
    const LanePair<float> p = lane_pair<16>(x);
    x = p.a + p.b;
  }
  if constexpr (LPR <= 32) {
    const LanePair<float> p = lane_pair<32>(x);
    x = p.a + p.b;
  }
  return x;
}

// The expert of slot v of a lane: V / 4 chunks of 4, chunk c at (c * LPR + sub) * 4.
template <int LPR>
__device__ __forceinline__ int slot_expert(int v, int sub) {
  return ((v >> 2) * LPR + sub) * 4 + (v & 3);
}

template <typename E, int LPR, int V>
__device__ __forceinline__ void load_row(const typename Elem<E>::type* row, int n, int sub,
                                         float (&x)[V]) {
  if (n % 4 == 0) {   // rows start on a 4-element boundary
#pragma unroll
    for (int c = 0; c < V / 4; ++c) {
      const int e = (c * LPR + sub) * 4;
      f32x4 q = {kNegInf, kNegInf, kNegInf, kNegInf};
      if (e < n) q = widen<E>(*reinterpret_cast<const typename Raw4<E>::type*>(row + e));
#pragma unroll
      for (int i = 0; i < 4; ++i) x[c * 4 + i] = q[i];
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = slot_expert<LPR>(v, sub);
      x[v] = e < n ? (float)row[e] : kNegInf;
    }
  }
}

struct GatePart {
  float sum;
  int32_t count;
};

struct GateArgs {
  const void* logits;
  const float* bias;
  const uint8_t* mask;
  int32_t* ids;
  float* weights;
  int32_t* counts;
  float* sums;
  float* loss;
  GatePart* part;   // [blocks, E + 1]; the last of a row counts the tokens
  int64_t T;
  int E, topk;
  int renorm, stats;
  float scale;
};

// counts, sums and loss from (sum, count) of each expert and the token count.
// Every thread of the block calls it; s_loss holds one double a wave.
template <typename Get>
__device__ __forceinline__ void gate_finish(const GateArgs& a, int n, Get get, double* s_loss) {
  const int t = threadIdx.x, waves = blockDim.x / 64;
  double dot = 0;
  for (int e = t; e < a.E; e += blockDim.x) {
    float sum;
    int cnt;
    get(e, sum, cnt);
    a.sums[e] = sum;
    a.counts[e] = cnt;
    dot += (double)sum * cnt;
  }
  dot = group_sum<64>(dot);
  if (t % 64 == 0) s_loss[t / 64] = dot;
  __syncthreads();
  if (t == 0) {
    double all = 0;
    for (int w = 0; w < waves; ++w) all += s_loss[w];
    const double nn = n > 0 ? (double)n : 1.0;
    a.counts[a.E] = n;
    a.loss[0] = (float)(all * a.E / (a.topk * nn * nn));
  }
}

template <typename E, int LPR, int V, bool BIAS, bool SIGMOID>
__global__ __launch_bounds__(kGateThreads) void gate_fwd(const GateArgs a) {
  constexpr int G = 64 / LPR;             // rows of a wave
  constexpr int RP = G * kGateWaves;      // rows of a block and pass
  __shared__ float s_x[RP][kGateMaxTopk];
  __shared__ int s_id[RP][kGateMaxTopk];
  __shared__ float s_m[RP], s_inv[RP];
  __shared__ int s_cnt[LPR * V + 1];
  __shared__ __align__(16) float s_sum[kGateWaves][LPR * V];
  __shared__ double s_loss[kGateWaves];
  typedef typename std::conditional<BIAS, double, float>::type Key;

  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int sub = lane % LPR, grp = lane / LPR, r = wave * G + grp;
  const int n = a.E, topk = a.topk;
  if (a.stats) {
    for (int e = t; e <= n; e += kGateThreads) s_cnt[e] = 0;
    __syncthreads();
  }
  float bias[V], acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    acc[v] = 0.f;
    const int e = slot_expert<LPR>(v, sub);
    bias[v] = BIAS && e < n ? a.bias[e] : 0.f;
  }
  int tokens = 0;
  for (int64_t base = (int64_t)blockIdx.x * RP; base < a.T; base += (int64_t)gridDim.x * RP) {
    const int64_t row = base + r;
    const bool live = row < a.T && (!a.mask || a.mask[row] != 0);
    float x[V];
    if (live) {
      load_row<E, LPR, V>(static_cast<const typename Elem<E>::type*>(a.logits) + row * n, n, sub, x);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = kNegInf;
    }
    if (a.stats || !SIGMOID) {
      float m = x[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
      m = group_max<LPR>(m);
      if (m == kNegInf) m = 0.f;          // every share becomes 0
      if (SIGMOID) m = fminf(m, 0.f);
      float p[V], dsig[V], sum = 0.f;
      share_nums<V>(x, SIGMOID, m, p, dsig);
#pragma unroll
      for (int v = 0; v < V; ++v) sum += p[v];
      sum = group_sum<LPR>(sum);
      const float inv = sum == 0.f ? 0.f : recip(sum);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += p[v] * inv;
      if (sub == 0) {
        s_m[r] = m;
        s_inv[r] = inv;
      }
    }
    Key key[V];
    if constexpr (BIAS) {
      if (SIGMOID) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const double sc = 1.0 / (1.0 + exp(-(double)x[v]));
          key[v] = x[v] == kNegInf ? (Key)kNegInf : sc + (Key)bias[v];
          __builtin_amdgcn_sched_barrier(0);   // one fp64 exponential at a time: else scalars spill
        }
      } else {
        double m = (double)x[0], sum = 0;
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmax(m, (double)x[v]);
        m = (double)group_max<LPR>((float)m);
        if (m == -__builtin_inf()) m = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          key[v] = exp((double)x[v] - m);
          sum += key[v];
          __builtin_amdgcn_sched_barrier(0);
        }
        sum = group_sum<LPR>(sum);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const double sc = key[v] / sum;   // sum is 0 only where every x is -inf
          key[v] = x[v] == kNegInf ? (Key)kNegInf : sc + (Key)bias[v];
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = x[v];
    }
    // topk times the largest key that is left; of equal ones the lowest expert.
    for (int k = 0; k < topk; ++k) {
      Key best = (Key)kNegInf;
      int at = 0x7fffffff;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (key[v] > best) {
          best = key[v];
          at = slot_expert<LPR>(v, sub);
        }
      auto join = [&](auto step) {
        constexpr int STEP = decltype(step)::value;
        if constexpr (STEP < LPR) {
          const LanePair<Key> pk = lane_pair<STEP>(best);
          const LanePair<int> pe = lane_pair<STEP>(at);
          const bool b = pk.b > pk.a || (pk.b == pk.a && pe.b < pe.a);
          best = b ? pk.b : pk.a;
          at = b ? pe.b : pe.a;
        }
      };
      join(std::integral_constant<int, 1>());
      join(std::integral_constant<int, 2>());
      join(std::integral_constant<int, 4>());
      join(std::integral_constant<int, 8>());
      join(std::integral_constant<int, 16>());
      join(std::integral_constant<int, 32>());
      if (best == (Key)kNegInf) at = -1;
      const int rel = at - sub * 4;   // of no slot where at is -1 or another lane's
      float mine = kNegInf;
      bool own = false;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool hit = rel == (v >> 2) * LPR * 4 + (v & 3);
        if (BIAS) {
          mine = hit ? x[v] : mine;
          own = own || hit;
        }
        key[v] = hit ? (Key)kNegInf : key[v];
      }
      if (BIAS ? own && at >= 0 : sub == 0) s_x[r][k] = BIAS ? mine : (float)best;
      if (sub == 0) s_id[r][k] = at;
    }
    wave_lds_sync();
    tokens += live && sub == 0;
    for (int i = lane; i < G * topk; i += 64) {
      const int q = wave * G + i / topk, k = i % topk;
      const int64_t to = base + q;
      if (to >= a.T) continue;
      const int id = s_id[q][k];
      float w = 0.f;
      if (id >= 0) {
        const float xk = s_x[q][k];
        if (a.renorm) {
          float m = kNegInf, sum = 0.f;
          for (int j = 0; j < topk; ++j) m = s_id[q][j] >= 0 ? fmaxf(m, s_x[q][j]) : m;
          if (SIGMOID) m = fminf(m, 0.f);
          for (int j = 0; j < topk; ++j)
            if (s_id[q][j] >= 0)
              sum += SIGMOID ? sigmoid_num(s_x[q][j], m) : exp_neg(s_x[q][j] - m);
          w = (SIGMOID ? sigmoid_num(xk, m) : exp_neg(xk - m)) * recip(sum);
        } else {
          w = SIGMOID ? sigmoid_num(xk, 0.f) : exp_neg(xk - s_m[q]) * s_inv[q];
        }
        w *= a.scale;
        if (a.stats) atomicAdd(&s_cnt[id], 1);
      }
      a.ids[to * topk + k] = id;
      a.weights[to * topk + k] = w;
    }
    wave_lds_sync();
  }
  if (!a.stats) return;
  tokens = group_sum<64>(tokens);
  if (lane == 0) atomicAdd(&s_cnt[n], tokens);
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = sum_over_groups<LPR>(acc[v]);
  if (grp == 0) {
#pragma unroll
    for (int c = 0; c < V / 4; ++c)
      *reinterpret_cast<f32x4*>(&s_sum[wave][(c * LPR + sub) * 4]) =
          f32x4{acc[c * 4], acc[c * 4 + 1], acc[c * 4 + 2], acc[c * 4 + 3]};
  }
  __syncthreads();
  auto block_sum = [&](int e) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kGateWaves; ++w) s += s_sum[w][e];
    return s;
  };
  if (gridDim.x == 1) {
    gate_finish(a, s_cnt[n], [&](int e, float& sum, int& cnt) {
      sum = block_sum(e);
      cnt = s_cnt[e];
    }, s_loss);
  } else {
    for (int e = t; e <= n; e += kGateThreads)
      a.part[(int64_t)blockIdx.x * (n + 1) + e] = {e < n ? block_sum(e) : 0.f, s_cnt[e]};
  }
}

// Joins the blocks' partial sums: S threads an expert, each over every S-th
// block, then the S parts in order.
__global__ __launch_bounds__(kGateFinishThreads) void gate_join(const GateArgs a, int blocks) {
  __shared__ GatePart s_part[2 * kGateFinishThreads];
  __shared__ double s_loss[kGateFinishThreads / 64];
  const int t = threadIdx.x, C = a.E + 1;   // columns
  const int S = C < kGateFinishThreads ? kGateFinishThreads / C : 1;
  // at most two columns a thread (C is at most one more than the threads)
  for (int i = t; i < S * C; i += kGateFinishThreads) {
    GatePart sum = {0.f, 0};
    const GatePart* from = a.part + i % C;
    // kGateBatch loads in flight; past the last block that one again, not added
    for (int b0 = i / C; b0 < blocks; b0 += kGateBatch * S) {
      GatePart p[kGateBatch];
#pragma unroll
      for (int u = 0; u < kGateBatch; ++u)
        p[u] = from[(int64_t)min(b0 + u * S, blocks - 1) * C];
#pragma unroll
      for (int u = 0; u < kGateBatch; ++u) {
        const bool in = b0 + u * S < blocks;
        sum.sum += in ? p[u].sum : 0.f;
        sum.count += in ? p[u].count : 0;
      }
    }
    s_part[i] = sum;
  }
  __syncthreads();
  auto get = [&](int e, float& s, int& c) {
    s = 0.f;
    c = 0;
    for (int j = 0; j < S; ++j) {
      s += s_part[j * C + e].sum;
      c += s_part[j * C + e].count;
    }
  };
  float none;
  int tokens;
  get(a.E, none, tokens);
  gate_finish(a, tokens, get, s_loss);
}

struct GateBwdArgs {
  const void* logits;
  const uint8_t* mask;
  const int32_t* ids;
  const float* d_weights;
  const int32_t* counts;
  const float* d_loss;
  void* d_logits;
  int64_t T;
  int E, topk;
  int renorm;
  float scale;
};

// With u, share p and the chosen slots' gradients d_k = scale * d_weights:
//   du = p * (a - sum p a) + slots,      a = d_loss * E / (topk n^2) * counts
//   slots: q_k (d_k - sum q d), q = softmax of u over the chosen (renormalised);
//          w_k d_k, less p * sum w d for a softmax score
//   dx = du (softmax) or du * sigmoid(-x).
template <typename E, int LPR, int V, bool SIGMOID>
__global__ __launch_bounds__(kGateBwdThreads) void gate_bwd(const GateBwdArgs a) {
  typedef typename Elem<E>::type L;
  constexpr int G = 64 / LPR;
  constexpr int RP = G * kGateBwdWaves;
  __shared__ float s_x[RP][kGateMaxTopk], s_d[RP][kGateMaxTopk], s_c[RP][kGateMaxTopk];
  __shared__ int s_id[RP][kGateMaxTopk];
  __shared__ float s_m[RP], s_inv[RP];
  __shared__ __align__(16) float s_du[RP][LPR * V];   // a row's du, where the slots are added
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int sub = lane % LPR, grp = lane / LPR, r = wave * G + grp;
  const int n = a.E, topk = a.topk;
  const L* logits = static_cast<const L*>(a.logits);
  float ae[V];
  {
    float coef = 0.f;
    if (a.counts) {
      const double nn = (double)a.counts[n];
      coef = nn > 0 ? (float)((double)a.d_loss[0] * n / (topk * nn * nn)) : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = slot_expert<LPR>(v, sub);
      ae[v] = a.counts && e < n ? coef * (float)a.counts[e] : 0.f;
    }
  }
  // A row and the first 64 slots of the wave's rows, asked for one pass ahead.
  float x[V];
  bool live;
  int next_id;
  float next_d;
  auto slot_of = [&](int64_t base, int i, int& id, float& d) {
    const int64_t at = base + wave * G + i / topk;
    id = -1;
    d = 0.f;
    if (i < G * topk && at < a.T) {
      id = a.ids[at * topk + i % topk];
      d = a.d_weights[at * topk + i % topk];
      if (a.mask && a.mask[at] == 0) id = -1;
    }
  };
  auto fetch = [&](int64_t base) {
    const int64_t row = base + r;
    live = row < a.T && (!a.mask || a.mask[row] != 0);
    if (live) {
      load_row<E, LPR, V>(logits + row * n, n, sub, x);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = kNegInf;
    }
    if (a.d_weights) slot_of(base, lane, next_id, next_d);
  };
  const int64_t pass = (int64_t)gridDim.x * RP;
  fetch((int64_t)blockIdx.x * RP);
  for (int64_t base = (int64_t)blockIdx.x * RP; base < a.T; base += pass) {
    const int64_t row = base + r;
    const bool now = live;
    // The chosen logits come from the row's copy in LDS (from memory they would be
    // a second wait).
    if (a.d_weights) {
      for (int i = lane; i < G * topk; i += 64) {
        const int q = wave * G + i / topk, k = i % topk;
        int id = next_id;
        float d = next_d;
        if (i >= 64) slot_of(base, i, id, d);
        if ((unsigned)id >= (unsigned)n) id = -1;
        s_id[q][k] = id;
        s_d[q][k] = id >= 0 ? d * a.scale : 0.f;
      }
#pragma unroll
      for (int c = 0; c < V / 4; ++c)
        *reinterpret_cast<f32x4*>(&s_du[r][(c * LPR + sub) * 4]) =
            f32x4{x[c * 4], x[c * 4 + 1], x[c * 4 + 2], x[c * 4 + 3]};
      wave_lds_sync();
      for (int i = lane; i < G * topk; i += 64) {
        const int q = wave * G + i / topk, k = i % topk, id = s_id[q][k];
        s_x[q][k] = id >= 0 ? s_du[q][id] : kNegInf;
      }
      wave_lds_sync();
    }
    float m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
    m = group_max<LPR>(m);
    if (m == kNegInf) m = 0.f;
    if (SIGMOID) m = fminf(m, 0.f);
    float p[V], dsig[V], sum = 0.f, dot = 0.f;
    share_nums<V>(x, SIGMOID, m, p, dsig);
    if (base + pass < a.T) fetch(base + pass);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      sum += p[v];
      dot += p[v] * ae[v];
    }
    sum = group_sum<LPR>(sum);
    dot = group_sum<LPR>(dot);
    const float inv = sum == 0.f ? 0.f : recip(sum);
    dot *= inv;
    if (a.d_weights) {
      if (sub == 0) {
        s_m[r] = m;
        s_inv[r] = inv;
      }
      wave_lds_sync();
      for (int i = lane; i < G * topk; i += 64) {
        const int q = wave * G + i / topk, k = i % topk;
        float c = 0.f;
        if (s_id[q][k] >= 0) {
          const float xk = s_x[q][k], d = s_d[q][k];
          if (a.renorm) {
            float mw = kNegInf, sw = 0.f, dw = 0.f;
            for (int j = 0; j < topk; ++j) mw = fmaxf(mw, s_x[q][j]);
            if (mw == kNegInf) mw = 0.f;
            if (SIGMOID) mw = fminf(mw, 0.f);
            for (int j = 0; j < topk; ++j) {
              const float w = SIGMOID ? sigmoid_num(s_x[q][j], mw) : exp_neg(s_x[q][j] - mw);
              sw += w;
              dw += w * s_d[q][j];
            }
            const float iw = sw == 0.f ? 0.f : recip(sw);
            const float w = SIGMOID ? sigmoid_num(xk, mw) : exp_neg(xk - mw);
            c = w * iw * (d - dw * iw);
          } else {
            c = d * (SIGMOID ? sigmoid_num(xk, 0.f) : exp_neg(xk - s_m[q]) * s_inv[q]);
          }
        }
        s_c[q][k] = c;
      }
      wave_lds_sync();
      if (!SIGMOID && !a.renorm)
        for (int k = 0; k < topk; ++k) dot += s_c[r][k];
    }
    float du[V];
#pragma unroll
    for (int v = 0; v < V; ++v) du[v] = p[v] * inv * (ae[v] - dot);
    if (a.d_weights) {
      // through LDS: the first slot of an expert adds what all slots of it give
#pragma unroll
      for (int c = 0; c < V / 4; ++c)
        *reinterpret_cast<f32x4*>(&s_du[r][(c * LPR + sub) * 4]) =
            f32x4{du[c * 4], du[c * 4 + 1], du[c * 4 + 2], du[c * 4 + 3]};
      wave_lds_sync();
      for (int i = lane; i < G * topk; i += 64) {
        const int q = wave * G + i / topk, k = i % topk, id = s_id[q][k];
        float add = 0.f;
        int first = k;
        for (int j = topk - 1; j >= 0; --j)
          if (s_id[q][j] == id) {
            add += s_c[q][j];
            first = j;
          }
        if (id >= 0 && first == k) s_du[q][id] += add;
      }
      wave_lds_sync();
#pragma unroll
      for (int c = 0; c < V / 4; ++c) {
        const f32x4 d = *reinterpret_cast<const f32x4*>(&s_du[r][(c * LPR + sub) * 4]);
#pragma unroll
        for (int i = 0; i < 4; ++i) du[c * 4 + i] = d[i];
      }
      wave_lds_sync();
    }
    if (SIGMOID) {
#pragma unroll
      for (int v = 0; v < V; ++v) du[v] *= dsig[v];
    }
    if (row < a.T) {
      L* to = static_cast<L*>(a.d_logits) + row * n;
#pragma unroll
      for (int v = 0; v < V; ++v) du[v] = now ? du[v] : 0.f;   // closed experts: share 0
      if (n % 4 == 0) {
#pragma unroll
        for (int c = 0; c < V / 4; ++c) {
          const int e = (c * LPR + sub) * 4;
          if (e < n) {
            const f32x4 q = {du[c * 4], du[c * 4 + 1], du[c * 4 + 2], du[c * 4 + 3]};
            *reinterpret_cast<typename Raw4<E>::type*>(to + e) = narrow<E>(q);
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int e = slot_expert<LPR>(v, sub);
          if (e < n) to[e] = (L)du[v];
        }
      }
    }
  }
}

// Lanes of a row: few, so that exchanges between lanes are few (16384 tokens, top 8:
// 64 experts with 8 lanes 13.8 us, 16 19.0; 256 experts with 16 lanes 28.9, 32 44.0),
// but 8 at least (32 experts 14.3 us, with 4 lanes 15.4; backward 6.9 and 8.9).
int gate_lanes(int E) {
  return E <= 64 ? 8 : E <= 256 ? 16 : E <= 512 ? 32 : 64;
}

// One block for two passes of rows: it joins its own sums, and a second pass costs
// less than the join's launch (4.9 us).
int gate_blocks(int64_t T, int E) {
  const int64_t rows = kGateThreads / gate_lanes(E);
  const int64_t passes = cdiv(T, rows);
  return (int)(passes <= 2 ? 1 : std::min<int64_t>(passes, kGateMaxBlocks));
}

size_t gate_ws(int64_t T, int E) {
  return (size_t)cdiv((int64_t)gate_blocks(T, E) * (E + 1) * sizeof(GatePart), 256) * 256;
}

fm_status_t check_gate(fm_dtype_t dt, int64_t T, int E, int topk, int score, int renorm,
                       const void* logits) {
  if (dt != FM_F16 && dt != FM_BF16 && dt != FM_F32) return FM_ERR_UNSUPPORTED;
  if (T < 0 || E < 1 || E > kGateMaxExperts || topk < 1 || topk > kGateMaxTopk || topk > E)
    return FM_ERR_INVALID_ARG;
  if ((score != FM_GATE_SOFTMAX && score != FM_GATE_SIGMOID) || renorm < 0 || renorm > 1)
    return FM_ERR_INVALID_ARG;
  if (T >= (1ll << 31) || T * topk >= (1ll << 31)) return FM_ERR_UNSUPPORTED;
  if (T > 0 && (!logits || !aligned16(logits))) return FM_ERR_INVALID_ARG;
  return FM_OK;
}

}  // namespace
}  // namespace fm

using namespace fm;

#define FM_GATE_LANES(CALL, E)                  \
  switch (gate_lanes(E)) {                      \
    case 8: CALL(8, 8); break;                  \
    case 16:                                    \
      if ((E) <= 128) CALL(16, 8);              \
      else CALL(16, 16);                        \
      break;                                    \
    case 32: CALL(32, 16); break;               \
    default: CALL(64, 16); break;               \
  }

extern "C" size_t fm_moe_gate_workspace_bytes(int64_t T, int32_t n_experts) {
  if (T < 0 || T >= (1ll << 31) || n_experts < 1 || n_experts > kGateMaxExperts) return 0;
  return gate_ws(T, n_experts);
}

extern "C" fm_status_t fm_moe_gate(fm_dtype_t dt, int64_t T, int32_t n_experts, int32_t topk,
                                   fm_gate_score_t score, int32_t renormalize, float scale,
                                   const void* logits, const float* bias,
                                   const uint8_t* token_mask, int32_t* topk_ids,
                                   float* topk_weights, int32_t* counts, float* prob_sums,
                                   float* loss, void* ws, size_t ws_bytes, hipStream_t stream) {
  const fm_status_t st = check_gate(dt, T, n_experts, topk, score, renormalize, logits);
  if (st != FM_OK) return st;
  const bool stats = counts || prob_sums || loss;
  if (T > 0 && (!topk_ids || !topk_weights)) return FM_ERR_INVALID_ARG;
  if (!aligned4(topk_ids) || !aligned4(topk_weights) || !aligned4(bias) || !aligned4(counts) ||
      !aligned4(prob_sums) || !aligned4(loss))
    return FM_ERR_INVALID_ARG;
  if (stats && (!counts || !prob_sums || !loss || !ws || !aligned16(ws) ||
                ws_bytes < gate_ws(T, n_experts)))
    return FM_ERR_INVALID_ARG;
  if (T == 0 && !stats) return FM_OK;
  GateArgs a = {};
  a.logits = logits;
  a.bias = bias;
  a.mask = token_mask;
  a.ids = topk_ids;
  a.weights = topk_weights;
  a.counts = counts;
  a.sums = prob_sums;
  a.loss = loss;
  a.T = T;
  a.E = n_experts;
  a.topk = topk;
  a.renorm = renormalize;
  a.stats = stats;
  a.scale = scale;
  int blocks = gate_blocks(T, n_experts);
  if (stats) {
    a.part = static_cast<GatePart*>(ws);
  } else {
    blocks = (int)std::min<int64_t>(cdiv(T, kGateThreads / gate_lanes(n_experts)), 4096);
  }
#define FM_GATE_FWD(LPR, V, B, S)                                                             \
  hipLaunchKernelGGL((gate_fwd<FM_E, LPR, V, B, S>), dim3(blocks), dim3(kGateThreads), 0, stream, \
                     a)
#define FM_GATE_CALL(LPR, V)                              \
  do {                                                    \
    if (score == FM_GATE_SIGMOID) {                       \
      if (bias) FM_GATE_FWD(LPR, V, true, true);          \
      else FM_GATE_FWD(LPR, V, false, true);              \
    } else {                                              \
      if (bias) FM_GATE_FWD(LPR, V, true, false);         \
      else FM_GATE_FWD(LPR, V, false, false);             \
    }                                                     \
  } while (0)
  if (dt == FM_F16) {
#define FM_E F16
    FM_GATE_LANES(FM_GATE_CALL, n_experts)
#undef FM_E
  } else if (dt == FM_BF16) {
#define FM_E BF16
    FM_GATE_LANES(FM_GATE_CALL, n_experts)
#undef FM_E
  } else {
#define FM_E F32
    FM_GATE_LANES(FM_GATE_CALL, n_experts)
#undef FM_E
  }
#undef FM_GATE_CALL
#undef FM_GATE_FWD
  if (stats && blocks > 1)
    hipLaunchKernelGGL(gate_join, dim3(1), dim3(kGateFinishThreads), 0, stream, a, blocks);
  return launch_status();
}

extern "C" fm_status_t fm_moe_gate_bwd(fm_dtype_t dt, int64_t T, int32_t n_experts,
                                       int32_t topk, fm_gate_score_t score, int32_t renormalize,
                                       float scale, const void* logits,
                                       const uint8_t* token_mask, const int32_t* topk_ids,
                                       const float* d_weights, const int32_t* counts,
                                       const float* d_loss, void* d_logits, hipStream_t stream) {
  const fm_status_t st = check_gate(dt, T, n_experts, topk, score, renormalize, logits);
  if (st != FM_OK) return st;
  if ((counts == nullptr) != (d_loss == nullptr)) return FM_ERR_INVALID_ARG;
  if (!aligned4(topk_ids) || !aligned4(d_weights) || !aligned4(counts) || !aligned4(d_loss))
    return FM_ERR_INVALID_ARG;
  if (T == 0) return FM_OK;
  if (!d_logits || !aligned16(d_logits) || (d_weights && !topk_ids)) return FM_ERR_INVALID_ARG;
  const int64_t bytes = T * n_experts * (dt == FM_F32 ? 4 : 2);
  const char *x = static_cast<const char*>(logits), *y = static_cast<const char*>(d_logits);
  if (x < y + bytes && y < x + bytes) return FM_ERR_INVALID_ARG;
  GateBwdArgs a = {};
  a.logits = logits;
  a.mask = token_mask;
  a.ids = topk_ids;
  a.d_weights = d_weights;
  a.counts = counts;
  a.d_loss = d_loss;
  a.d_logits = d_logits;
  a.T = T;
  a.E = n_experts;
  a.topk = topk;
  a.renorm = renormalize;
  a.scale = scale;
  const int blocks = (int)std::min<int64_t>(cdiv(T, kGateBwdThreads / gate_lanes(n_experts)),
                                           kGateBwdBlocks);
#define FM_GATE_CALL(LPR, V)                                                                  \
  do {                                                                                        \
    if (score == FM_GATE_SIGMOID)                                                             \
      hipLaunchKernelGGL((gate_bwd<FM_E, LPR, V, true>), dim3(blocks), dim3(kGateBwdThreads), 0, \
                         stream, a);                                                          \
    else                                                                                      \
      hipLaunchKernelGGL((gate_bwd<FM_E, LPR, V, false>), dim3(blocks), dim3(kGateBwdThreads), 0, \
                         stream, a);                                                          \
  } while (0)
  if (dt == FM_F16) {
#define FM_E F16
    FM_GATE_LANES(FM_GATE_CALL, n_experts)
#undef FM_E
  } else if (dt == FM_BF16) {
#define FM_E BF16
    FM_GATE_LANES(FM_GATE_CALL, n_experts)
#undef FM_E
  } else {
#define FM_E F32
    FM_GATE_LANES(FM_GATE_CALL, n_experts)
#undef FM_E
  }
#undef FM_GATE_CALL
  return launch_status();
}
