// Top-k expert choice from router logits, forward and backward.
//
// Forward, per token with logits l, scores s (softmax or sigmoid of l; 0 where l is -inf
// or NaN, a masked expert):
//   key_e = l_e, or s_e + bias_e with a bias (the bias takes part in the choice only);
//   with groups, the experts of the topk_groups best groups stay (a group's score is the
//   sum of its topn best keys, of its topn best scores without a bias);
//   the k largest keys, ties to the lower index, masked experts after all others;
//   w_i = scale * s_i / sum of the chosen s, or scale * s_i.
// Two experts may be nearly equal, so a choice that goes by computed scores compares them
// in 64 bits: the answer is then that of the formula, not of a kernel's rounding.  A
// choice by the logits themselves compares the 32-bit logits.
//
// Layout: ROW lanes own a token and hold up to V consecutive experts each, so that every
// reduction over a token is a few DPP and lane-swap steps.  With groups, a group starts on a
// lane and takes a power of two of them (its last lanes may be short), so that a group's best
// meet in the first of those steps.  ROW is 16 (one DPP row; fewest instructions
// a token) or, for few tokens, 64 (a quarter of the dependent steps: latency).
//
// The choice: a token's keys become 24-bit steps below its largest key, over the span of its
// keys, with the expert's index in the low 8 bits.  These integers are distinct and order as
// (key descending, index ascending), so a round is the smallest difference to the last one
// taken, modulo 2^32: one subtract and half a three-way minimum an expert, with no search for
// the winner and no removal.  The comparison in 64 bits costs an fp64 exponential for every
// expert; instead the fp32 choice is certified.  With the bounds on the keys' errors below it
// is the formula's choice if neighbouring slots are further apart than the bound, or are equal
// because their inputs are.  Otherwise slots 0 .. k alone are put in order by 64-bit keys, one
// a lane, or, where more experts could belong to the choice, a wave makes it in 64 bits.
// (All in 64 bits, 16384 tokens of 256 experts with a sigmoid, a bias and groups took 78 us.)
//
// Measured, kernel alone, where an empty launch takes 4 us: 4 tokens x 256 experts (sigmoid,
// bias, 8 groups) 3.9 us; 16384 of them 15 us, bound by vector issue (1060 instructions a wave,
// four waves a SIMD, 70% of the slots; the 17 MB alone are 3.6 us); 32768 x 8, softmax, bf16 5.6 us.
#include <math.h>

#include <type_traits>

#include "mge_common.hpp"
#include "mge_internal.hpp"

namespace mge {

constexpr int TK_THREADS = 256;
constexpr int TK_ROW = 16;                       // lanes per token (backward)
constexpr int TK_TOKENS = TK_THREADS / TK_ROW;   // tokens per workgroup (backward)

// order-preserving unsigned keys; -0 and +0 are one value, NaN must not come in
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float val_of(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t u = uint64_t(__double_as_longlong(v + 0.0));
  return u ^ ((u >> 63) ? ~uint64_t(0) : (uint64_t(1) << 63));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_xchg(uint32_t v) {
  return uint32_t(__builtin_amdgcn_mov_dpp(int(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ uint64_t dpp_xchg(uint64_t v) {
  return (uint64_t(dpp_xchg<CTRL>(uint32_t(v >> 32))) << 32) | dpp_xchg<CTRL>(uint32_t(v));
}
template <int CTRL>
__device__ __forceinline__ float dpp_xchg(float v) { return __uint_as_float(dpp_xchg<CTRL>(__float_as_uint(v))); }
template <int CTRL>
__device__ __forceinline__ double dpp_xchg(double v) {
  return __longlong_as_double(int64_t(dpp_xchg<CTRL>(uint64_t(__double_as_longlong(v)))));
}
// the value of the lane's even and odd 16-lane row (lower and upper half of the wave)
template <bool HALF>
__device__ __forceinline__ U32Pair swap_rows(uint32_t v) { return HALF ? permlane32_swap(v, v) : permlane16_swap(v, v); }
template <bool HALF, typename Op>
__device__ __forceinline__ uint32_t across(uint32_t v, Op op) {
  const U32Pair p = swap_rows<HALF>(v);
  return op(p.a, p.b);
}
template <bool HALF, typename Op>
__device__ __forceinline__ float across(float v, Op op) {
  const U32Pair p = swap_rows<HALF>(__float_as_uint(v));
  return op(__uint_as_float(p.a), __uint_as_float(p.b));
}
template <bool HALF, typename Op>
__device__ __forceinline__ uint64_t across(uint64_t v, Op op) {
  const U32Pair h = swap_rows<HALF>(uint32_t(v >> 32)), l = swap_rows<HALF>(uint32_t(v));
  return op((uint64_t(h.a) << 32) | l.a, (uint64_t(h.b) << 32) | l.b);
}
template <bool HALF, typename Op>
__device__ __forceinline__ double across(double v, Op op) {
  const uint64_t u = uint64_t(__double_as_longlong(v));
  const U32Pair h = swap_rows<HALF>(uint32_t(u >> 32)), l = swap_rows<HALF>(uint32_t(u));
  return op(__longlong_as_double(int64_t((uint64_t(h.a) << 32) | l.a)), __longlong_as_double(int64_t((uint64_t(h.b) << 32) | l.b)));
}
// all-reduce over a token's lanes: lane ^ 1, lane ^ 2, mirror in 8, mirror in 16, then the
// wave's 16-lane rows
template <int ROW = TK_ROW, typename T, typename Op>
__device__ __forceinline__ T row_reduce(T v, Op op) {
  v = op(v, dpp_xchg<0xB1>(v));
  v = op(v, dpp_xchg<0x4E>(v));
  v = op(v, dpp_xchg<0x141>(v));
  v = op(v, dpp_xchg<0x140>(v));
  if constexpr (ROW == 64) {
    v = across<false>(v, op);
    v = across<true>(v, op);
  }
  return v;
}
struct MaxOp {
  template <typename T> __device__ T operator()(T a, T b) const { return a > b ? a : b; }
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct MinOp {
  template <typename T> __device__ T operator()(T a, T b) const { return a < b ? a : b; }
  __device__ float operator()(float a, float b) const { return fminf(a, b); }
};
struct AddOp { template <typename T> __device__ T operator()(T a, T b) const { return a + b; } };

// V logits of a row from expert e0 on, as fp32; from `end` on, and NaN: -inf
template <int V, typename LT>
__device__ __forceinline__ void load_logits(const LT* row, int e0, int end, bool vec, float* l) {
  constexpr int PER = 16 / sizeof(LT);
  if (V >= PER && vec && e0 + V <= end) {
#pragma unroll
    for (int i = 0; i < V / PER; ++i) {
      const uint4 q = *reinterpret_cast<const uint4*>(row + e0 + i * PER);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(LT) == 4) {
          l[i * PER + j] = __uint_as_float(w[j]);
        } else {
          l[i * PER + 2 * j] = __uint_as_float(w[j] << 16);
          l[i * PER + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (e0 + v < end) {
        if constexpr (sizeof(LT) == 4) l[v] = row[e0 + v];
        else l[v] = bf16_to_f32(row[e0 + v]);
      } else {
        l[v] = -INFINITY;
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = fmaxf(l[v], -INFINITY);   // (the maximum of a NaN and a number is the number)
}

// Differences to the largest logit that stay defined when both are infinite
template <typename F>
__device__ __forceinline__ F diff_to(F l, F m) { return l == m ? F(0) : l - m; }

// A round of the 64-bit choice: the wave's largest key, the lowest expert that has it, which
// then leaves.
template <int V>
__device__ __forceinline__ int take_best(uint64_t* key, int e0) {
  uint64_t best = key[0];
#pragma unroll
  for (int v = 1; v < V; ++v) best = key[v] > best ? key[v] : best;
  const uint64_t top = row_reduce<64>(best, MaxOp());
  uint32_t at = 0xffffffffu;
#pragma unroll
  for (int v = V - 1; v >= 0; --v) at = key[v] == top ? uint32_t(e0 + v) : at;
  at = row_reduce<64>(at, MinOp());
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = at == uint32_t(e0 + v) ? 0 : key[v];
  return int(at);
}

// min and max of numbers as one instruction (fminf and fmaxf first canonicalize what they
// cannot see to be the result of arithmetic)
__device__ __forceinline__ float max_num(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, INFINITY); }
__device__ __forceinline__ float min_num(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, -INFINITY); }
// the two largest so far, a >= b
__device__ __forceinline__ void two_best(float x, float& a, float& b) {
  b = __builtin_amdgcn_fmed3f(a, b, x);
  a = max_num(a, x);
}
__device__ __forceinline__ void two_best(double x, double& a, double& b) {
  b = x > a ? a : (x > b ? x : b);
  a = x > a ? x : a;
}

enum TopkGroups { TK_NO_GROUPS = 0, TK_LANES = 1, TK_WALK = 2 };   // no groups, whole lanes, any

// The lane's experts: from e0 up to (not including) end, at most V of them
struct LaneExperts {
  int e0, end;
};
template <int V, int GROUPS>
__device__ __forceinline__ LaneExperts lane_experts(int E, int G, int rl, int lanes) {
  if constexpr (GROUPS == TK_LANES) {
    const int g = rl >> (31 - __builtin_clz(lanes)), gs = E / G;   // (lanes is a power of two)
    const int e0 = g * gs + (rl - g * lanes) * V;
    return LaneExperts{e0, g < G ? (g + 1) * gs : 0};
  } else {
    return LaneExperts{rl * V, E};
  }
}

// Groups.  by[v]: what groups are ranked by (-inf: masked or no expert).  Sets the keys of the
// experts of dropped groups to `gone` and returns by how much the worst kept group is ahead of
// the best dropped one (+inf: nothing dropped that counts).  TK_WALK, for groups that do not
// fit the lanes: through LDS, where a lane walks a group.
template <int ROW, int V, int GROUPS, typename KF, typename UK>
__device__ __forceinline__ KF keep_groups(const KF* by, UK* key, UK gone, const TopkParams& p, int e0, int rl, int lanes,
                                          KF* lds) {
  const int E = p.E, G = p.G, gs = E / G;
  const KF none = -INFINITY;
  KF kept = INFINITY, dropped = none;
  if constexpr (GROUPS == TK_LANES) {
    KF a = by[0], b = none;
#pragma unroll
    for (int v = 1; v < V; ++v) two_best(by[v], a, b);
    auto merge = [&](KF a2, KF b2) {
      const KF lo = a < a2 ? a : a2;
      const KF hb = b > b2 ? b : b2;
      a = a > a2 ? a : a2;
      b = lo > hb ? lo : hb;
    };
    if (lanes >= 2) merge(dpp_xchg<0xB1>(a), dpp_xchg<0xB1>(b));
    if (lanes >= 4) merge(dpp_xchg<0x4E>(a), dpp_xchg<0x4E>(b));
    if (lanes >= 8) merge(dpp_xchg<0x141>(a), dpp_xchg<0x141>(b));
    if constexpr (ROW == 64) {
      if (lanes >= 16) merge(dpp_xchg<0x140>(a), dpp_xchg<0x140>(b));
      if (lanes >= 32) merge(__shfl_xor(a, 16), __shfl_xor(b, 16));
    }
    const KF mine = p.topn == 2 && b > none ? a + b : a;
    const int g = rl >> (31 - __builtin_clz(lanes));
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < G; ++j) {
      const KF x = __shfl(mine, j * lanes, ROW);
      before += (x > mine || (x == mine && j < g)) ? 1 : 0;
    }
    const bool keep = before < p.topg;
    if (!keep) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = gone;
    }
    if (g < G) {
      if (keep) kept = mine;
      else dropped = mine;
    }
  } else {
    KF* sk = lds;                // this token's share
    KF* sg = sk + E + 1;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e0 + v < E) sk[e0 + v] = by[v];
    __builtin_amdgcn_wave_barrier();   // a token's lanes are one wave, whose LDS accesses keep their order
    for (int g = rl; g < G; g += ROW) {
      KF a = none, b = none;
      for (int i = 0; i < gs; ++i) two_best(sk[g * gs + i], a, b);
      sg[g] = p.topn == 2 && b > none ? a + b : a;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (e0 + v < E) {
        const int g = (e0 + v) / gs;
        const KF mine = sg[g];
        int before = 0;
        for (int j = 0; j < G; ++j) {
          const KF x = sg[j];
          before += (x > mine || (x == mine && j < g)) ? 1 : 0;
        }
        if (before < p.topg) {
          kept = mine < kept ? mine : kept;
        } else {
          dropped = mine > dropped ? mine : dropped;
          key[v] = gone;
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
  kept = row_reduce<ROW>(kept, MinOp());
  dropped = row_reduce<ROW>(dropped, MaxOp());
  return dropped == none ? KF(INFINITY) : kept - dropped;
}

// The choice in 64 bits for one token, by a whole wave: expert of slot i in lane i.  Rare, so
// it is kept small (code that is not in the instruction cache costs more than its work).
template <int V, int GROUPS, typename LT>
__device__ __forceinline__ int choose64(const TopkParams& p, const LT* row, int lanes, double* lds) {
  const int rl = threadIdx.x & 63;
  const LaneExperts le = lane_experts<V, GROUPS>(p.E, p.G, rl, lanes);
  const int e0 = le.e0;
  float l[V];
  load_logits<V>(row, e0, le.end, false, l);
  float m = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
  m = row_reduce<64>(m, MaxOp());
  const bool sigmoid = p.score == MGE_SCORE_SIGMOID;
  double by[V];
  uint64_t key[V];
  double sum = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // e^-l, or e^(l - m) (0 for a masked expert)
    const double x = exp(sigmoid ? -double(l[v]) : l[v] == -INFINITY ? -INFINITY : diff_to<double>(l[v], m));
    by[v] = x;
    sum += x;
  }
  sum = row_reduce<64>(sum, AddOp());
#pragma unroll
  for (int v = 0; v < V; ++v) {
    by[v] = sigmoid ? 1.0 / (1.0 + by[v]) : sum > 0 ? by[v] / sum : 0.0;
    const bool in = e0 + v < le.end;
    double x = p.bias ? by[v] + double(in ? p.bias[e0 + v] : 0.f) : double(l[v]);
    if (l[v] == -INFINITY || !(x == x)) x = -INFINITY;
    key[v] = in ? key_of(x) : 0;
    if (p.bias || p.topn == 1 || x == -INFINITY) by[v] = x;
  }
  if constexpr (GROUPS != TK_NO_GROUPS) keep_groups<64, V, GROUPS>(by, key, uint64_t(0), p, e0, rl, lanes, lds);
  int mine = 0;
#pragma unroll 1
  for (int r = 0; r < p.k; ++r) {
    const int at = take_best<V>(key, e0);
    if (rl == r) mine = at;
  }
  return mine;
}

// BY_SCORE: the choice needs the scores (a bias, or groups ranked by a sum of two scores)
template <int ROW, int V, typename LT, bool BY_SCORE, int GROUPS>
__global__ __launch_bounds__(TK_THREADS) void route_topk2_kernel(TopkParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int rl = tid & (ROW - 1);
  const int64_t t = int64_t(blockIdx.x) * (TK_THREADS / ROW) + tid / ROW;
  const bool live = t < p.T;
  const int E = p.E;
  const LaneExperts le = lane_experts<V, GROUPS>(E, p.G, rl, p.lanes);
  const int e0 = le.e0, end = le.end;
  const LT* row = static_cast<const LT*>(p.logits) + (live ? t : 0) * p.ld;
  // LDS of groups that walk: E + G + 2 values of up to 64 bits for each token
  float* walk = reinterpret_cast<float*>(reinterpret_cast<double*>(smem) + (tid / ROW) * (E + p.G + 2));
  float l[V];
  load_logits<V>(row, e0, end, p.vec, l);

  // keys x (-inf: masked) and what groups are ranked by, in fp32
  const bool sigmoid = p.score == MGE_SCORE_SIGMOID;   // uniform
  float x[V], by[V];
  float m = l[0], inv = 0.f;                           // softmax: the largest logit, 1 / sum
  if (!sigmoid && (BY_SCORE || !p.renorm)) {
    float sum = 0.f;
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
    m = row_reduce<ROW>(m, MaxOp());
#pragma unroll
    for (int v = 0; v < V; ++v) {
      by[v] = l[v] == -INFINITY ? 0.f : __expf(diff_to(l[v], m));
      sum += by[v];
    }
    sum = row_reduce<ROW>(sum, AddOp());
    inv = sum > 0.f ? 1.f / sum : 0.f;
  }
  if constexpr (BY_SCORE) {
    // (the branches are uniform and outside the loops, so that the loops are straight code)
    if (sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) by[v] = __builtin_amdgcn_rcpf(1.f + __expf(-l[v]));
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) by[v] *= inv;
    }
    if (p.bias) {
      float b[V];
      load_logits<V>(p.bias, e0, end, p.bvec, b);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float k = by[v] + b[v];
        x[v] = l[v] == -INFINITY ? -INFINITY : k;
        by[v] = x[v];
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[v] = l[v];
        by[v] = l[v] == -INFINITY ? -INFINITY : by[v];
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = by[v] = l[v];
  }

  // 24-bit steps below the largest key.  Masked experts: kMasked, in index order; keys under
  // -2^100 (masks by the type's lowest value) are left out of the span and share its last step.
  constexpr uint32_t kSteps = 0xfffff0u, kMasked = 0xfffffcu, kGone = 0xffffffffu;
  float hi = x[0], lo = INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    hi = max_num(hi, x[v]);
    lo = min_num(lo, x[v] > -0x1p100f ? x[v] : INFINITY);
  }
  hi = row_reduce<ROW>(hi, MaxOp());
  lo = row_reduce<ROW>(lo, MinOp());
  const float scale = hi > lo ? float(kSteps) / (hi - lo) : 1.f;
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // (where hi or the scale is not finite, many steps are equal, and checked below; NaN: 0)
    uint32_t q = uint32_t(fminf(fmaxf((hi - x[v]) * scale, 0.f), float(kSteps)));
    q = x[v] == -INFINITY ? kMasked : q;
    key[v] = (q << 8) | uint32_t(e0 + v);
  }
  if (!p.full) {   // uniform: some lanes have fewer than V experts
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e0 + v >= end) key[v] = kGone;
  }
  // Bound on how far the difference of two fp32 keys is from the formula's.  u = 2^-24.
  // Sigmoid: the argument's rounding moves s by |l| s (1 - s) 1.5 u < 0.4 u, exp, add and
  // reciprocal by under 3.5 u: 4 u.  Softmax: |l - m| s 1.5 u <= 0.6 u, exp, reciprocal and
  // product 5 u s, the sum V + 6 roundings: under 28 u s.  The bias adds u |key|.  Two keys,
  // and a margin of two.
  const float base = sigmoid ? 0x1p-20f : 0x1p-17f * inv;
  const float eps = p.bias ? base + 0x1p-22f * fmaxf(fabsf(hi), fabsf(lo)) : 0.f;
  bool again = false;               // the token needs the choice in 64 bits
  if constexpr (GROUPS != TK_NO_GROUPS) {
    const float ahead = keep_groups<ROW, V, GROUPS>(by, key, kGone, p, e0, rl, p.lanes, walk);
    if constexpr (BY_SCORE) again = !(ahead > 2.f * (p.bias ? eps : base));
  }
  // k + 1 rounds; lane r of the row keeps round r's
  uint32_t from = 0, slot = kGone;
  auto round = [&]() {
    uint32_t d = key[0] - from;
#pragma unroll
    for (int v = 1; v < V; ++v) d = min(d, key[v] - from);
    const uint32_t got = row_reduce<ROW>(d, MinOp()) + from;
    from = got == kGone ? got : got + 1;
    return got;
  };
#pragma unroll 1
  for (int r = 0; r <= p.k; ++r) {
    const uint32_t got = round();
    if (rl == r) slot = got;
  }
  int mine = int(slot & 255u);
  {
    // slot rl against slot rl + 1: a step is 2^-24 of the span, and subtract, product and
    // truncation move a key by up to 3 of them
    const uint32_t step = slot >> 8, next = dpp_xchg<0x101>(slot) >> 8;   // row_shl:1
    const int ni = int(dpp_xchg<0x101>(slot) & 255u);
    const uint32_t reach = 8u + uint32_t(fminf(eps * scale * 1.01f, 0x1p25f));
    bool close = rl < p.k && next < kMasked && next - step <= reach;
    if (__any(close)) {
      auto logit = [&](int e) {
        if constexpr (sizeof(LT) == 4) return float(row[e]);
        else return bf16_to_f32(row[e]);
      };
      const uint32_t last = __shfl(step, p.k - 1, ROW), out = round() >> 8;   // slots k - 1, k + 1
      const bool masked = step >= kMasked;
      const float lm = masked ? -INFINITY : logit(mine);
      // gap: slot k + 1 is clearly behind slot k - 1, the choice is among slots 0 .. k.  alike:
      // every expert left that could belong to the choice has the inputs of slot k - 1.
      const bool gap = out >= kMasked || out - last > reach;
      const uint32_t lkey = __shfl(slot, p.k - 1, ROW);
      const float ll = __shfl(lm, p.k - 1, ROW), lb = p.bias ? p.bias[lkey & 255u] : 0.f;
      bool other = false;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (key[v] > lkey && key[v] < (kMasked << 8) && (key[v] >> 8) - last <= reach)
          other = other || l[v] != ll || (p.bias && p.bias[e0 + v] != lb);
      const bool alike = row_reduce<ROW>(uint32_t(other), MaxOp()) == 0;
      // slots of equal inputs are in index order as they are
      if (close && step == next && (rl < p.k - 1 || gap || alike) && lm == logit(ni) && (!p.bias || p.bias[mine] == p.bias[ni]))
        close = false;
      // (a biased softmax needs the sum in 64 bits: left to the wave)
      const bool few = gap && (sigmoid || !p.bias);
      if (row_reduce<ROW>(uint32_t(close), MaxOp()) && !few) again = true;
      double d = lm;
      if (p.bias) d = masked ? double(-INFINITY) : 1.0 / (1.0 + exp(-double(lm))) + double(p.bias[mine]);
      int place = 0;
#pragma unroll 1
      for (int j = 0; j <= p.k; ++j) {
        const double o = __shfl(d, j, ROW);
        const int oi = __shfl(mine, j, ROW);
        if (o > d || (o == d && oi < mine)) ++place;
      }
      int got = mine;               // slot i takes the expert whose place is i
#pragma unroll 1
      for (int j = 0; j <= p.k; ++j) {
        const int pj = __shfl(place, j, ROW), ij = __shfl(mine, j, ROW);
        if (pj == rl) got = ij;
      }
      if (few && rl < p.k) mine = got;
    }
  }
  {
    // tokens that are still open: the whole wave chooses again for each
    for (uint64_t todo = __ballot(again && live); todo != 0;) {
      const int first = __builtin_ctzll(todo) & ~(ROW - 1);   // the token's first lane
      todo &= ROW == 64 ? 0 : ~(((uint64_t(1) << (ROW & 63)) - 1) << first);
      const int64_t tt = t - (lane / ROW) + first / ROW;
      constexpr int VW = ROW * V <= 64 ? 1 : ROW * V / 64;
      // (a group's experts on the wave's lanes; LDS: the share of the wave's first token)
      const int c = choose64<VW, GROUPS>(p, static_cast<const LT*>(p.logits) + tt * p.ld, p.lanes * V / VW,
                                        reinterpret_cast<double*>(smem) + ((tid & ~63) / ROW) * (E + p.G + 2));
      const int moved = __shfl(c, rl & 15);
      if ((lane & ~(ROW - 1)) == first) mine = moved;
    }
  }
  // weights: lane i of the row has choice i
  const bool have = rl < p.k;
  float li = -INFINITY;
  if (have) {
    if constexpr (sizeof(LT) == 4) li = row[mine];
    else li = bf16_to_f32(row[mine]);
    if (!(li == li)) li = -INFINITY;
  }
  float w;
  if (p.score == MGE_SCORE_SIGMOID) {
    // with c = min(0, the chosen logits' largest), s_i e^-c = 1 / (e^c + e^(c - l_i)): the
    // ratios stay defined when every s_i underflows
    float c = 0.f;
    if (p.renorm) c = fminf(0.f, row_reduce(li, MaxOp()));
    if (c == -INFINITY) c = 0.f;
    w = 1.f / (expf(c) + expf(c - li));
  } else {
    const float mm = p.renorm ? row_reduce(li, MaxOp()) : m;   // (lanes 0 .. k - 1 are in one row of 16)
    w = li == -INFINITY ? 0.f : expf(diff_to(li, mm));
    if (!p.renorm) w *= inv;
  }
  if (!have) w = 0.f;
  if (p.renorm) {
    const float total = row_reduce(w, AddOp());
    w = total > 0.f ? w / total : 0.f;
  }
  if (have && live) {
    p.topk_idx[t * p.k + rl] = mine;
    p.topk_prob[t * p.k + rl] = w * p.scale;
  }
}

// Backward.  With d_i = scale * d_prob_i over the chosen experts (an index outside [0, E)
// takes no part):
//   sigmoid               dl_i = d'_i s_i (1 - s_i),  d'_i = d_i, or renormalised
//                         (d_i - sum_j w_j d_j) / S  with w_j = s_j / S, S = sum s_j
//   softmax, renormalised dl_i = w_i (d_i - sum_j w_j d_j)   (all other terms cancel)
//   softmax               dl_e = s_e ([e chosen] d_e - sum_j s_j d_j) for every expert
// and 0 elsewhere.  The row is built in LDS (the chosen experts are scattered) and leaves
// as whole lines.  A repeated index adds its slots in slot order.  Bound by its writes:
// 16384 x 256 fp32 7.7 us, of which an empty launch is 4 (16.8 MB written).
template <int V, typename LT>
__global__ __launch_bounds__(TK_THREADS) void route_topk_bwd_kernel(TopkBwdParams p) {
  constexpr int LD = TK_ROW * V;
  __shared__ __attribute__((aligned(16))) float so[TK_TOKENS * LD];
  const int tid = threadIdx.x;
  const int rl = tid & (TK_ROW - 1);
  const int tok = tid / TK_ROW;
  const int64_t t = int64_t(blockIdx.x) * TK_TOKENS + tok;
  const bool live = t < p.T;
  const int E = p.E, e0 = rl * V;
  const LT* row = static_cast<const LT*>(p.logits) + (live ? t : 0) * p.ld;
  const bool dense = p.score != MGE_SCORE_SIGMOID && !p.renorm;   // uniform
  bool have = live && rl < p.k;
  const int idx = have ? p.topk_idx[t * p.k + rl] : -1;
  have = have && idx >= 0 && idx < E;
  const float d = have ? p.d_prob[t * p.k + rl] * p.scale : 0.f;
  float li = -INFINITY;
  if (have) {
    if constexpr (sizeof(LT) == 4) li = row[idx];
    else li = bf16_to_f32(row[idx]);
    if (!(li == li)) li = -INFINITY;
  }
  float g;   // gradient of slot rl's logit
  if (dense) {
    float l[V];
    load_logits<V>(row, e0, E, p.vec, l);
    float m = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
    m = row_reduce(m, MaxOp());
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      l[v] = l[v] == -INFINITY ? 0.f : expf(diff_to(l[v], m));
      sum += l[v];
    }
    sum = row_reduce(sum, AddOp());
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const float s = li == -INFINITY ? 0.f : expf(diff_to(li, m)) * inv;
    const float dot = row_reduce(s * d, AddOp());
    g = s * d;
#pragma unroll
    for (int v = 0; v < V; ++v) so[tok * LD + e0 + v] = -(l[v] * inv) * dot;
  } else {
    // (every thread 16 bytes of a line, so that the zeros meet no bank conflicts)
#pragma unroll
    for (int i = tid * 4; i < TK_TOKENS * LD; i += TK_THREADS * 4) *reinterpret_cast<float4*>(so + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.score == MGE_SCORE_SIGMOID) {
      if (p.renorm) {
        float c = fminf(0.f, row_reduce(li, MaxOp()));
        if (c == -INFINITY) c = 0.f;
        float w = have ? 1.f / (expf(c) + expf(c - li)) : 0.f;
        const float sum = row_reduce(w, AddOp());
        w = sum > 0.f ? w / sum : 0.f;
        const float dot = row_reduce(w * d, AddOp());
        g = w * (d - dot) / (1.f + expf(li));          // 1 - s_i = 1 / (1 + e^l)
      } else {
        const float s = 1.f / (1.f + expf(-li));
        g = d * s / (1.f + expf(li));
      }
    } else {
      const float m = row_reduce(li, MaxOp());
      float w = li == -INFINITY ? 0.f : expf(diff_to(li, m));
      const float sum = row_reduce(w, AddOp());
      w = sum > 0.f ? w / sum : 0.f;
      const float dot = row_reduce(w * d, AddOp());
      g = w * (d - dot);
    }
  }
  // slots that share an expert: the first of them adds them up
  float total = 0.f;
  bool first = have;
  for (int j = 0; j < p.k; ++j) {
    const int oi = __shfl(have ? idx : -1, j, TK_ROW);
    const float og = __shfl(g, j, TK_ROW);
    if (oi == idx) {
      total += og;
      if (j < rl) first = false;
    }
  }
  lds_barrier();
  if (first) so[tok * LD + idx] += total;
  lds_barrier();
  // the rows of the workgroup are contiguous in the output: 16 bytes a thread where rows are
  // whole numbers of them
  const int64_t t0 = int64_t(blockIdx.x) * TK_TOKENS;
  const int rows = int(p.T - t0 < TK_TOKENS ? p.T - t0 : TK_TOKENS);
  LT* out = static_cast<LT*>(p.d_logits) + t0 * E;
  constexpr int PER = 16 / sizeof(LT);
  if (p.ovec) {   // uniform
    const int n = E / PER;
    for (int i = tid; i < rows * n; i += TK_THREADS) {
      const int r = E == LD ? 0 : i / n;   // (uniform; whole rows follow one another)
      const float* f = so + r * LD + (i - r * n) * PER;
      uint4 q;
      if constexpr (sizeof(LT) == 4) {
        q = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      } else {
        q = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
      }
      reinterpret_cast<uint4*>(out)[i] = q;
    }
  } else {
    for (int i = tid; i < rows * E; i += TK_THREADS) {
      const int r = i / E;
      const float x = so[r * LD + (i - r * E)];
      if constexpr (sizeof(LT) == 4) out[i] = x;
      else out[i] = f32_to_bf16(x);
    }
  }
}

template <typename F>
static void with_width(int E, F&& f) {
  if (E <= 16) f(std::integral_constant<int, 1>{});
  else if (E <= 32) f(std::integral_constant<int, 2>{});
  else if (E <= 64) f(std::integral_constant<int, 4>{});
  else if (E <= 128) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

// Tokens up to which a token takes a whole wave: the chip's SIMDs have few waves each then,
// and the call is as long as one wave's chain of dependent steps.
constexpr int64_t TK_WAVE_TOKENS = 2048;
// Tokens of one launch, which has to stay below 2^32 threads (64 a token at most); more of them
// follow in further launches.
constexpr int64_t TK_LAUNCH_TOKENS = int64_t(1) << 25;

template <int ROW, int V, typename LT, int GROUPS>
static void launch_topk_form(const TopkParams& p, bool by_score, hipStream_t s) {
  const int tokens = TK_THREADS / ROW;
  const dim3 grid(unsigned((p.T + tokens - 1) / tokens)), block(TK_THREADS);
  const unsigned lds = GROUPS == TK_WALK ? unsigned(tokens * (p.E + p.G + 2) * 8) : 0u;
  if (by_score) hipLaunchKernelGGL((route_topk2_kernel<ROW, V, LT, true, GROUPS>), grid, block, lds, s, p);
  else hipLaunchKernelGGL((route_topk2_kernel<ROW, V, LT, false, GROUPS>), grid, block, lds, s, p);
}

template <int ROW, int V>
static void launch_topk_row(TopkParams p, int dtype, bool by_score, bool groups, hipStream_t s) {
  p.full = p.E == ROW * V;   // (groups: then every group is whole lanes too)
  auto form = [&](auto lt) {
    using LT = decltype(lt);
    if (!groups) launch_topk_form<ROW, V, LT, TK_NO_GROUPS>(p, by_score, s);
    else if (p.lanes > 0) launch_topk_form<ROW, V, LT, TK_LANES>(p, by_score, s);
    else if constexpr (ROW == 64 && V == 4) launch_topk_form<ROW, V, LT, TK_WALK>(p, by_score, s);
  };
  if (dtype == MGE_DTYPE_F32) form(float{});
  else form(uint16_t{});
}

// The fewest experts a lane (a power of two up to vmax) with which a token's experts fit `row`
// lanes, each group on its own power of two of them; 0: they do not.  *lanes: a group's.
static int fit_lanes(int row, int vmax, int G, int gs, int* lanes) {
  for (int v = 1; v <= vmax; v *= 2)
    for (int n = 1; n * G <= row; n *= 2)
      if (n * v >= gs) {
        *lanes = n;
        return v;
      }
  return 0;
}

mge_status launch_topk(const TopkParams& p0, int dtype, hipStream_t s) {
  if (p0.T <= 0) return MGE_OK;
  TopkParams p = p0;
  const bool groups = p.G > 1 && p.topg < p.G;
  const bool by_score = p.bias != nullptr || (groups && p.topn == 2);
  const int G = groups ? p.G : 1, gs = p.E / G;
  int l16 = 0, l64 = 0;
  const int v16 = fit_lanes(16, 16, G, gs, &l16), v64 = fit_lanes(64, 4, G, gs, &l64);
  // 16-byte reads: a group's first expert has to be aligned too
  if (groups && (gs * (dtype == MGE_DTYPE_F32 ? 4 : 2)) % 16 != 0) p.vec = false;
  if (groups && (gs * 4) % 16 != 0) p.bvec = false;
  ProfScope prof(s, "route_topk2");
  const bool wave = v16 == 0 || (p0.T <= TK_WAVE_TOKENS && v16 > 1);
  // (v64 = 0: groups that fit no power of two of lanes walk LDS, a token a wave)
  p.lanes = wave ? (v64 ? l64 : 0) : l16;
  const int64_t esz = dtype == MGE_DTYPE_F32 ? 4 : 2;
  for (int64_t t0 = 0; t0 < p0.T; t0 += TK_LAUNCH_TOKENS) {
    p.T = p0.T - t0 < TK_LAUNCH_TOKENS ? p0.T - t0 : TK_LAUNCH_TOKENS;
    p.logits = static_cast<const uint8_t*>(p0.logits) + t0 * p.ld * esz;
    p.topk_idx = p0.topk_idx + t0 * p.k;
    p.topk_prob = p0.topk_prob + t0 * p.k;
    if (!wave) {
      if (v16 == 1) launch_topk_row<16, 1>(p, dtype, by_score, groups, s);
      else if (v16 == 2) launch_topk_row<16, 2>(p, dtype, by_score, groups, s);
      else if (v16 == 4) launch_topk_row<16, 4>(p, dtype, by_score, groups, s);
      else if (v16 == 8) launch_topk_row<16, 8>(p, dtype, by_score, groups, s);
      else launch_topk_row<16, 16>(p, dtype, by_score, groups, s);
    } else if (v64 == 1) {
      launch_topk_row<64, 1>(p, dtype, by_score, groups, s);
    } else if (v64 == 2) {
      launch_topk_row<64, 2>(p, dtype, by_score, groups, s);
    } else {
      launch_topk_row<64, 4>(p, dtype, by_score, groups, s);
    }
    const mge_status st = hip_check("route_topk2_kernel");
    if (st != MGE_OK) return st;
  }
  return MGE_OK;
}

mge_status launch_topk_bwd(const TopkBwdParams& p0, int dtype, hipStream_t s) {
  if (p0.T <= 0) return MGE_OK;
  TopkBwdParams p = p0;
  const int64_t esz = dtype == MGE_DTYPE_F32 ? 4 : 2;
  ProfScope prof(s, "route_topk_bwd");
  for (int64_t t0 = 0; t0 < p0.T; t0 += TK_LAUNCH_TOKENS) {
    p.T = p0.T - t0 < TK_LAUNCH_TOKENS ? p0.T - t0 : TK_LAUNCH_TOKENS;
    p.logits = static_cast<const uint8_t*>(p0.logits) + t0 * p.ld * esz;
    p.topk_idx = p0.topk_idx + t0 * p.k;
    p.d_prob = p0.d_prob + t0 * p.k;
    p.d_logits = static_cast<uint8_t*>(p0.d_logits) + t0 * p.E * esz;
    const dim3 grid(unsigned((p.T + TK_TOKENS - 1) / TK_TOKENS)), block(TK_THREADS);
    with_width(p.E, [&](auto w) {
      constexpr int V = decltype(w)::value;
      if (dtype == MGE_DTYPE_F32) hipLaunchKernelGGL((route_topk_bwd_kernel<V, float>), grid, block, 0, s, p);
      else hipLaunchKernelGGL((route_topk_bwd_kernel<V, uint16_t>), grid, block, 0, s, p);
    });
    const mge_status st = hip_check("route_topk_bwd_kernel");
    if (st != MGE_OK) return st;
  }
  return MGE_OK;
}

}  // namespace mge
