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
// Layout: 16 lanes (one DPP row) own a token and hold V consecutive experts each, so that
// every reduction over a token is 4 DPP steps and the lowest expert of equal keys is in the
// lowest lane.  Keys are unsigned integers in the order of the floating-point values:
// a masked expert is the key of -inf, an expert out of the choice (dropped group, past E,
// already chosen) is 0, below all of them.
#include <math.h>

#include "mge_common.hpp"
#include "mge_internal.hpp"

namespace mge {

constexpr int TK_THREADS = 256;
constexpr int TK_ROW = 16;                       // lanes per token
constexpr int TK_TOKENS = TK_THREADS / TK_ROW;   // tokens per workgroup
constexpr int TK_MAXK = 8;

// order-preserving unsigned keys; -0 and +0 are one value, NaN must not come in
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t u = uint64_t(__double_as_longlong(v + 0.0));
  return u ^ ((u >> 63) ? ~uint64_t(0) : (uint64_t(1) << 63));
}
__device__ __forceinline__ double val_of(uint64_t k) {
  return __longlong_as_double(int64_t(k ^ ((k >> 63) ? (uint64_t(1) << 63) : ~uint64_t(0))));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_xchg(uint32_t v) {
  return uint32_t(__builtin_amdgcn_mov_dpp(int(v), CTRL, 0xf, 0xf, false));
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
// all-reduce over the 16 lanes of a row: lane ^ 1, lane ^ 2, mirror in 8, mirror in 16
template <typename T, typename Op>
__device__ __forceinline__ T row_reduce(T v, Op op) {
  v = op(v, dpp_xchg<0xB1>(v));
  v = op(v, dpp_xchg<0x4E>(v));
  v = op(v, dpp_xchg<0x141>(v));
  return op(v, dpp_xchg<0x140>(v));
}
struct MaxOp { template <typename T> __device__ T operator()(T a, T b) const { return a > b ? a : b; } };
struct MinOp { template <typename T> __device__ T operator()(T a, T b) const { return a < b ? a : b; } };
struct AddOp { template <typename T> __device__ T operator()(T a, T b) const { return a + b; } };

// V logits of a row from expert e0, as fp32; past E and NaN: -inf
template <int V, typename LT>
__device__ __forceinline__ void load_logits(const LT* row, int e0, int E, bool vec, float* l) {
  constexpr int PER = 16 / sizeof(LT);
  if (V >= PER && vec && e0 + V <= E) {
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
      if (e0 + v < E) {
        if constexpr (sizeof(LT) == 4) l[v] = row[e0 + v];
        else l[v] = bf16_to_f32(row[e0 + v]);
      } else {
        l[v] = -INFINITY;
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = l[v] == l[v] ? l[v] : -INFINITY;
}

// Differences to the largest logit that stay defined when both are infinite
template <typename F>
__device__ __forceinline__ F diff_to(F l, F m) { return l == m ? F(0) : l - m; }

// k rounds over the row: the largest key, the lowest expert that has it.  Lane r of the row
// keeps the choice of round r.
template <int V, typename UK>
__device__ __forceinline__ int choose(UK* key, int e0, int k, int rl) {
  int mine = 0;
  for (int r = 0; r < k; ++r) {
    UK best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = key[v] > best ? key[v] : best;
    const UK top = row_reduce(best, MaxOp());
    uint32_t at = 0xffffffffu;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) at = key[v] == top ? uint32_t(e0 + v) : at;
    at = row_reduce(at, MinOp());
    if (rl == r) mine = int(at);
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = at == uint32_t(e0 + v) ? UK(0) : key[v];
  }
  return mine;
}

// BY_SCORE: the choice needs the scores (a bias, or groups ranked by a sum of two scores)
template <int V, typename LT, bool BY_SCORE>
__global__ __launch_bounds__(TK_THREADS) void route_topk2_kernel(TopkParams p) {
  typedef typename std::conditional<BY_SCORE, uint64_t, uint32_t>::type UK;
  constexpr int LD = TK_ROW * V + 1;
  __shared__ float sl[TK_TOKENS * LD];           // the logits, for the weights of the chosen
  __shared__ UK sk[TK_TOKENS * LD];              // keys the groups are ranked by
  __shared__ UK sg[TK_TOKENS * (TK_ROW * V + 1)];   // group scores
  const int tid = threadIdx.x;
  const int rl = tid & (TK_ROW - 1);
  const int tok = tid / TK_ROW;
  const int64_t t = int64_t(blockIdx.x) * TK_TOKENS + tok;
  const bool live = t < p.T;
  const int E = p.E, e0 = rl * V;
  float l[V];
  load_logits<V>(static_cast<const LT*>(p.logits) + (live ? t : 0) * p.ld, e0, E, p.vec, l);
#pragma unroll
  for (int v = 0; v < V; ++v) sl[tok * LD + e0 + v] = l[v];

  // the softmax's largest logit and sum (32 bits: for the weights)
  float m = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
  m = row_reduce(m, MaxOp());

  UK key[V];
  double sc[V];
  if constexpr (BY_SCORE) {
    double sum = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (p.score == MGE_SCORE_SIGMOID) {
        sc[v] = 1.0 / (1.0 + exp(-double(l[v])));
      } else {
        sc[v] = isinf(l[v]) && l[v] < 0 ? 0.0 : exp(diff_to<double>(l[v], m));
        sum += sc[v];
      }
    }
    if (p.score != MGE_SCORE_SIGMOID) {
      sum = row_reduce(sum, AddOp());
#pragma unroll
      for (int v = 0; v < V; ++v) sc[v] = sum > 0 ? sc[v] / sum : 0.0;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool off = isinf(l[v]) && l[v] < 0;
      double x = p.bias ? sc[v] + double(e0 + v < E ? p.bias[e0 + v] : 0.f) : double(l[v]);
      if (off || !(x == x)) x = -INFINITY;
      key[v] = key_of(x);
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key_of(l[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (e0 + v >= E) key[v] = 0;

  if (p.G > 1 && p.topg < p.G) {   // uniform
    // the groups' scores: lane j of the row takes groups j, j + 16, ...
    const int gs = E / p.G;
    const UK none = key_of(decltype(BY_SCORE ? 0.0 : 0.f)(-INFINITY));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      UK by = key[v];
      if constexpr (BY_SCORE) {
        if (!p.bias && p.topn == 2) by = key[v] > none ? key_of(sc[v]) : key[v];
      }
      sk[tok * LD + e0 + v] = by;
    }
    lds_barrier();
    for (int g = rl; g < p.G; g += TK_ROW) {
      UK a = 0, b = 0;
      for (int i = 0; i < gs; ++i) {
        const UK x = sk[tok * LD + g * gs + i];
        if (x > a) { b = a; a = x; }
        else if (x > b) b = x;
      }
      if constexpr (BY_SCORE) {
        if (p.topn == 2 && b > none) a = key_of(val_of(a) + val_of(b));
      }
      sg[tok * LD + g] = a;
    }
    lds_barrier();
    // a group stays if fewer than topg groups come before it
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = e0 + v;
      if (e < E) {
        const int g = e / gs;
        const UK mine = sg[tok * LD + g];
        int before = 0;
        for (int j = 0; j < p.G; ++j) {
          const UK x = sg[tok * LD + j];
          before += (x > mine || (x == mine && j < g)) ? 1 : 0;
        }
        if (before >= p.topg) key[v] = 0;
      }
    }
  }
  const int mine = choose<V>(key, e0, p.k, rl);
  lds_barrier();
  // weights: lane i of the row has choice i
  const bool have = rl < p.k;
  const float li = have ? sl[tok * LD + mine] : -INFINITY;
  float w;
  if (p.score == MGE_SCORE_SIGMOID) {
    // with c = min(0, the chosen logits' largest), s_i e^-c = 1 / (e^c + e^(c - l_i)): the
    // ratios stay defined when every s_i underflows
    float c = 0.f;
    if (p.renorm) c = fminf(0.f, row_reduce(li, MaxOp()));
    if (c == -INFINITY) c = 0.f;
    w = 1.f / (expf(c) + expf(c - li));
  } else {
    const float mm = p.renorm ? row_reduce(li, MaxOp()) : m;
    w = li == -INFINITY ? 0.f : expf(diff_to(li, mm));
    if (!p.renorm) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) sum += l[v] == -INFINITY ? 0.f : expf(diff_to(l[v], m));
      sum = row_reduce(sum, AddOp());
      w = sum > 0.f ? w / sum : 0.f;
    }
  }
  if (!have) w = 0.f;
  if (p.renorm) {
    const float sum = row_reduce(w, AddOp());
    w = sum > 0.f ? w / sum : 0.f;
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
// as whole lines.  A repeated index adds its slots in slot order.
template <int V, typename LT>
__global__ __launch_bounds__(TK_THREADS) void route_topk_bwd_kernel(TopkBwdParams p) {
  constexpr int LD = TK_ROW * V;
  __shared__ float so[TK_TOKENS * LD];
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
#pragma unroll
    for (int v = 0; v < V; ++v) so[tok * LD + e0 + v] = 0.f;
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
  // the rows of the workgroup are contiguous in the output
  const int64_t t0 = int64_t(blockIdx.x) * TK_TOKENS;
  const int rows = int(p.T - t0 < TK_TOKENS ? p.T - t0 : TK_TOKENS);
  LT* out = static_cast<LT*>(p.d_logits) + t0 * E;
  for (int i = tid; i < rows * E; i += TK_THREADS) {
    const int r = i / E;
    const float x = so[r * LD + (i - r * E)];
    if constexpr (sizeof(LT) == 4) out[i] = x;
    else out[i] = f32_to_bf16(x);
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

mge_status launch_topk(const TopkParams& p, int dtype, hipStream_t s) {
  if (p.T <= 0) return MGE_OK;
  const dim3 grid(unsigned((p.T + TK_TOKENS - 1) / TK_TOKENS)), block(TK_THREADS);
  const bool groups = p.G > 1 && p.topg < p.G;
  const bool by_score = p.bias != nullptr || (groups && p.topn == 2);
  ProfScope prof(s, "route_topk2");
  with_width(p.E, [&](auto w) {
    constexpr int V = decltype(w)::value;
    if (dtype == MGE_DTYPE_F32) {
      if (by_score) hipLaunchKernelGGL((route_topk2_kernel<V, float, true>), grid, block, 0, s, p);
      else hipLaunchKernelGGL((route_topk2_kernel<V, float, false>), grid, block, 0, s, p);
    } else {
      if (by_score) hipLaunchKernelGGL((route_topk2_kernel<V, uint16_t, true>), grid, block, 0, s, p);
      else hipLaunchKernelGGL((route_topk2_kernel<V, uint16_t, false>), grid, block, 0, s, p);
    }
  });
  return hip_check("route_topk2_kernel");
}

mge_status launch_topk_bwd(const TopkBwdParams& p, int dtype, hipStream_t s) {
  if (p.T <= 0) return MGE_OK;
  const dim3 grid(unsigned((p.T + TK_TOKENS - 1) / TK_TOKENS)), block(TK_THREADS);
  ProfScope prof(s, "route_topk_bwd");
  with_width(p.E, [&](auto w) {
    constexpr int V = decltype(w)::value;
    if (dtype == MGE_DTYPE_F32) hipLaunchKernelGGL((route_topk_bwd_kernel<V, float>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((route_topk_bwd_kernel<V, uint16_t>), grid, block, 0, s, p);
  });
  return hip_check("route_topk_bwd_kernel");
}

}  // namespace mge
