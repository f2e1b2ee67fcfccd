// Root-mean-square norm with the residual's addition, and its backward.
//
//   r = x + residual, rounded to x's type (the residual stream that goes on; the norm is taken of
//       the rounded sum, so that the backward, which reads it, sees the same values)
//   rstd = 1 / sqrt(mean(r^2) + eps),  y = r rstd w
// and with g = dy w, xhat = r rstd:
//   dx = rstd (g - xhat mean(g xhat)) + d_residual,  dw = sum over the rows of dy xhat
// Everything in between is fp32; y, the codes and dx are rounded once from it.
//
// Both are one pass over HBM, which bounds them.  A row stays in the registers of NT threads (64: a wave, no
// barrier; 256, 512: a workgroup), 8 consecutive values a thread and step, so that 16 neighbouring lanes hold one
// block of 128 and its scale is a maximum over a DPP row.  Measured on MI355X: forward of 16384 x 4096 bf16 with a
// residual, bf16 and 8-bit output 118 us (606 MB, 5.1 TB/s, a copy's rate), of 8 rows 3 us; backward of 16384 x 4096
// with a residual's gradient 95 us, of 2048 x 16384 45 us.
#include "mge_common.hpp"

#include "fp8b.hpp"

namespace mge {

// 8 values of a matrix in bf16 or fp32
template <bool F32>
struct Vec8;
template <>
struct Vec8<false> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p, int64_t i) { v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  // the values rounded to the type
  __device__ __forceinline__ void set(const float* f) { v = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7])); }
  __device__ __forceinline__ void store(void* p, int64_t i) const { *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = v; }
};
template <>
struct Vec8<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void set(const float* f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = a;
    q[1] = b;
  }
};
// ... in a type known at run time only
__device__ __forceinline__ void get8(const void* p, int64_t i, int f32, float* f) {
  if (f32) {
    Vec8<true> v;
    v.load(p, i);
    v.get(f);
  } else {
    Vec8<false> v;
    v.load(p, i);
    v.get(f);
  }
}

// Sum of v over the NT threads of a row; slot: LDS of NT / 64 floats (of the row's workgroup)
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum64(v);
  if constexpr (NT == 64) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  const float4 q = *reinterpret_cast<const float4*>(slot);
  v = (q.x + q.y) + (q.z + q.w);
  if constexpr (NT == 512) {
    const float4 u = *reinterpret_cast<const float4*>(slot + 4);
    v += (u.x + u.y) + (u.z + u.w);
  }
  return v;
}

constexpr int norm_threads(int nt) { return nt > 256 ? nt : 256; }

template <bool F32, int NT, int NV>
__global__ __launch_bounds__(norm_threads(NT)) void rmsnorm_kernel(NormParams p) {
  __shared__ __attribute__((aligned(16))) float s_part[2][NT == 512 ? 8 : 4];
  constexpr int RPW = norm_threads(NT) / NT;   // rows of a workgroup at a time
  const int t = threadIdx.x % NT;
  const int chunks = p.H / 8;
  const int kb = (p.H + FB - 1) / FB;
  const float inv_h = 1.f / float(p.H);
  int par = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * RPW; row0 < p.T; row0 += int64_t(gridDim.x) * RPW) {
    const int64_t row = row0 + threadIdx.x / NT;
    const bool live = row < p.T;   // (uniform over a row's threads)
    Vec8<F32> x[NV], res[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * NT + t;
      x[i].zero();
      res[i].zero();
      if (live && c < chunks) {
        x[i].load(p.x, row * p.x_ld + c * 8);
        if (p.residual) res[i].load(p.residual, row * p.H + c * 8);
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * NT + t;
      float f[8];
      x[i].get(f);
      if (p.residual) {
        float r[8];
        res[i].get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += r[j];
        x[i].set(f);
        x[i].get(f);
        if (live && c < chunks) x[i].store(p.res_out, row * p.H + c * 8);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
    }
    ss = row_sum<NT>(ss, s_part[par]);
    par ^= 1;
    const float rstd = 1.f / sqrtf(ss * inv_h + p.eps);
    if (live && t == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * NT + t;
      const bool in = live && c < chunks;
      float y[8], w[8];
      x[i].get(y);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 0.f;
      if (in) get8(p.weight, c * 8, p.w_f32, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = y[j] * rstd * w[j];
      if (p.y && in) {
        if (p.y_f32) {
          Vec8<true> v;
          v.set(y);
          v.store(p.y, row * p.H + c * 8);
        } else {
          Vec8<false> v;
          v.set(y);
          v.store(p.y, row * p.H + c * 8);
        }
      }
      if (p.codes) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = umax(m, __float_as_uint(y[j]) & 0x7fffffffu);
        const FbScale sc = fb_scale(row16_umax(m));
        if (in) {
          *reinterpret_cast<uint2*>(p.codes + row * p.H + c * 8) =
              make_uint2(fb_codes4(y[0] * sc.inv, y[1] * sc.inv, y[2] * sc.inv, y[3] * sc.inv),
                         fb_codes4(y[4] * sc.inv, y[5] * sc.inv, y[6] * sc.inv, y[7] * sc.inv));
          if ((t & 15) == 0) p.scales[row * kb + c / 16] = sc.s;
        }
      }
    }
  }
}

// The backward.  A thread's columns are the same in every row, so dw's share of a workgroup
// accumulates in registers; the workgroups' shares (in `part`) are summed by rmsnorm_dw_kernel in
// their order.  The next row's x and dy are on their way while a row is reduced.
template <bool F32, int NT, int NV>
__global__ __launch_bounds__(norm_threads(NT)) void rmsnorm_bwd_kernel(NormBwdParams p) {
  constexpr int RPW = norm_threads(NT) / NT;
  __shared__ __attribute__((aligned(16))) float s_part[2][NT == 512 ? 8 : 4];
  const int t = threadIdx.x % NT;
  const int chunks = p.H / 8;
  const float inv_h = 1.f / float(p.H);
  float dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  // x and dy as they are in memory (dy: 16 bytes more where it is fp32)
  Vec8<F32> xv[NV];
  Vec8<true> yv[NV];
  float rstd = 0.f;
  auto fetch = [&](int64_t row) {
    const bool live = row < p.T;
    rstd = live ? p.rstd[row] : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * NT + t;
      xv[i].zero();
      yv[i].zero();
      if (live && c < chunks) {
        xv[i].load(p.x, row * p.x_ld + c * 8);
        if (p.dy_f32) yv[i].load(p.dy, row * p.dy_ld + c * 8);
        else yv[i].a = *reinterpret_cast<const float4*>(static_cast<const uint16_t*>(p.dy) + row * p.dy_ld + c * 8);
      }
    }
  };
  int par = 0;
  const int64_t step = int64_t(gridDim.x) * RPW;
  constexpr bool NEXT = NT < 512 || NV < 4;   // (the longest rows leave no registers for it)
  if constexpr (NEXT) fetch(int64_t(blockIdx.x) * RPW + threadIdx.x / NT);
  for (int64_t row0 = int64_t(blockIdx.x) * RPW; row0 < p.T; row0 += step) {
    const int64_t row = row0 + threadIdx.x / NT;
    const bool live = row < p.T;
    if constexpr (!NEXT) fetch(row);
    float xh[NV][8], g[NV][8];
    const float rs = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xv[i].get(xh[i]);
      if (p.dy_f32) {
        yv[i].get(g[i]);
      } else {
        Vec8<false> y;
        y.v = make_uint4(__float_as_uint(yv[i].a.x), __float_as_uint(yv[i].a.y), __float_as_uint(yv[i].a.z), __float_as_uint(yv[i].a.w));
        y.get(g[i]);
      }
    }
    Vec8<F32> res[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * NT + t;
      res[i].zero();
      if (p.d_res && live && c < chunks) res[i].load(p.d_res, row * p.H + c * 8);
    }
    if constexpr (NEXT) fetch(row + step);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * NT + t;
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 0.f;
      if (c < chunks) get8(p.weight, c * 8, p.w_f32, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] *= rs;
        dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
        g[i][j] *= w[j];
        dot = fmaf(g[i][j], xh[i][j], dot);
      }
    }
    dot = row_sum<NT>(dot, s_part[par]) * inv_h;
    par ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * NT + t;
      if (live && c < chunks) {
        float d[8], f[8];
        res[i].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = rs * fmaf(-xh[i][j], dot, g[i][j]) + f[j];
        Vec8<F32> o;
        o.set(d);
        o.store(p.dx, row * p.H + c * 8);
      }
    }
  }
  if (!p.dw) return;
  if constexpr (RPW > 1) {
    // the waves' shares, added in their order
    extern __shared__ __attribute__((aligned(16))) float s_dw[];   // [RPW - 1][H]
    const int w = threadIdx.x / NT;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * NT + t;
      if (w > 0 && c < chunks) {
        float4* q = reinterpret_cast<float4*>(s_dw + (w - 1) * p.H + c * 8);
        q[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
        q[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
      }
    }
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * NT + t;
      if (c >= chunks) continue;
      for (int v = 0; v < RPW - 1; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] += s_dw[v * p.H + c * 8 + j];
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * NT + t;
    if (c >= chunks) continue;
    float4* q = reinterpret_cast<float4*>(p.part + int64_t(blockIdx.x) * p.H + c * 8);
    q[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
    q[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
  }
}

// dw[h] = sum over n rows of part[.][h], in a fixed order: 16 column groups of 4, 64 slices of rows
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float* part, int n, int H, float* dw) {
  __shared__ float4 s[64][16];
  const int x = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int c = int(blockIdx.x) * 16 + x;
  float4 a = make_float4(0, 0, 0, 0);
  if (c * 4 < H) {
#pragma unroll 4
    for (int r = k; r < n; r += 64) {
      const float4 v = *reinterpret_cast<const float4*>(part + int64_t(r) * H + c * 4);
      a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
  }
  s[k][x] = a;
  for (int o = 32; o > 0; o >>= 1) {
    __syncthreads();
    if (k < o) {
      const float4 v = s[k + o][x];
      a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
      s[k][x] = a;
    }
  }
  if (k == 0 && c * 4 < H) *reinterpret_cast<float4*>(dw + c * 4) = a;
}

// A wave a row for short rows, else a workgroup (us, a wave and a workgroup a row, bf16 with a residual and 8-bit
// output: 8192 x 512 7.7, 14.6; 8192 x 1024 13.8, 16.5; 1024 x 1024 4.1, 4.4; 16 x 1024 3.4, 2.9; 8192 x 2048 24.5,
// 24.2; 16384 x 4096 122, 118; 256 x 4096 8.1, 4.3).
static bool wave_rows(int64_t T, int H) { return H <= 512 || (H <= 1024 && T >= 1024); }
// Workgroups of a launch at most, 8 for each CU (16384 x 4096: 512 workgroups 126 us, 2048 120, 16384 122)
constexpr int kNormGrid = 2048;

template <bool F32, int NT, int NV>
static mge_status launch_fwd(const NormParams& p, hipStream_t s) {
  constexpr int threads = norm_threads(NT);
  const int64_t n = (p.T * NT + threads - 1) / threads;
  ProfScope prof(s, "rmsnorm_fwd");
  hipLaunchKernelGGL((rmsnorm_kernel<F32, NT, NV>), dim3(unsigned(n < kNormGrid ? n : kNormGrid)), dim3(threads), 0, s, p);
  return hip_check("rmsnorm_fwd");
}
template <bool F32>
static mge_status fwd_by_size(const NormParams& p, hipStream_t s) {
  const int ch = p.H / 8;
  if (wave_rows(p.T, p.H)) return ch <= 64 ? launch_fwd<F32, 64, 1>(p, s) : launch_fwd<F32, 64, 2>(p, s);
  if (ch <= 256) return launch_fwd<F32, 256, 1>(p, s);
  if (ch <= 512) return launch_fwd<F32, 256, 2>(p, s);
  if (ch <= 1024) return launch_fwd<F32, 256, 4>(p, s);
  return launch_fwd<F32, 256, 8>(p, s);
}
mge_status launch_rmsnorm(const NormParams& p, bool x_f32, hipStream_t s) {
  return x_f32 ? fwd_by_size<true>(p, s) : fwd_by_size<false>(p, s);
}

// The backward, in the same way (8192 x 512 10.1, 18.8; 8192 x 1024 16.7, 22.2; 1024 x 1024 7.3, 8.3; 256 x 1024 6.1,
// 6.0).  It keeps a row's xhat and g, the next row and dw: about 17 registers a value and thread, so that longer rows go
// to 512 threads before they would spill.
static bool wave_rows_bwd(int64_t T, int H) { return H <= 512 || (H <= 1024 && T >= 1024); }
// As many workgroups as the 256 CUs hold at once (bf16, 8192 x 4096: 512 workgroups 46 us, 768 39, 1024 48; 2048 x 8192:
// 512 31, 768 35; 8192 x 2048: 512 26.3, 1280 25.7; fp32 8192 x 4096: 512 74, 768 79); of the shortest rows fewer, since
// each costs a share of dw (8192 x 512: 512 10.0, 1280 12.5)
int rmsnorm_bwd_parts(int64_t T, int H) {
  const bool wave = wave_rows_bwd(T, H);
  const int64_t n = wave ? (T + 3) / 4 : T;
  const int most = H <= 512 ? 512 : (H <= 2048 && !wave ? 1280 : (H <= 4096 ? 768 : (H <= 8192 ? 512 : 256)));
  return int(n < most ? n : most);
}
template <bool F32, int NT, int NV>
static mge_status launch_bwd(const NormBwdParams& p, hipStream_t s) {
  const int n = rmsnorm_bwd_parts(p.T, p.H);
  const int lds = NT == 64 && p.dw ? 3 * p.H * 4 : 0;
  {
    ProfScope prof(s, "rmsnorm_bwd");
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<F32, NT, NV>), dim3(unsigned(n)), dim3(norm_threads(NT)), lds, s, p);
  }
  mge_status st = hip_check("rmsnorm_bwd");
  if (st != MGE_OK || !p.dw) return st;
  ProfScope prof(s, "rmsnorm_dw");
  hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3(unsigned((p.H / 4 + 15) / 16)), dim3(1024), 0, s, p.part, n, p.H, p.dw);
  return hip_check("rmsnorm_dw");
}
mge_status launch_rmsnorm_dw_zero(int H, float* dw, hipStream_t s) {
  ProfScope prof(s, "rmsnorm_dw");
  hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3(unsigned((H / 4 + 15) / 16)), dim3(1024), 0, s, nullptr, 0, H, dw);
  return hip_check("rmsnorm_dw");
}
template <bool F32>
static mge_status bwd_by_size(const NormBwdParams& p, hipStream_t s) {
  const int ch = p.H / 8;
  if (wave_rows_bwd(p.T, p.H)) return ch <= 64 ? launch_bwd<F32, 64, 1>(p, s) : launch_bwd<F32, 64, 2>(p, s);
  if (ch <= 256) return launch_bwd<F32, 256, 1>(p, s);
  if (ch <= 512) return launch_bwd<F32, 256, 2>(p, s);
  if (ch <= 1024) return launch_bwd<F32, F32 ? 512 : 256, F32 ? 2 : 4>(p, s);
  return launch_bwd<F32, 512, 4>(p, s);
}
mge_status launch_rmsnorm_bwd(const NormBwdParams& p, bool x_f32, hipStream_t s) {
  return x_f32 ? bwd_by_size<true>(p, s) : bwd_by_size<false>(p, s);
}

}  // namespace mge
