// Grouped products of FP8 operands with one fp32 scale per block of 128, for few rows per expert
// (token-by-token serving): C[r][n] = sum over blocks b of sa[r][b] sw[n / 128][b] (sum over k in b of
// A[r][k] W_e[n][k]).
//
// One read of the weights, so the kernels are built around that stream: a wave reads its rows' share of
// the weights straight into registers (16 rows x 128 bytes an instruction pair, whole lines), as the
// matrix unit's row operand, 16 tokens a block (MB = 1, 2, 4 blocks) as its columns; more rows than that in
// a group take further passes over the same weights.  Measured on MI355X: 8 x [4096][14336], 4 rows each, 86 us
// (5.4 TB/s), 64 rows each 217 us; 1 row x [2048][1024] 3.8 us, an empty launch about 3.  As in the tile kernels a block's products are
// summed from zero on the matrix unit (v_mfma_f32_16x16x128_f8f6f4: lane 16q + i feeds row / column i
// with bytes 16q .. 16q + 15 and 64 + 16q .. of the block; result register r is row 4q + r, column i)
// and added, scaled, to fp32 accumulators.  Rows past N, tokens past the group and bytes past K are
// outside the buffer resources' bounds and read as zeros.
#include "mge_common.hpp"

#include "fp8b.hpp"

namespace mge {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kSfOut = 0x80000000u;   // an offset past every bound

__device__ __forceinline__ __amdgpu_buffer_rsrc_t sf_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, int(bytes), 0x00020000);
}
__device__ __forceinline__ u32x4 sf_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, int(off), 0, 0);
}
__device__ __forceinline__ float sf_load4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, int(off), 0, 0));
}
__device__ __forceinline__ i32x8 sf_frag(u32x4 a, u32x4 b) {
  return i32x8{int(a.x), int(a.y), int(a.z), int(a.w), int(b.x), int(b.y), int(b.z), int(b.w)};
}
// a wave-uniform scale, by a scalar load
__device__ __forceinline__ float sf_uniform(const float* p, int i) {
  typedef const __attribute__((address_space(4))) float const_t;
  return reinterpret_cast<const_t*>(reinterpret_cast<uintptr_t>(p))[i];
}

// The group of this workgroup: the blockIdx.y-th expert that has rows (at most min(E, rows) of them, which
// is the grid); e < 0: none.  off, size: clamped into the rows of the groups.
struct SfGroup {
  int e, off, size;
};
__device__ __forceinline__ SfGroup sf_group(const FbGemm& p) {
  __shared__ int32_t s_pick, s_cnt[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  SfGroup g{0, 0, p.rows};
  if (p.sizes) {
    if (tid == 0) s_pick = -1;
    const bool some = tid < p.E && p.sizes[tid] > 0;
    const uint64_t mask = __ballot(some);
    if (lane == 0 && wave < 4) s_cnt[wave] = __popcll(mask);
    __syncthreads();
    int before = __popcll(mask & ((uint64_t(1) << lane) - 1));
    for (int w = 0; w < wave && w < 4; ++w) before += s_cnt[w];
    if (some && before == int(blockIdx.y)) s_pick = tid;
    __syncthreads();
    g.e = __builtin_amdgcn_readfirstlane(s_pick);
    if (g.e < 0) return g;
    g.off = p.offs[g.e];
    g.size = p.sizes[g.e];
    g.off = g.off < 0 ? 0 : (g.off > p.rows ? p.rows : g.off);
    g.size = g.size > p.rows - g.off ? p.rows - g.off : g.size;
    g.off = __builtin_amdgcn_readfirstlane(g.off);
    g.size = __builtin_amdgcn_readfirstlane(g.size);
  }
  return g;
}
// Byte offset of a group's row m in A (through the map), past every bound where there is none; the row itself
struct SfRow {
  uint32_t a, s;
};
__device__ __forceinline__ SfRow sf_row(const FbGemm& p, const SfGroup& g, int m, int KB) {
  if (m >= g.size) return SfRow{kSfOut, kSfOut};
  int src = g.off + m;
  if (p.map) src = p.map[src];
  if (src < 0 || src >= p.src_rows) return SfRow{kSfOut, kSfOut};
  return SfRow{uint32_t(src) * uint32_t(p.K), uint32_t(src) * uint32_t(KB) * 4};
}

// One step of U blocks: NB blocks of 16 weight rows times MB of 16 tokens.  w_off, rows: byte offsets of the
// lane's row; sw(b, kb): the weight scale.
template <int NB, int MB, int U, typename SW>
__device__ __forceinline__ void sf_step(f32x4 (&acc)[NB][MB], __amdgpu_buffer_rsrc_t rW, __amdgpu_buffer_rsrc_t rA,
                                        __amdgpu_buffer_rsrc_t rS, const uint32_t (&w_off)[NB], const SfRow (&rows)[MB], int kb0, int K,
                                        int KB, int q, SW&& sw) {
  u32x4 w[U][NB][2], a[U][MB][2];
  float ts[U][MB];
  const bool whole = (kb0 + U) * FB <= K;   // uniform
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t k = uint32_t(kb0 + u) * FB + 16 * q;
    const uint32_t o0 = whole || k < uint32_t(K) ? 0u : kSfOut, o1 = whole || k + 64 < uint32_t(K) ? 0u : kSfOut;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      w[u][b][0] = sf_load16(rW, (w_off[b] + k) | o0 | (w_off[b] & kSfOut));
      w[u][b][1] = sf_load16(rW, (w_off[b] + k + 64) | o1 | (w_off[b] & kSfOut));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t k = uint32_t(kb0 + u) * FB + 16 * q;
    const uint32_t o0 = whole || k < uint32_t(K) ? 0u : kSfOut, o1 = whole || k + 64 < uint32_t(K) ? 0u : kSfOut;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      a[u][m][0] = sf_load16(rA, (rows[m].a + k) | o0 | (rows[m].a & kSfOut));
      a[u][m][1] = sf_load16(rA, (rows[m].a + k + 64) | o1 | (rows[m].a & kSfOut));
      ts[u][m] = sf_load4(rS, (rows[m].s + uint32_t(kb0 + u) * 4) | (kb0 + u < KB ? 0u : kSfOut) | (rows[m].s & kSfOut));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float s = sw(b, kb0 + u < KB ? kb0 + u : KB - 1);
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const f32x4 z = {0.f, 0.f, 0.f, 0.f};
        const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(sf_frag(w[u][b][0], w[u][b][1]), sf_frag(a[u][m][0], a[u][m][1]),
                                                                         z, 0, 0, 0, 0, 0, 0);
        const float f = ts[u][m] * s;
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[b][m][r] = fmaf(d[r], f, acc[b][m][r]);
      }
    }
}

// C: a workgroup owns NB blocks of 16 weight rows; its W waves split K (U blocks of 128 at a time, then the
// next wave's follow) and add their partial sums through LDS in wave order.
template <int W, int NB, int MB, int U, bool F32>
__global__ __launch_bounds__(64 * W) void fb_stream_kernel(FbGemm p) {
  static_assert(W >= 4, "a thread for each of up to 256 experts");
  __shared__ __attribute__((aligned(16))) f32x4 red[W][NB * MB][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, q = lane >> 4;
  const SfGroup g = sf_group(p);
  if (g.e < 0) return;
  const int K = p.K, KB = (K + FB - 1) / FB;
  const int chunks = (KB + U - 1) / U;
  const __amdgpu_buffer_rsrc_t rW = sf_rsrc(p.W ? p.W[g.e] : p.Wv[g.e], uint32_t(p.N) * uint32_t(K));
  const float* wsc = p.W ? p.Ws[g.e] : p.Wsv[g.e];
  const __amdgpu_buffer_rsrc_t rA = sf_rsrc(p.A, uint32_t(p.src_rows) * uint32_t(K));
  const __amdgpu_buffer_rsrc_t rS = sf_rsrc(p.As, uint32_t(p.src_rows) * uint32_t(KB) * 4);
  const int n0 = int(blockIdx.x) * (NB * 16);
  uint32_t w_off[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) w_off[b] = n0 + b * 16 + i16 < p.N ? uint32_t(n0 + b * 16 + i16) * uint32_t(K) : kSfOut;
  auto sw = [&](int b, int kb) { return sf_uniform(wsc, min(n0 + b * 16, p.N - 1) / FB * KB + kb); };
  for (int m0 = 0; m0 < g.size; m0 += 16 * MB) {
    SfRow rows[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) rows[m] = sf_row(p, g, m0 + m * 16 + i16, KB);
    f32x4 acc[NB][MB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int m = 0; m < MB; ++m) acc[b][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int c = wave; c < chunks; c += W) sf_step<NB, MB, U>(acc, rW, rA, rS, w_off, rows, c * U, K, KB, q, sw);
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int m = 0; m < MB; ++m) red[wave][b * MB + m][lane] = acc[b][m];
    __syncthreads();
    for (int j = wave; j < NB * MB; j += W) {
      f32x4 c = red[0][j][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) {
        const f32x4 x = red[w][j][lane];
        c.x += x.x; c.y += x.y; c.z += x.z; c.w += x.w;
      }
      const int row = m0 + (j % MB) * 16 + i16;
      const int n = n0 + (j / MB) * 16 + 4 * q;
      if (row < g.size && n < p.N) {   // N is a multiple of 32
        const int64_t o = (int64_t(g.off) + row) * p.N + n;
        if constexpr (F32) *reinterpret_cast<float4*>(static_cast<float*>(p.C) + o) = make_float4(c.x, c.y, c.z, c.w);
        else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.C) + o) = make_uint2(bf16x2(c.x, c.y), bf16x2(c.z, c.w));
      }
    }
    __syncthreads();
  }
}

struct SwigluArgs {
  int rows, F, E;
  const float* prob;
  const int32_t *map, *sizes, *offs;
  uint8_t* codes;
  float* scales;
};

// h = p silu(G) U of fp32 rows [G U], one block of 128 for 16 lanes, 8 columns each.  A launch of its own: with the
// epilogue of the product above a workgroup would need all 256 weight rows of a block, and however its waves
// share them it reads slower and fills fewer CUs (whole MLP, fused and not: 16 tokens, top-2 of 8 experts
// 4096 x 14336 283 and 251 us; one token, 4096 x 4096 47 and 19 us).
__global__ __launch_bounds__(256) void fb_swiglu_kernel(SwigluArgs p, const float* gu, int64_t ld) {
  const int F = p.F, nb = (F + FB - 1) / FB;
  const int64_t blk = int64_t(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (blk >= int64_t(p.rows) * nb) return;
  const int r = int(blk / nb), b = int(blk - int64_t(r) * nb);
  if (p.map && p.map[r] < 0 && p.sizes) {   // (the same for the 16 lanes)
    // without a token: padding between the groups, whose G U nobody wrote, or a group's row of zeros
    bool mine = false;
    for (int e = threadIdx.x & 15; e < p.E; e += 16) mine |= r >= p.offs[e] && r - p.offs[e] < p.sizes[e];
    if (row16_umax(mine ? 1u : 0u) == 0) return;
  }
  const int f = b * FB + (threadIdx.x & 15) * 8;
  const bool in = f < F;
  float h[8];
  uint32_t am = 0;
  const float pr = p.prob ? p.prob[r] : 1.f;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    float4 g = make_float4(0, 0, 0, 0), u = g;
    if (in) {
      g = *reinterpret_cast<const float4*>(gu + int64_t(r) * 2 * F + f + i);
      u = *reinterpret_cast<const float4*>(gu + int64_t(r) * 2 * F + F + f + i);
    }
    h[i] = pr * silu_f(g.x) * u.x;
    h[i + 1] = pr * silu_f(g.y) * u.y;
    h[i + 2] = pr * silu_f(g.z) * u.z;
    h[i + 3] = pr * silu_f(g.w) * u.w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) am = umax(am, __float_as_uint(h[i]) & 0x7fffffffu);
  const FbScale sc = fb_scale(row16_umax(am));
  if (!in) return;
  *reinterpret_cast<uint2*>(p.codes + int64_t(r) * F + f) =
      make_uint2(fb_codes4(h[0] * sc.inv, h[1] * sc.inv, h[2] * sc.inv, h[3] * sc.inv),
                 fb_codes4(h[4] * sc.inv, h[5] * sc.inv, h[6] * sc.inv, h[7] * sc.inv));
  if ((threadIdx.x & 15) == 0) p.scales[ld > 0 ? int64_t(b) * ld + r : int64_t(r) * nb + b] = sc.s;
}
mge_status launch_fb_swiglu(const FbGemm& g, const float* gu, int64_t ld, hipStream_t s) {
  const int64_t blocks = int64_t(g.rows) * ((g.F + FB - 1) / FB);
  const SwigluArgs p{g.rows, g.F, g.E, g.prob, g.map, g.sizes, g.offs, g.h_codes, g.h_scales};
  ProfScope prof(s, "fp8_block_swiglu");
  hipLaunchKernelGGL(fb_swiglu_kernel, dim3(unsigned((blocks + 15) / 16)), dim3(256), 0, s, p, gu, ld);
  return hip_check("fp8_block_swiglu");
}

// Groups that can have rows: the kernels' grid in y
static unsigned groups_upper(const FbGemm& p) { return !p.sizes ? 1u : unsigned(p.E < p.total ? p.E : p.total); }

template <int W, int NB, int MB, int U>
static mge_status launch_store(const FbGemm& p, hipStream_t s) {
  const dim3 grid(unsigned((p.N + NB * 16 - 1) / (NB * 16)), groups_upper(p));
  ProfScope prof(s, "fp8_block_stream");
  if (p.out_f32) hipLaunchKernelGGL((fb_stream_kernel<W, NB, MB, U, true>), grid, dim3(64 * W), 0, s, p);
  else hipLaunchKernelGGL((fb_stream_kernel<W, NB, MB, U, false>), grid, dim3(64 * W), 0, s, p);
  return hip_check("fp8_block_stream");
}

mge_status launch_fb_stream(const FbGemm& p, hipStream_t s) {
  if (p.total <= 0 || p.rows <= 0) return MGE_OK;
  // Token blocks of a pass by the mean group (some groups are longer): 8 x [4096][14336], rows of each group 8, 16, 20, 32,
  // 48, 64: one block 92, 107, 177, 199, 283, 372 us, two 98, 112, 119, 140, 236, 267, four 126, 141, 146, 158, 187, 217.
  // One block of 16 weight rows a workgroup, four slices in flight, while two would leave CUs idle (1 row, [4096][4096],
  // 256 blocks: 6.1 us, two rows' blocks 7.9; 16 x [1024][2048], 1024 blocks: 11.3, 8.4).
  const int64_t blocks = int64_t((p.N + 15) / 16) * groups_upper(p);
  if (p.total > 32 * int64_t(p.E)) return launch_store<8, 2, 4, 2>(p, s);
  if (p.total > 12 * int64_t(p.E)) return launch_store<8, 2, 2, 2>(p, s);
  if (blocks < 1024) return launch_store<8, 1, 1, 4>(p, s);
  return launch_store<8, 2, 1, 2>(p, s);
}

}  // namespace mge
