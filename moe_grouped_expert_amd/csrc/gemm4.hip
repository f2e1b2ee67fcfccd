// Grouped products with MXFP4 weights for few rows per expert (token-by-token serving):
// C[r][n] = sum over k of A[r][k] W_e[n][k] for the rows r of expert e, A in MXFP8 or
// MXFP4, W in MXFP4, fp32 accumulation on the block-scaled matrix units.
//
// With few rows the product is one read of the weights, so the kernel is built around that
// stream.  A workgroup owns NB blocks of 16 weight rows of one expert; its 4 waves split K
// (a wave takes 4 steps of 128 elements, then the next wave's follow), read their share of
// those rows once, straight into registers, and add their partial sums through LDS at the
// end.  The weights are the matrix unit's row operand and up to 16 MB tokens its columns
// (v_mfma_scale_f32_16x16x128_f8f6f4); more rows than that in a group take further passes
// over the same weights, which then come from L2.
//   Operand layout (measured on gfx950): lane 16q + i feeds row / column i.  A 4-bit
//   operand is the 32 elements of K block q (16 bytes); an 8-bit one is elements
//   16q .. 16q + 15 and 64 + 16q .. 64 + 16q + 15 of the 128; both are scaled by the E8M0
//   byte of block q that the lane supplies.  Result lane 16q + i, register r: row 4q + r,
//   column i.
// Rows past N, tokens past the group and K blocks past the end are outside the buffer
// resources' bounds and read as zeros.
//
// SWIGLU: the 4 blocks are 32 gate rows and the 32 up rows of the same 32 ffn columns, and
// the epilogue writes h = p silu(G) U, quantized to MXFP8 (one block of 32 per token).
#include "mge_common.hpp"
#include "mge_internal.hpp"

#include <type_traits>

namespace mge {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int S4_WAVES = 4;
constexpr int S4_THREADS = 64 * S4_WAVES;
constexpr int S4_STEP = 128;     // elements of K per matrix instruction
constexpr int S4_U = 4;          // steps whose loads are in flight together
constexpr int kS4Rsrc = 0x00020000;
constexpr uint32_t kS4Out = 0x80000000u;   // an offset past every bound

__device__ __forceinline__ __amdgpu_buffer_rsrc_t s4_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, int(bytes), kS4Rsrc);
}
__device__ __forceinline__ u32x4 s4_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, int(off), 0, 0);
}
__device__ __forceinline__ uint32_t s4_load1(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b8(r, int(off), 0, 0);
}
__device__ __forceinline__ i32x8 s4_frag(u32x4 a, u32x4 b) {
  return i32x8{int(a.x), int(a.y), int(a.z), int(a.w), int(b.x), int(b.y), int(b.z), int(b.w)};
}

template <bool A4, int NB, int MB, bool SWIGLU, bool F32>
__global__ __launch_bounds__(S4_THREADS) void gemm4_stream_kernel(Gemm4Params p) {
  __shared__ __attribute__((aligned(16))) f32x4 red[S4_WAVES][NB * MB][64];
  __shared__ int32_t s_pick;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int i16 = lane & 15;
  const int q = lane >> 4;

  // the group of this workgroup: the blockIdx.y-th expert that has rows (there are at most
  // min(E, rows) of them, which is the grid)
  int e = 0;
  if (p.sizes) {
    if (tid == 0) s_pick = -1;
    __syncthreads();
    const bool some = tid < p.E && p.sizes[tid] > 0;
    const uint64_t mask = __ballot(some);
    __shared__ int32_t s_cnt[S4_WAVES];
    if (lane == 0) s_cnt[wave] = __popcll(mask);
    __syncthreads();
    int before = __popcll(mask & ((uint64_t(1) << lane) - 1));
    for (int w = 0; w < wave; ++w) before += s_cnt[w];
    if (some && before == int(blockIdx.y)) s_pick = tid;
    __syncthreads();
    e = __builtin_amdgcn_readfirstlane(s_pick);
    if (e < 0) return;
  }
  int off = p.sizes ? p.offs[e] : 0;
  int size = p.sizes ? p.sizes[e] : p.rows;
  // clamped into the rows of A and C: other maps give wrong results, not other accesses
  off = off < 0 ? 0 : (off > p.rows ? p.rows : off);
  size = size > p.rows - off ? p.rows - off : size;
  off = __builtin_amdgcn_readfirstlane(off);
  size = __builtin_amdgcn_readfirstlane(size);

  const int K = p.K, KB = K / 32;
  const int steps = (K + S4_STEP - 1) / S4_STEP;
  const uint32_t wrow = uint32_t(K) / 2;
  const int nrows = SWIGLU ? 2 * p.F : p.N;
  const __amdgpu_buffer_rsrc_t rW = s4_rsrc(p.W[e], uint32_t(nrows) * wrow);
  const __amdgpu_buffer_rsrc_t rS = s4_rsrc(p.Ws[e], uint32_t(nrows) * uint32_t(KB));
  // first weight row of block b
  auto brow = [&](int b) {
    if constexpr (SWIGLU) return int(blockIdx.x) * 32 + (b & 1) * 16 + (b >= 2 ? p.F : 0);
    else return int(blockIdx.x) * (NB * 16) + b * 16;
  };
  uint32_t w_off[NB], s_off[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int n = brow(b) + i16;
    const bool in = n < nrows;
    w_off[b] = in ? uint32_t(n) * wrow + 16u * q : kS4Out;
    s_off[b] = in ? uint32_t(n) * uint32_t(KB) + q : kS4Out;
  }

  const uint32_t arow = A4 ? wrow : uint32_t(K);
  for (int m0 = 0; m0 < size; m0 += 16 * MB) {
    const int mv = size - m0 < 16 * MB ? size - m0 : 16 * MB;
    const __amdgpu_buffer_rsrc_t rA = s4_rsrc(p.A + (int64_t(off) + m0) * arow, uint32_t(mv) * arow);
    const __amdgpu_buffer_rsrc_t rAs = s4_rsrc(p.As + (int64_t(off) + m0) * KB, uint32_t(mv) * uint32_t(KB));
    f32x4 acc[NB][MB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int m = 0; m < MB; ++m) acc[b][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s0 = wave * S4_U; s0 < steps; s0 += S4_WAVES * S4_U) {
      u32x4 w[S4_U][NB], a[S4_U][MB], a2[S4_U][MB];
      uint32_t ws[S4_U][NB], as[S4_U][MB];
#pragma unroll
      for (int u = 0; u < S4_U; ++u) {
        const int s = s0 + u;
        const bool kin = s * 4 + q < KB;                 // the lane's K block exists
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          w[u][b] = s4_load16(rW, kin ? w_off[b] + uint32_t(s) * 64u : kS4Out);
          ws[u][b] = s4_load1(rS, kin ? s_off[b] + uint32_t(s) * 4u : kS4Out);
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          const uint32_t row = uint32_t(m * 16 + i16);
          as[u][m] = s4_load1(rAs, kin ? row * uint32_t(KB) + uint32_t(s) * 4u + q : kS4Out);
          if constexpr (A4) {
            a[u][m] = s4_load16(rA, kin ? row * arow + uint32_t(s) * 64u + 16u * q : kS4Out);
          } else {
            const uint32_t k0 = uint32_t(s) * 128u + 16u * q;
            a[u][m] = s4_load16(rA, k0 < uint32_t(K) ? row * arow + k0 : kS4Out);
            a2[u][m] = s4_load16(rA, k0 + 64u < uint32_t(K) ? row * arow + k0 + 64u : kS4Out);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < S4_U; ++u)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            const u32x4 z = {0, 0, 0, 0};
            const i32x8 fw = s4_frag(w[u][b], z);
            const i32x8 fa = A4 ? s4_frag(a[u][m], z) : s4_frag(a[u][m], a2[u][m]);
            acc[b][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fa, acc[b][m], 4, A4 ? 4 : 0, 0,
                                                                         int(ws[u][b]), 0, int(as[u][m]));
          }
    }
    // join the waves' sums in wave order
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int m = 0; m < MB; ++m) red[wave][b * MB + m][lane] = acc[b][m];
    __syncthreads();
    if constexpr (!SWIGLU) {
      for (int j = wave; j < NB * MB; j += S4_WAVES) {
        f32x4 c = red[0][j][lane];
#pragma unroll
        for (int w = 1; w < S4_WAVES; ++w) {
          const f32x4 x = red[w][j][lane];
          c.x += x.x; c.y += x.y; c.z += x.z; c.w += x.w;
        }
        const int row = (j % MB) * 16 + i16;
        const int n = brow(j / MB) + 4 * q;
        if (row < mv && n < p.N) {   // N is a multiple of 4
          const int64_t o = (int64_t(off) + m0 + row) * p.N + n;
          if constexpr (F32) *reinterpret_cast<float4*>(static_cast<float*>(p.C) + o) = make_float4(c.x, c.y, c.z, c.w);
          else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.C) + o) = make_uint2(bf16x2(c.x, c.y), bf16x2(c.z, c.w));
        }
      }
    } else {
      // token block m: wave m % 4.  Blocks 0, 1 hold gate columns 0..15, 16..31, blocks 2, 3
      // the up columns; the lane has columns 4q .. 4q + 3 of each, token i16
      for (int m = wave; m < MB; m += S4_WAVES) {
        f32x4 c[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          c[b] = red[0][b * MB + m][lane];
#pragma unroll
          for (int w = 1; w < S4_WAVES; ++w) {
            const f32x4 x = red[w][b * MB + m][lane];
            c[b].x += x.x; c[b].y += x.y; c[b].z += x.z; c[b].w += x.w;
          }
        }
        const int row = m * 16 + i16;
        const bool live = row < mv;
        const int64_t r = int64_t(off) + m0 + row;
        const float pr = live ? p.prob[r] : 0.f;
        float h[8];
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float G = c[j >> 2][j & 3], U = c[2 + (j >> 2)][j & 3];
          h[j] = pr * silu_f(G) * U;
          amax = fmaxf(amax, fabsf(h[j]));
        }
        amax = fmaxf(amax, __shfl_xor(amax, 16));
        amax = fmaxf(amax, __shfl_xor(amax, 32));
        const uint32_t sc = mx_scale_byte(amax);
        const float inv = mx_inv_scale(sc);
        if (live) {
          uint8_t* hc = p.h_codes + r * p.F + int64_t(blockIdx.x) * 32;
          *reinterpret_cast<uint32_t*>(hc + 4 * q) = e4m3x4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
          *reinterpret_cast<uint32_t*>(hc + 16 + 4 * q) = e4m3x4(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv);
          if (q == 0) p.h_scales[r * (p.F / 32) + blockIdx.x] = uint8_t(sc);
        }
      }
    }
    __syncthreads();
  }
}

// Groups that can have rows: the kernel's grid in y
static int groups_upper(const Gemm4Params& p) { return !p.sizes ? 1 : int(p.E < p.total ? p.E : p.total); }

template <bool A4, int NB, int MB, bool SWIGLU, bool F32>
static mge_status launch_stream(const Gemm4Params& p, int nblocks, const char* name, hipStream_t s) {
  ProfScope prof(s, name);
  hipLaunchKernelGGL((gemm4_stream_kernel<A4, NB, MB, SWIGLU, F32>), dim3(unsigned(nblocks), unsigned(groups_upper(p))),
                     dim3(S4_THREADS), 0, s, p);
  return hip_check(name);
}

mge_status launch_gemm4_store(const Gemm4Params& p, bool a4, bool f32, hipStream_t s) {
  if (p.total <= 0 || p.rows <= 0 || p.N <= 0) return MGE_OK;
  const int nb = (p.N + 31) / 32;
  if (a4)
    return f32 ? launch_stream<true, 2, 1, false, true>(p, nb, "gemm4_stream_mxfp4", s)
               : launch_stream<true, 2, 1, false, false>(p, nb, "gemm4_stream_mxfp4", s);
  return f32 ? launch_stream<false, 2, 1, false, true>(p, nb, "gemm4_stream_mxfp8", s)
             : launch_stream<false, 2, 1, false, false>(p, nb, "gemm4_stream_mxfp8", s);
}

mge_status launch_gemm4_swiglu(const Gemm4Params& p, hipStream_t s) {
  if (p.total <= 0 || p.rows <= 0) return MGE_OK;
  return launch_stream<false, 4, 1, true, false>(p, p.F / 32, "gemm4_swiglu", s);
}

}  // namespace mge
