// Grouped products with MXFP4 weights for few rows per expert (token-by-token serving):
// C[r][n] = sum over k of A[r][k] W_e[n][k] for the rows r of expert e, A in MXFP8 or
// MXFP4, W in MXFP4, fp32 accumulation on the block-scaled matrix units.
//
// With few rows the product is one read of the weights, so the kernel is built around that
// stream.  A workgroup owns NB blocks of 16 weight rows of one expert; its W waves split K
// (a wave takes S4_CHUNK blocks of 32, then the next wave's follow), read their share of
// those rows once, straight into registers, and add their partial sums through LDS at the
// end, in wave order.  The weights are the matrix unit's row operand and 16 or 32 tokens (MB
// = 1, 2) its columns (v_mfma_scale_f32_16x16x128_f8f6f4); more rows than that in a group take
// further passes over the same weights.  Those come from L2 only where the rows that the
// workgroups of an XCD go over fit it: a further pass over 8 experts x [4096][14336] takes as long
// as the first (32 rows an expert 72 us, 64 129, 96 184).  A chunk's 16 blocks are
// dealt to the 4 matrix instructions so that the loads of two of them read whole lines and
// the row's 16 scale bytes are one load (VEC: rows of scales aligned to it).
//   HBM-bound: 8 experts x [28672][4096], 32 rows 97 us (5.3 TB/s of codes and scales); the
// gate-up and down products of 8 tokens, top-2 of 8 experts (4096 x 14336) 84 and 50 us, of 64 (MB
// = 2) 127 and 64.  One row x [2048][4096] takes 5.3 us, where an empty launch takes 4.
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

constexpr int S4_CHUNK = 16;     // K blocks (of 32) a wave takes at a time: 4 matrix instructions a row block
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

template <int W, bool A4, int NB, int MB, bool SWIGLU, bool F32, bool VEC>
__global__ __launch_bounds__(64 * W) void gemm4_stream_kernel(Gemm4Params p) {
  __shared__ __attribute__((aligned(16))) f32x4 red[W][NB * MB][64];
  __shared__ int32_t s_pick, s_cnt[4];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int i16 = lane & 15;
  const int q = lane >> 4;

  // the group of this workgroup: the blockIdx.y-th expert that has rows (there are at most
  // min(E, rows) of them, which is the grid)
  int e = 0;
  if (p.sizes) {
    static_assert(W >= 4, "a thread for each of up to 256 experts");
    if (tid == 0) s_pick = -1;
    const bool some = tid < p.E && p.sizes[tid] > 0;
    const uint64_t mask = __ballot(some);
    if (lane == 0 && wave < 4) s_cnt[wave] = __popcll(mask);
    __syncthreads();
    int before = __popcll(mask & ((uint64_t(1) << lane) - 1));
    for (int w = 0; w < wave && w < 4; ++w) before += s_cnt[w];
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
  const int chunks = (KB + S4_CHUNK - 1) / S4_CHUNK;
  const uint32_t wrow = uint32_t(K) / 2;
  const int nrows = SWIGLU ? 2 * p.F : p.N;
  const __amdgpu_buffer_rsrc_t rW = s4_rsrc(p.W ? p.W[e] : p.Wv[e], uint32_t(nrows) * wrow);
  const __amdgpu_buffer_rsrc_t rS = s4_rsrc(p.W ? p.Ws[e] : p.Wsv[e], uint32_t(nrows) * uint32_t(KB));
  // first weight row of block b
  auto brow = [&](int b) {
    if constexpr (SWIGLU) return int(blockIdx.x) * (NB * 8) + (b % (NB / 2)) * 16 + (b >= NB / 2 ? p.F : 0);
    else return int(blockIdx.x) * (NB * 16) + b * 16;
  };
  uint32_t w_off[NB], s_off[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int n = brow(b) + i16;
    // (SwiGLU: ffn columns past F are neither gate nor up rows of this workgroup)
    const bool in = SWIGLU ? n - (b >= NB / 2 ? p.F : 0) < p.F : n < nrows;
    w_off[b] = in ? uint32_t(n) * wrow : kS4Out;
    s_off[b] = in ? uint32_t(n) * uint32_t(KB) : kS4Out;
  }
  // K blocks of a chunk: step 2t + j takes block 8t + 2q + j in the lanes q (so that two steps
  // read whole lines of 128 bytes); an 8-bit operand's lane q has halves q % 2 of the blocks
  // that its lanes q / 2 and 2 + q / 2 scale
  const uint32_t sh0 = 16 * (q & 1);
  const bool odd2 = (q >> 1) != 0;
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
    for (int c = wave; c < chunks; c += W) {
      const uint32_t k0 = uint32_t(c) * S4_CHUNK;
      u32x4 w[4][NB], a[4][MB], a2[4][MB];
      u32x4 ws[NB], as[MB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t blk = k0 + 8 * (u >> 1) + 2 * q + (u & 1);
          w[u][b] = s4_load16(rW, VEC || blk < uint32_t(KB) ? w_off[b] + blk * 16 : kS4Out);
        }
        if constexpr (VEC) {
          ws[b] = s4_load16(rS, s_off[b] + k0);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t blk = k0 + 8 * (u >> 1) + 2 * q + (u & 1);
            ws[b][u] = s4_load1(rS, blk < uint32_t(KB) ? s_off[b] + blk : kS4Out);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const uint32_t row = uint32_t(m * 16 + i16);
        if constexpr (VEC) as[m] = s4_load16(rAs, row * uint32_t(KB) + k0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t blk = k0 + 8 * (u >> 1) + 2 * q + (u & 1);
          if constexpr (!VEC) as[m][u] = s4_load1(rAs, blk < uint32_t(KB) ? row * uint32_t(KB) + blk : kS4Out);
          if constexpr (A4) {
            a[u][m] = s4_load16(rA, VEC || blk < uint32_t(KB) ? row * arow + blk * 16 : kS4Out);
          } else {
            const uint32_t b1 = k0 + 8 * (u >> 1) + 2 * (q >> 1) + (u & 1);
            a[u][m] = s4_load16(rA, VEC || b1 < uint32_t(KB) ? row * arow + b1 * 32 + 16 * (q & 1) : kS4Out);
            a2[u][m] = s4_load16(rA, VEC || b1 + 4 < uint32_t(KB) ? row * arow + (b1 + 4) * 32 + 16 * (q & 1) : kS4Out);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // the scale byte of block 8 (u / 2) + 2 q + u % 2
        auto sc = [&](const u32x4& v) {
          if constexpr (VEC) return int((odd2 ? v[2 * (u >> 1) + 1] : v[2 * (u >> 1)]) >> (sh0 + 8 * (u & 1)));
          else return int(v[u]);
        };
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            const u32x4 z = {0, 0, 0, 0};
            const i32x8 fw = s4_frag(w[u][b], z);
            const i32x8 fa = A4 ? s4_frag(a[u][m], z) : s4_frag(a[u][m], a2[u][m]);
            acc[b][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw, fa, acc[b][m], 4, A4 ? 4 : 0, 0, sc(ws[b]), 0,
                                                                         sc(as[m]));
          }
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
      for (int j = wave; j < NB * MB; j += W) {
        f32x4 c = red[0][j][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) {
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
      // item j: 32 ffn columns (set j / MB) of token block j % MB.  Their gate columns 0..15
      // and 16..31 are blocks 2 set, 2 set + 1, their up columns NB / 2 blocks further; the
      // lane has columns 4q .. 4q + 3 of each, token i16
      for (int j = wave; j < (NB / 4) * MB; j += W) {
        const int m = j % MB, set = j / MB;
        const int f0 = int(blockIdx.x) * (NB * 8) + set * 32;
        if (f0 >= p.F) continue;   // uniform
        f32x4 c[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int at = (2 * set + (b & 1) + (b >= 2 ? NB / 2 : 0)) * MB + m;
          c[b] = red[0][at][lane];
#pragma unroll
          for (int w = 1; w < W; ++w) {
            const f32x4 x = red[w][at][lane];
            c[b].x += x.x; c[b].y += x.y; c[b].z += x.z; c[b].w += x.w;
          }
        }
        const int row = m * 16 + i16;
        const bool live = row < mv;
        const int64_t r = int64_t(off) + m0 + row;
        const float pr = live ? p.prob[r] : 0.f;
        float h[8];
        uint32_t amax = 0;   // as bits: a NaN or infinity stays on top and makes the block a NaN block
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float G = c[i >> 2][i & 3], U = c[2 + (i >> 2)][i & 3];
          h[i] = pr * silu_f(G) * U;
          amax = umax(amax, __float_as_uint(h[i]) & 0x7fffffffu);
        }
        amax = umax(amax, uint32_t(__shfl_xor(int(amax), 16)));
        amax = umax(amax, uint32_t(__shfl_xor(int(amax), 32)));
        const uint32_t sc = mx_scale_byte_nan(amax);
        const float inv = mx_inv_scale(sc);
        if (live) {
          uint8_t* hc = p.h_codes + r * p.F + f0;
          *reinterpret_cast<uint32_t*>(hc + 4 * q) = e4m3x4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
          *reinterpret_cast<uint32_t*>(hc + 16 + 4 * q) = e4m3x4(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv);
          if (q == 0) p.h_scales[r * (p.F / 32) + f0 / 32] = uint8_t(sc);
        }
      }
    }
    __syncthreads();
  }
}

// Groups that can have rows: the kernel's grid in y
static int groups_upper(const Gemm4Params& p) { return !p.sizes ? 1 : int(p.E < p.total ? p.E : p.total); }

template <int W, bool A4, int NB, int MB, bool SWIGLU, bool F32>
static mge_status launch_stream(const Gemm4Params& p, const char* name, hipStream_t s) {
  const int cols = SWIGLU ? p.F : p.N, per = SWIGLU ? NB * 8 : NB * 16;
  const dim3 grid(unsigned((cols + per - 1) / per), unsigned(groups_upper(p)));
  ProfScope prof(s, name);
  if (p.vec) hipLaunchKernelGGL((gemm4_stream_kernel<W, A4, NB, MB, SWIGLU, F32, true>), grid, dim3(64 * W), 0, s, p);
  else hipLaunchKernelGGL((gemm4_stream_kernel<W, A4, NB, MB, SWIGLU, F32, false>), grid, dim3(64 * W), 0, s, p);
  return hip_check(name);
}

// Workgroups from which a wider workgroup (fewer reads of the tokens) beats a narrower one
// (more CUs at work), and 8 waves for each below a CU's fill of 4-wave ones.  Down product of 2
// experts x [4096][14336], 1 row each (512 blocks of 16 rows): 16 rows a workgroup 14.5 us, 32
// 16.5, 64 23; of 7 experts, 8 waves x 64 rows 44 us, 4 waves x 64 rows 47, 8 waves x 32 rows 60.
// Two token blocks a pass (MB = 2) past 12 rows an expert on average: gate-up and down of 64
// tokens, top-2 of 8 experts, 249 -> 219 us; of 32 tokens it costs 201 for 165.
constexpr int64_t kStreamWgs = 512;
constexpr int kStreamRows2 = 12;

template <bool A4, bool F32>
static mge_status launch_store(const Gemm4Params& p, const char* name, hipStream_t s) {
  const int64_t blocks = int64_t((p.N + 15) / 16) * groups_upper(p);
  if (p.total > int64_t(kStreamRows2) * p.E) {
    if (blocks < 4 * kStreamWgs) return launch_stream<8, A4, 2, 2, false, F32>(p, name, s);
    return launch_stream<4, A4, 4, 2, false, F32>(p, name, s);
  }
  if (blocks < 2 * kStreamWgs) return launch_stream<8, A4, 1, 1, false, F32>(p, name, s);
  if (blocks < 4 * kStreamWgs) return launch_stream<8, A4, 2, 1, false, F32>(p, name, s);
  if (blocks < 8 * kStreamWgs) return launch_stream<8, A4, 4, 1, false, F32>(p, name, s);
  return launch_stream<4, A4, 4, 1, false, F32>(p, name, s);
}

mge_status launch_gemm4_store(const Gemm4Params& p, bool a4, bool f32, hipStream_t s) {
  if (p.total <= 0 || p.rows <= 0 || p.N <= 0) return MGE_OK;
  if (a4) return f32 ? launch_store<true, true>(p, "gemm4_stream_mxfp4", s) : launch_store<true, false>(p, "gemm4_stream_mxfp4", s);
  return f32 ? launch_store<false, true>(p, "gemm4_stream_mxfp8", s) : launch_store<false, false>(p, "gemm4_stream_mxfp8", s);
}

mge_status launch_gemm4_swiglu(const Gemm4Params& p, hipStream_t s) {
  if (p.total <= 0 || p.rows <= 0) return MGE_OK;
  if (p.total > int64_t(kStreamRows2) * p.E) return launch_stream<4, false, 4, 2, true, false>(p, "gemm4_swiglu", s);
  return launch_stream<4, false, 4, 1, true, false>(p, "gemm4_swiglu", s);
}

}  // namespace mge
