// bf16 -> E4M3 with one fp32 scale per block of 128 (1 x 128 along the rows, or 128 x 128), in row
// form and transposed, rows optionally gathered, and back.
//
// HBM-bound: one read of the input, one write of each form.  A workgroup takes a tile of 128 rows x
// 128 columns (a block is never split), 8 columns of 4 consecutive rows a thread: a row's 128
// values are in the 16 lanes of a DPP row, a column's 4 rows make one dword of the transposed form,
// which goes through LDS so that it leaves in whole lines.  At most 64 registers, so that a CU holds 32 waves
// (128 registers: 80 us for the first figure).  Measured on MI355X: 8192 x 4096 gathered to 16384 rows, both forms
// 63 us, the bytes at a copy's rate 41; [28672][4096] in 128 x 128 blocks, both forms and each read back, 229 us, the bytes
// at that rate 230.
#include "mge_common.hpp"

#include "fp8b.hpp"

namespace mge {

constexpr int QF_LD = 132;   // bytes of a column in LDS: a dword of skew spreads the dword writes over the banks

constexpr int QF_THREADS = 512;

// larger of each 16-bit half; magnitudes of two bf16 values in that form; the larger half as the bits of an fp32 value
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t pk_abs(uint32_t v) { return v & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t pk_fold(uint32_t v) { return umax(v << 16, v & 0xffff0000u); }

template <bool TILE, bool ROW, bool COL>
__global__ __launch_bounds__(QF_THREADS, 8) void quant_fb_kernel(QuantFbParams p, int64_t tiles, int nr, int nc) {
  __shared__ __attribute__((aligned(16))) uint8_t s_col[COL ? FB * QF_LD : 4];
  __shared__ __attribute__((aligned(16))) uint32_t s_max[TILE ? 8 : (COL ? 8 * FB / 2 : 4)];   // (columns: 16 bits each)
  __shared__ float s_inv[!TILE && COL ? FB : 1];
  const int tid = threadIdx.x, wave = tid >> 6;
  const int cl = (tid & 15) * 8;         // first of the thread's 8 columns
  const int rg = tid >> 4;               // its rows: 4 rg + j
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t b = tile / (int64_t(nr) * nc);
    const int rem = int(tile - b * nr * nc);
    const int tr = rem / nc, tc = rem - tr * nc;
    const int64_t r0 = int64_t(tr) * FB;
    const int c0 = tc * FB + cl;
    const bool cin = c0 < p.C;
    const uint16_t* src = p.in + b * p.in_bstride + c0;
    const int64_t rt = r0 + 4 * rg;
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = make_uint4(0, 0, 0, 0);
      if (cin && rt + j < p.R) {
        int64_t sr = rt + j;
        if (p.map) {
          sr = p.map[sr];
          if (sr < 0 || sr >= p.src_rows) sr = -1;
        }
        if (sr >= 0) x[j] = *reinterpret_cast<const uint4*>(src + sr * p.in_ld);
      }
    }
    // (between the phases the values are unpacked again: kept as floats they would halve the waves)
    auto repack = [&]() {
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(x[j].x), "+v"(x[j].y), "+v"(x[j].z), "+v"(x[j].w));
    };
    auto val = [&](int j, int k) {
      const uint32_t w = k < 4 ? (k < 2 ? x[j].x : x[j].y) : (k < 6 ? x[j].z : x[j].w);
      return __uint_as_float((k & 1) ? w & 0xffff0000u : w << 16);
    };
    // largest magnitudes, as bit patterns, two values at a time
    auto row_max = [&](int j) { return pk_fold(pk_max(pk_max(pk_abs(x[j].x), pk_abs(x[j].y)), pk_max(pk_abs(x[j].z), pk_abs(x[j].w)))); };
    uint32_t all = 0;
    if constexpr (TILE) {
#pragma unroll
      for (int j = 0; j < 4; ++j) all = umax(all, row_max(j));
    }
    FbScale ts;
    if constexpr (TILE) {
      all = row16_umax(all);
      const U32Pair a = permlane16_swap(all, all);
      all = umax(a.a, a.b);
      const U32Pair c = permlane32_swap(all, all);
      all = umax(c.a, c.b);
      if ((tid & 63) == 0) s_max[wave] = all;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) all = umax(all, s_max[w]);
      ts = fb_scale(all);
      if (tid == 0) {
        if constexpr (ROW) p.row_scales[(b * nr + tr) * nc + tc] = ts.s;
        if constexpr (COL) p.col_scales[(b * nc + tc) * nr + tr] = ts.s;
      }
    }
    if constexpr (ROW) {
      uint8_t* rbase = p.row_codes + (b * p.R + r0) * p.C;   // (the same in every lane; 128 rows are below 2^32 bytes)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (!TILE && COL) __builtin_amdgcn_sched_barrier(0);   // a row at a time
        FbScale sc = ts;
        const int64_t r = rt + j;
        if constexpr (!TILE) {
          sc = fb_scale(row16_umax(row_max(j)));
          if (cl == 0 && r < p.R) p.row_scales[(b * p.R + r) * nc + tc] = sc.s;
        }
        if (cin && r < p.R)
          *reinterpret_cast<uint2*>(rbase + (uint32_t(4 * rg + j) * uint32_t(p.C) + uint32_t(c0))) =
              make_uint2(fb_codes4(val(j, 0) * sc.inv, val(j, 1) * sc.inv, val(j, 2) * sc.inv, val(j, 3) * sc.inv),
                         fb_codes4(val(j, 4) * sc.inv, val(j, 5) * sc.inv, val(j, 6) * sc.inv, val(j, 7) * sc.inv));
      }
    }
    if constexpr (COL) {
      if constexpr (!TILE && ROW) repack();
      float inv[8];
      if constexpr (TILE) {
#pragma unroll
        for (int k = 0; k < 8; ++k) inv[k] = ts.inv;
      } else {
        // over the wave's 4 row groups (lanes 16 and 32 apart), then the 8 waves
        uint32_t cm[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          auto at = [&](int j) { return pk_abs(k < 2 ? (k < 1 ? x[j].x : x[j].y) : (k < 3 ? x[j].z : x[j].w)); };
          cm[k] = pk_max(pk_max(at(0), at(1)), pk_max(at(2), at(3)));
          const U32Pair a = permlane16_swap(cm[k], cm[k]);
          cm[k] = pk_max(a.a, a.b);
          const U32Pair c = permlane32_swap(cm[k], cm[k]);
          cm[k] = pk_max(c.a, c.b);
        }
        if ((tid & 48) == 0) *reinterpret_cast<uint4*>(s_max + (wave * FB + cl) / 2) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
        __syncthreads();
        if (tid < FB) {
          const uint16_t* s = reinterpret_cast<const uint16_t*>(s_max) + tid;
          uint32_t m = s[0];
#pragma unroll
          for (int w = 1; w < 8; ++w) m = umax(m, s[w * FB]);
          const FbScale sc = fb_scale(m << 16);
          s_inv[tid] = sc.inv;
          const int c = tc * FB + tid;
          if (c < p.C) p.col_scales[(b * p.C + c) * nr + tr] = sc.s;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) inv[k] = s_inv[cl + k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint32_t*>(s_col + (cl + k) * QF_LD + 4 * rg) =
            fb_codes4(val(0, k) * inv[k], val(1, k) * inv[k], val(2, k) * inv[k], val(3, k) * inv[k]);
      __syncthreads();
      // 16 bytes a thread: 8 threads a column
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = i * 64 + (tid >> 3), q = (tid & 7) * 16;
        if (tc * FB + c < p.C && r0 + q < p.Rp) {
          const uint32_t* s = reinterpret_cast<const uint32_t*>(s_col + c * QF_LD + q);
          *reinterpret_cast<uint4*>(p.col_codes + (b * p.C + tc * FB + c) * p.Rp + r0 + q) = make_uint4(s[0], s[1], s[2], s[3]);
        }
      }
    }
    __syncthreads();   // the LDS is read before the next tile writes it
  }
}

template <bool TILE>
static void launch_q(const QuantFbParams& p, int64_t tiles, int nr, int nc, hipStream_t s) {
  const unsigned grid = unsigned(tiles < (1 << 20) ? tiles : (1 << 20));
  if (p.row_codes && p.col_codes) hipLaunchKernelGGL((quant_fb_kernel<TILE, true, true>), dim3(grid), dim3(QF_THREADS), 0, s, p, tiles, nr, nc);
  else if (p.row_codes) hipLaunchKernelGGL((quant_fb_kernel<TILE, true, false>), dim3(grid), dim3(QF_THREADS), 0, s, p, tiles, nr, nc);
  else hipLaunchKernelGGL((quant_fb_kernel<TILE, false, true>), dim3(grid), dim3(QF_THREADS), 0, s, p, tiles, nr, nc);
}
mge_status launch_quant_fb(const QuantFbParams& p, hipStream_t s) {
  const int nr = int(fb_blocks(p.R)), nc = int(fb_blocks(p.C));
  ProfScope prof(s, "fp8_block_quantize");
  if (p.tile) launch_q<true>(p, int64_t(p.batch) * nr * nc, nr, nc, s);
  else launch_q<false>(p, int64_t(p.batch) * nr * nc, nr, nc, s);
  return hip_check("fp8_block_quantize");
}

// Values of 16 codes a thread.  A thread keeps its columns and goes over rows, so that the division
// of its index happens once.
template <bool F32>
__global__ __launch_bounds__(256) void dequant_fb_kernel(int64_t rows, int R, int C, int tile, int per, int rpb, const uint8_t* codes,
                                                         const float* scales, void* out) {
  const int chunks = C / 16, kb = (C + FB - 1) / FB;
  const int r = int(threadIdx.x) / per;
  const int c = int(blockIdx.x) * per + int(threadIdx.x) - r * per;
  if (r >= rpb || c >= chunks) return;
  const int nr = (R + FB - 1) / FB;
  for (int64_t row = int64_t(blockIdx.y) * rpb + r; row < rows; row += int64_t(gridDim.y) * rpb) {
    const uint4 q = *reinterpret_cast<const uint4*>(codes + row * C + c * 16);
    int64_t srow = row;
    if (tile) {
      const int64_t b = row / R;
      srow = b * nr + (row - b * R) / FB;
    }
    const float s = scales[srow * kb + c / 8];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    float v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[i]), false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w[i]), true);
      v[4 * i] = lo[0] * s; v[4 * i + 1] = lo[1] * s; v[4 * i + 2] = hi[0] * s; v[4 * i + 3] = hi[1] * s;
    }
    if constexpr (F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + row * C + c * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * C + c * 16);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        o[i] = make_uint4(bf16x2(v[8 * i], v[8 * i + 1]), bf16x2(v[8 * i + 2], v[8 * i + 3]), bf16x2(v[8 * i + 4], v[8 * i + 5]),
                          bf16x2(v[8 * i + 6], v[8 * i + 7]));
    }
  }
}

mge_status launch_dequant_fb(int64_t batch, int64_t R, int C, bool tile, const uint8_t* codes, const float* scales, int dtype,
                             void* out, hipStream_t s) {
  const int chunks = C / 16;
  const int per = chunks < 256 ? chunks : 256, rpb = 256 / per;
  const int64_t rows = batch * R;
  const unsigned gx = unsigned((chunks + per - 1) / per);
  int64_t gy = (rows + rpb - 1) / rpb;
  const int64_t most = 16384 / gx + 1;
  if (gy > most) gy = most;
  ProfScope prof(s, "fp8_block_dequantize");
  if (dtype == MGE_DTYPE_F32)
    hipLaunchKernelGGL((dequant_fb_kernel<true>), dim3(gx, unsigned(gy)), dim3(256), 0, s, rows, int(R), C, tile ? 1 : 0, per, rpb,
                       codes, scales, out);
  else
    hipLaunchKernelGGL((dequant_fb_kernel<false>), dim3(gx, unsigned(gy)), dim3(256), 0, s, rows, int(R), C, tile ? 1 : 0, per, rpb,
                       codes, scales, out);
  return hip_check("fp8_block_dequantize");
}

}  // namespace mge
