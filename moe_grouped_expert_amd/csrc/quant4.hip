// MXFP4 block quantization (E2M1 + E8M0 per 32) of bf16 matrices in row and column
// orientation, and its inverse.
//
// OCP Microscaling Formats v1.0: E2M1 magnitudes are 0, .5, 1, 1.5, 2, 3, 4, 6; the shared
// exponent of a block is floor(log2(amax)) - 2 (2 = the largest E2M1 exponent), clamped to
// the E8M0 range; an element is v / 2^e rounded to the nearest E2M1 value (ties to even),
// saturating at 6.  Two codes share a byte, the even element in the low half.
//
// E2M1 has no code for infinity or NaN: a block that holds one gets the scale byte 255, the
// format's NaN, so that it shows in what is computed from it.
//
// The amax of bf16 values is taken on their bits (magnitudes order as integers), so the
// scale needs no arithmetic, and v_cvt_scalef32_pk_fp4_bf16 divides by the scale, rounds to
// nearest even and saturates (equal to the definition over all finite bf16 values at every
// scale, on MI355X).
//
// One workgroup (512 threads) owns a tile of 128 rows x 256 columns, staged in LDS; a thread
// quantizes two blocks of 32 values of a row, then two of a column.  A tile row's codes are
// then a whole line of 128 bytes (128 columns: 10% slower); a tile of 256 x 256, whose column
// pieces are whole lines too, leaves one workgroup a CU and is 13% slower, and scale bytes
// gathered into dwords change nothing.  HBM-bound: 2 B read and 17/32 B written per element and
// orientation.  [28672][4096]: rows 60 us (4.9 TB/s), columns 65, both 86 (4.2 TB/s).
#include "mge_common.hpp"
#include "mge_internal.hpp"

namespace mge {

constexpr int Q4_ROWS = 128;
constexpr int Q4_COLS = 256;
constexpr int Q4_THREADS = 512;
constexpr int Q4_STRIDE = Q4_COLS + 8;   // bf16 elements per LDS row
constexpr int Q4_GRP = 16;               // extra bf16 per 32 rows: the row groups of a column fall on other banks
__device__ __forceinline__ int q4_at(int row, int col) { return row * Q4_STRIDE + (row >> 5) * Q4_GRP + col; }

typedef __bf16 bf16v2 __attribute__((ext_vector_type(2)));

// fp32 value 2^(s - 127) of an E8M0 byte s < 255
__device__ __forceinline__ float e8m0_value(uint32_t s) { return __uint_as_float(s == 0 ? 0x00400000u : s << 23); }

// 32 bf16 values as 16 packed pairs (low half first) -> 16 code bytes (4 dwords) and the
// block's E8M0 byte
__device__ __forceinline__ uint32_t quant32_fp4(const uint32_t* w, uint32_t* out) {
  uint32_t hi = 0, lo = 0;   // largest magnitudes of the odd and of the even elements
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    hi = umax(hi, w[i] & 0x7fff0000u);
    lo = umax(lo, w[i] & 0x00007fffu);
  }
  const int field = int(umax(hi >> 16, lo) >> 7);   // exponent field of the amax (255: an infinity or NaN in the block)
  const uint32_t s = uint32_t(field < 2 ? 0 : field - 2);
  const float scale = e8m0_value(s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = 0;
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(v, __builtin_bit_cast(bf16v2, w[4 * i]), scale, 0);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(v, __builtin_bit_cast(bf16v2, w[4 * i + 1]), scale, 1);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(v, __builtin_bit_cast(bf16v2, w[4 * i + 2]), scale, 2);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(v, __builtin_bit_cast(bf16v2, w[4 * i + 3]), scale, 3);
    out[i] = v;
  }
  return field == 255 ? 255u : s;
}

__global__ __launch_bounds__(Q4_THREADS) void quant4_kernel(Quant4Params p) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[Q4_ROWS * Q4_STRIDE + (Q4_ROWS / 32) * Q4_GRP];
  const int tid = threadIdx.x;
  const int c0 = blockIdx.x * Q4_COLS;
  const int64_t r0 = int64_t(blockIdx.y) * Q4_ROWS;
  const int b = blockIdx.z;
  const uint16_t* in = p.in + int64_t(b) * p.in_batch_stride;
  // whole lines into LDS: Q4_COLS / 8 lanes per tile row, all of a thread's loads in flight
  // together; outside: zeros
  constexpr int LANES = Q4_COLS / 8, ROUND = Q4_THREADS / LANES, NL = Q4_ROWS / ROUND;
  const int lr = tid / LANES, ch = (tid % LANES) * 8;
  uint4 val[NL];
  bool ok[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int64_t rg = r0 + ROUND * i + lr;
    ok[i] = rg < p.R && c0 + ch < p.C;
    val[i] = *reinterpret_cast<const uint4*>(in + (ok[i] ? rg * p.in_row_stride + c0 + ch : 0));
  }
#pragma unroll
  for (int i = 0; i < NL; ++i)
    *reinterpret_cast<uint4*>(tile + q4_at(ROUND * i + lr, ch)) = ok[i] ? val[i] : make_uint4(0, 0, 0, 0);
  lds_barrier();
  if (p.row_codes) {   // uniform
    constexpr int PER = Q4_COLS / 32;   // blocks of a tile row
#pragma unroll
    for (int i = tid; i < Q4_ROWS * PER; i += Q4_THREADS) {
      const int rl = i / PER, cl = (i % PER) * 32;
      const int64_t r = r0 + rl;
      if (r < p.R && c0 + cl < p.C) {
        uint32_t w[16], out[4];
        const uint4* t4 = reinterpret_cast<const uint4*>(tile + q4_at(rl, cl));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 q = t4[j];
          w[4 * j] = q.x; w[4 * j + 1] = q.y; w[4 * j + 2] = q.z; w[4 * j + 3] = q.w;
        }
        const uint32_t s = quant32_fp4(w, out);
        const int64_t blk = ((int64_t(b) * p.R + r) * p.C + c0 + cl) / 32;
        reinterpret_cast<uint4*>(p.row_codes)[blk] = make_uint4(out[0], out[1], out[2], out[3]);
        p.row_scales[blk] = uint8_t(s);
      }
    }
  }
  if (p.col_codes) {
    constexpr int PER = Q4_ROWS / 32;   // blocks of a tile column
#pragma unroll
    for (int i = tid; i < Q4_COLS * PER; i += Q4_THREADS) {
      const int cc = i / PER, rb = (i % PER) * 32;
      const int col = c0 + cc;
      const int64_t row = r0 + rb;
      if (col < p.C && row < p.Rp) {
        uint32_t w[16], out[4];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          w[j] = uint32_t(tile[q4_at(rb + 2 * j, cc)]) | (uint32_t(tile[q4_at(rb + 2 * j + 1, cc)]) << 16);
        const uint32_t s = quant32_fp4(w, out);
        const int64_t blk = ((int64_t(b) * p.C + col) * p.Rp + row) / 32;
        reinterpret_cast<uint4*>(p.col_codes)[blk] = make_uint4(out[0], out[1], out[2], out[3]);
        p.col_scales[blk] = uint8_t(s);
      }
    }
  }
}

mge_status launch_quant4(const Quant4Params& p, hipStream_t s) {
  if (p.R <= 0 || p.C <= 0 || p.batch <= 0) return MGE_OK;
  const dim3 grid(unsigned((p.C + Q4_COLS - 1) / Q4_COLS), unsigned((p.Rp + Q4_ROWS - 1) / Q4_ROWS), unsigned(p.batch));
  ProfScope prof(s, "quant_fp4");
  hipLaunchKernelGGL(quant4_kernel, grid, dim3(Q4_THREADS), 0, s, p);
  return hip_check("quant4_kernel");
}

// Dequantize: a lane takes 4 code bytes (8 values), so that a wave's stores are whole lines
// (a lane with a whole block of 32 is 1.8 times slower).  HBM-bound: 17/32 B read, 2 or 4
// written per value; [28672][4096] to bf16 55 us (5.4 TB/s, the codes partly from cache).
// A scale byte of 255 is the format's NaN and gives NaN.
constexpr int DQ_THREADS = 256;
constexpr int DQ_PER = 4;   // dwords of codes a thread takes, DQ_THREADS apart

template <bool F32>
__global__ __launch_bounds__(DQ_THREADS) void dequant4_kernel(int64_t dwords, const uint32_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, void* __restrict__ out) {
  const int64_t base = int64_t(blockIdx.x) * (DQ_THREADS * DQ_PER) + threadIdx.x;
  uint32_t c[DQ_PER], s[DQ_PER];
#pragma unroll
  for (int j = 0; j < DQ_PER; ++j) {
    const int64_t i = base + j * DQ_THREADS;
    if (i < dwords) {
      c[j] = codes[i];
      s[j] = scales[i >> 2];
    }
  }
#pragma unroll
  for (int j = 0; j < DQ_PER; ++j) {
    const int64_t i = base + j * DQ_THREADS;
    if (i >= dwords) return;
    const float scale = s[j] == 255 ? __uint_as_float(0x7fc00000u) : e8m0_value(s[j]);
    float v[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const uint32_t x = (c[j] >> (4 * n)) & 15u;
      const uint32_t m = x & 7u;
      // magnitude: 0, .5, then (1 + low bit / 2) 2^(m/2 - 1)
      const float mag = m < 2 ? 0.5f * float(m) : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
      v[n] = ((x & 8u) ? -mag : mag) * scale;
    }
    if constexpr (F32) {
      float4* o = static_cast<float4*>(out) + i * 2;
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      static_cast<uint4*>(out)[i] = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    }
  }
}

mge_status launch_dequant4(int64_t blocks, const uint8_t* codes, const uint8_t* scales, int dtype, void* out, hipStream_t s) {
  if (blocks <= 0) return MGE_OK;
  const int64_t dwords = blocks * 4;
  const dim3 grid(unsigned((dwords + DQ_THREADS * DQ_PER - 1) / (DQ_THREADS * DQ_PER)));
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  ProfScope prof(s, "dequant_fp4");
  if (dtype == MGE_DTYPE_F32) hipLaunchKernelGGL(dequant4_kernel<true>, grid, dim3(DQ_THREADS), 0, s, dwords, c, scales, out);
  else hipLaunchKernelGGL(dequant4_kernel<false>, grid, dim3(DQ_THREADS), 0, s, dwords, c, scales, out);
  return hip_check("dequant4_kernel");
}

}  // namespace mge
