// Parameter blocks and launchers of the norm and of FP8 with one fp32 scale per block of 128.
//
// Format: E4M3 codes; a block of values (1 x 128 along the reduction, or 128 x 128 of a weight)
// has the scale s = max(amax, 2^-100) / 448 in fp32 and the codes of v * (448 / max(amax, 2^-100)),
// both quotients correctly rounded, the product rounded to the nearest E4M3 value (ties to even).
// The floor keeps both factors normal fp32 numbers (an all-zero block has codes 0).  A block with
// an infinity or NaN has the scale NaN (its codes have no meaning), so that what is computed from
// it is NaN.
#pragma once

#include "mge_internal.hpp"

namespace mge {

constexpr int FB = 128;   // values of a block along an axis
inline int64_t fb_blocks(int64_t n) { return (n + FB - 1) / FB; }

// What a wave of the tile kernels reads of a matrix's scales, 64 rows from `row` on and block `blk` first: where that
// begins (elements) and the bytes that its buffer resource covers.  by_row: [rows][nb], else block-major [nb][rows].
// A slice's place goes into the scalar offset, which a resource does not bound in every form of its range check, so the
// resource of a wave that starts past the last row is empty: past the last block's row `rows` it would read behind the
// table.  What starts before it ends at most 63 elements behind (fb_scales_bytes has them).
struct FbSpan {
  int64_t at;
  uint32_t bytes;
};
constexpr FbSpan fb_scale_span(int64_t row, int64_t rows, int64_t blk, int64_t nb, bool by_row) {
  const int64_t at = by_row ? row * nb + blk : blk * rows + row;
  return FbSpan{at, row < rows && blk < nb ? uint32_t(rows * nb - at) * 4 : 0};
}
// Workspace of block-major scales [ceil(K/128)][rows], and what the last wave of a row reads behind them
inline size_t fb_scales_bytes(int64_t rows, int64_t K) {
  const size_t n = size_t(rows) * size_t(fb_blocks(K)) * 4;
  return n ? up256(n) + 256 : 0;
}

#ifdef __HIPCC__
// Scale and factor of a block from the largest of its values' bit patterns without signs
struct FbScale {
  float s, inv;
};
__device__ __forceinline__ FbScale fb_scale(uint32_t bits) {
  const float m = fmaxf(__uint_as_float(bits), 0x1p-100f);
  const bool fin = bits < 0x7f800000u;
  return FbScale{fin ? m / 448.f : __uint_as_float(0x7fc00000u), fin ? 448.f / m : 0.f};
}
// Codes of four values of a block times its factor.  Such a product is at most 448 (1 + 2^-23), which rounds to E4M3's
// largest value: no clamp.  (In a block with an infinity or NaN they have no meaning.)
__device__ __forceinline__ uint32_t fb_codes4(float a, float b, float c, float d) {
  const int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, __float_as_int(a), false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}
// max of the bit patterns over the 16 lanes of a DPP row (every lane gets it)
__device__ __forceinline__ uint32_t row16_umax(uint32_t v) {
  v = umax(v, dpp_u<0xB1>(v));    // lane ^ 1
  v = umax(v, dpp_u<0x4E>(v));    // lane ^ 2
  v = umax(v, dpp_u<0x141>(v));   // mirror in 8
  return umax(v, dpp_u<0x140>(v));   // mirror in 16
}
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp_f<0xB1>(v);
  v += dpp_f<0x4E>(v);
  v += dpp_f<0x141>(v);
  return v + dpp_f<0x140>(v);
}
// sum over the wave (every lane gets it; a fixed order)
__device__ __forceinline__ float wave_sum64(float v) {
  v = row16_sum(v);
  const U32Pair a = permlane16_swap(__float_as_uint(v), __float_as_uint(v));
  v = __uint_as_float(a.a) + __uint_as_float(a.b);
  const U32Pair b = permlane32_swap(__float_as_uint(v), __float_as_uint(v));
  return __uint_as_float(b.a) + __uint_as_float(b.b);
}
#endif

// ------------------------------------------------------------ norm
struct NormParams {
  int64_t T;
  int H;
  int64_t x_ld;             // row stride of x (elements); every other matrix is contiguous
  float eps;
  int w_f32, y_f32;
  const void* x;
  const void* residual;     // optional
  const void* weight;
  void* res_out;            // with residual
  void* y;                  // optional
  float* rstd;              // optional [T]
  uint8_t* codes;           // optional [T][H]
  float* scales;            // [T][ceil(H/128)]
};
mge_status launch_rmsnorm(const NormParams& p, bool x_f32, hipStream_t s);
struct NormBwdParams {
  int64_t T;
  int H;
  int64_t x_ld, dy_ld;
  int w_f32, dy_f32;
  const void* dy;
  const void* x;
  const void* weight;
  const float* rstd;
  const void* d_res;        // optional
  void* dx;
  float* dw;                // optional [H]
  float* part;              // workspace [rmsnorm_bwd_parts(T, H)][H]
};
int rmsnorm_bwd_parts(int64_t T, int H);
constexpr int kNormMaxH = 16384;
mge_status launch_rmsnorm_bwd(const NormBwdParams& p, bool x_f32, hipStream_t s);
mge_status launch_rmsnorm_dw_zero(int H, float* dw, hipStream_t s);   // no rows: zeros

// ------------------------------------------------------------ quantizer
struct QuantFbParams {
  const uint16_t* in;
  int64_t in_bstride, in_ld;    // elements
  const int32_t* map;           // optional: source row of each row (outside [0, src_rows): zeros)
  int64_t src_rows;
  int batch;
  int64_t R, Rp;                // rows, rows padded to 32 (transposed form)
  int C;
  bool tile;                    // 128 x 128 blocks
  uint8_t* row_codes;  float* row_scales;
  uint8_t* col_codes;  float* col_scales;
};
mge_status launch_quant_fb(const QuantFbParams& p, hipStream_t s);
// tile: scales [batch][ceil(R/128)][ceil(C/128)], else [batch][R][ceil(C/128)]
mge_status launch_dequant_fb(int64_t batch, int64_t R, int C, bool tile, const uint8_t* codes, const float* scales, int dtype,
                             void* out, hipStream_t s);

// ------------------------------------------------------------ products
constexpr int kFbInline = kInlineExperts;   // experts whose pointers may travel in the arguments
struct FbGemm {
  int E, N, K, F;                   // F: SwiGLU (N = 2F)
  int rows;                         // rows of the groups: every group is clamped into them
  int total;                        // at most this many rows in all groups
  const int32_t* sizes;             // [E], or NULL: one group of all rows
  const int32_t* offs;
  const int32_t* map;               // optional: row of A of each row (outside [0, src_rows): zeros)
  int src_rows;
  const uint8_t* A;                 // [src_rows][K]
  const float* As;                  // [src_rows][ceil(K/128)]
  const float* Ast;                 // tiles: [ceil(K/128)][ast_ld], by row of the groups (NULL: As, where fb_tail_only)
  int64_t ast_ld;
  const uint8_t* const* W;          // device tables (NULL: Wv, Wsv): [N][K] codes of each expert
  const float* const* Ws;           // [ceil(N/128)][ceil(K/128)]
  const uint8_t* Wv[kFbInline];
  const float* Wsv[kFbInline];
  void* C;                          // [rows][N]
  int out_f32;
  const float* prob;                // SwiGLU: [rows] or NULL (1)
  uint8_t* h_codes;                 // SwiGLU: [rows][F]
  float* h_scales;                  // SwiGLU: [ceil(F/128)][ast_ld]
  int grid_main;                    // workgroups of the main launch's whole rounds (set by the launcher)
};
mge_status launch_fb_stream(const FbGemm& p, hipStream_t s);
bool fb_tail_only(int64_t E, int64_t N, int64_t total);
mge_status launch_fb_tile(const FbGemm& p, bool swiglu, hipStream_t s);

// h_codes, h_scales of fp32 rows gu = [G U] (rows behind and between the groups may be left out); scales
// [rows][ceil(F/128)], or with ld > 0 [ceil(F/128)][ld]
mge_status launch_fb_swiglu(const FbGemm& p, const float* gu, int64_t ld, hipStream_t s);

// dw_e[n][k] = sum over the tokens of expert e: columns [offs[e], offs[e] + sizes[e]) of both
struct FbWgrad {
  int E, N, K;
  int rows;                         // token columns (codes' row length)
  const int32_t* sizes;
  const int32_t* offs;
  const uint8_t* Y;                 // [N][rows]
  const uint8_t* X;                 // [K][rows]
  const float* Ys;                  // [N][ceil(rows/128)]
  const float* Xs;                  // [K][ceil(rows/128)]
  const float* Yst;                 // [ceil(rows/128)][N], unless fb_wgrad_small
  const float* Xst;                 // [ceil(rows/128)][K]
  void* const* D;                   // device table (NULL: Dv): [N][K] of each expert
  void* Dv[kFbInline];
  int out;                          // OutForm
};
bool fb_wgrad_small(const FbWgrad& p);
mge_status launch_fb_wgrad(const FbWgrad& p, hipStream_t s);

// out[j][r] = in[row(r)][j]: fp32 scales, block-major; row(r) = map ? map[r] : r, 0 where outside [0, src_rows)
struct FbScaleT {
  const float* in;
  const int32_t* map;
  int64_t src_rows;
  int64_t rows;
  int kb;
  float* out;                       // [kb][ld]
  int64_t ld;
};
mge_status launch_fb_scale_t(const FbScaleT* list, int n, hipStream_t s);

}  // namespace mge
