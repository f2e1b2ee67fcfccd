// The grouped-GEMM kernels with MXFP4 weights (block-scaled 4-bit MFMA), for groups of many
// rows: the tile kernel of gemm_impl.hpp in its 4-bit formats.  mxfp8_mxfp4: rows in MXFP8
// (the expert MLP's activations), mxfp4: rows in MXFP4 too, at twice the matrix rate.
// Measured, 8192 x 8192 x 8192: 2.84 PFLOP/s with MXFP8 rows, 4.15 with MXFP4 rows; expert MLP of
// 8192 tokens, top-2 of 8 experts (4096 x 14336): gate-up with SwiGLU 1.56-1.62 ms (2.4 PFLOP/s,
// matrix units 58% busy), down 0.65 + 0.07 ms (69% busy).  Like the MXFP8 products they run at
// 1.9-2.1 GHz, and a CU takes in operands at 33 bytes a ns whatever their format: a third LDS
// stage (they fit, at 48 KB) and an earlier or later refill change nothing, 3% slower to none.
#include "gemm_impl.hpp"

namespace mge {

#define MGE_GEMM_KERNEL(name, FMT, EPI, OUT) \
  __global__ __launch_bounds__(G_THREADS, 1) void name(GemmParams p) { gemm_body<FMT, EPI, RAGGED_M, OUT>(p); }
#define MGE_GEMM_TAIL_KERNEL(name, FMT, OUT) \
  __global__ __launch_bounds__(G_THREADS, 2) void name(GemmParams p) { gemm_body<FMT, EPI_STORE, RAGGED_M, OUT, 2>(p); }

MGE_GEMM_KERNEL(gemm_gateup_swiglu_mxfp8_mxfp4, FMT_MXFP8_MXFP4, EPI_SWIGLU, OUT_NONE)
MGE_GEMM_KERNEL(gemm_store_mxfp8_mxfp4, FMT_MXFP8_MXFP4, EPI_STORE, OUT_BF16)
MGE_GEMM_KERNEL(gemm_store_f32_mxfp8_mxfp4, FMT_MXFP8_MXFP4, EPI_STORE, OUT_F32)
MGE_GEMM_KERNEL(gemm_store_mxfp4, FMT_MXFP4, EPI_STORE, OUT_BF16)
MGE_GEMM_KERNEL(gemm_store_f32_mxfp4, FMT_MXFP4, EPI_STORE, OUT_F32)
MGE_GEMM_TAIL_KERNEL(gemm_store_tail_mxfp8_mxfp4, FMT_MXFP8_MXFP4, OUT_BF16)
MGE_GEMM_TAIL_KERNEL(gemm_store_f32_tail_mxfp8_mxfp4, FMT_MXFP8_MXFP4, OUT_F32)
MGE_GEMM_TAIL_KERNEL(gemm_store_tail_mxfp4, FMT_MXFP4, OUT_BF16)
MGE_GEMM_TAIL_KERNEL(gemm_store_f32_tail_mxfp4, FMT_MXFP4, OUT_F32)

// 64-row tiles of SM columns with NST LDS stages; PER_CU workgroups share a CU.  Stages against
// workgroups at the same LDS: down product of 128 tokens, top-2 of 8 experts [4096][14336], 64
// columns: 4 stages x 2 workgroups 67 us, 2 x 4 86; one [8192][8192] of 512 rows, 128 columns: 3 x 2
// 39 us, 2 x 3 51; in 4 bits, 300 rows over 8 experts, 64 columns: 3 x 2 59 us, 2 x 3 69; 512 rows,
// 128 columns: 2 x 2 70 us, 3 x 1 74.
#define MGE_GEMM_SMALL_KERNEL(name, FMT, EPI, OUT, SM, PER_CU, NST) \
  __global__ __launch_bounds__(G_THREADS, PER_CU) void name(GemmParams p) { gemm_body<FMT, EPI, RAGGED_M, OUT, 0, SM, NST>(p); }

MGE_GEMM_SMALL_KERNEL(gemm_gateup_swiglu64_mxfp8_mxfp4, FMT_MXFP8_MXFP4, EPI_SWIGLU, OUT_NONE, 256, 2, 2)
MGE_GEMM_SMALL_KERNEL(gemm_store64x128_mxfp8_mxfp4, FMT_MXFP8_MXFP4, EPI_STORE, OUT_BF16, 128, 2, 3)
MGE_GEMM_SMALL_KERNEL(gemm_store64x128_f32_mxfp8_mxfp4, FMT_MXFP8_MXFP4, EPI_STORE, OUT_F32, 128, 2, 3)
MGE_GEMM_SMALL_KERNEL(gemm_store64x64_mxfp8_mxfp4, FMT_MXFP8_MXFP4, EPI_STORE, OUT_BF16, 64, 2, 4)
MGE_GEMM_SMALL_KERNEL(gemm_store64x64_f32_mxfp8_mxfp4, FMT_MXFP8_MXFP4, EPI_STORE, OUT_F32, 64, 2, 4)
MGE_GEMM_SMALL_KERNEL(gemm_store64x128_mxfp4, FMT_MXFP4, EPI_STORE, OUT_BF16, 128, 2, 2)
MGE_GEMM_SMALL_KERNEL(gemm_store64x128_f32_mxfp4, FMT_MXFP4, EPI_STORE, OUT_F32, 128, 2, 2)
MGE_GEMM_SMALL_KERNEL(gemm_store64x64_mxfp4, FMT_MXFP4, EPI_STORE, OUT_BF16, 64, 2, 3)
MGE_GEMM_SMALL_KERNEL(gemm_store64x64_f32_mxfp4, FMT_MXFP4, EPI_STORE, OUT_F32, 64, 2, 3)

#undef MGE_GEMM_SMALL_KERNEL
#undef MGE_GEMM_TAIL_KERNEL
#undef MGE_GEMM_KERNEL

mge_status launch_gemm_mxfp4(const GemmParams& p, bool a4, hipStream_t s) {
  if (p.role == GEMM_GATEUP) return launch_gemm_kernel(gemm_gateup_swiglu_mxfp8_mxfp4, "gemm_gateup_swiglu_mxfp4", p, s);
  const bool f32 = p.out_dtype == MGE_DTYPE_F32;
  constexpr int lds8 = gemm_stage_lds(128, 128, G_BKB / 2, 2), lds4 = gemm_stage_lds(128, 128, G_BKB, 2);
  if (a4)
    return f32 ? launch_gemm_split(gemm_store_f32_mxfp4, gemm_store_f32_tail_mxfp4, "gemm_mxfp4", p, s, 2, lds4)
               : launch_gemm_split(gemm_store_mxfp4, gemm_store_tail_mxfp4, "gemm_mxfp4", p, s, 2, lds4);
  return f32 ? launch_gemm_split(gemm_store_f32_mxfp8_mxfp4, gemm_store_f32_tail_mxfp8_mxfp4, "gemm_mxfp8_mxfp4", p, s, 2, lds8)
             : launch_gemm_split(gemm_store_mxfp8_mxfp4, gemm_store_tail_mxfp8_mxfp4, "gemm_mxfp8_mxfp4", p, s, 2, lds8);
}

// 64-row tiles, of 64 columns where 128 would leave CUs without one.  Whole calls with 64 x 64 and
// 64 x 128 tiles (number of the wide ones by the rule's count), MXFP8 rows: 8 groups x [4096][14336],
// 256 rows 79 and 99 us (256), 512 rows 83 and 105 (384), 768 rows 122 and 96 (512); [8192][8192],
// 256 rows 40 and 49 (320), 512 rows 69 and 51 (576); 8 x [2048][4096], 512 rows 26.7 and 23.4 (192);
// [2048][2048], 128 rows 14.6 and 15.6 (48).  Between 320 and about 450 tiles the narrow ones, with
// their deeper stages, are the faster by a fifth: the bound was read before they had them.
constexpr int64_t kWideTiles = 320;
mge_status launch_gemm_mxfp4_small(const GemmParams& p0, bool a4, int64_t rows_bound, hipStream_t s) {
  GemmParams p = p0;
  const int64_t mt = (rows_bound + 63) / 64 + p.E;
  constexpr int B8 = G_BKB / 2, B4 = G_BKB;
  if (p.role == GEMM_GATEUP) {
    p.tiles_upper = int(mt * ((p.F + 127) / 128));
    return launch_gemm_small(gemm_gateup_swiglu64_mxfp8_mxfp4, "gemm_gateup_swiglu64_mxfp4", p, 2,
                             gemm_stage_lds(64, 256, B8, 2), s);
  }
  const bool f32 = p.out_dtype == MGE_DTYPE_F32;
  const bool wide = (mt - p.E / 2) * ((p.N + 127) / 128) >= kWideTiles;
  p.tiles_upper = int(mt * (wide ? (p.N + 127) / 128 : (p.N + 63) / 64));
  if (wide) {
    if (a4)
      return launch_gemm_small(f32 ? gemm_store64x128_f32_mxfp4 : gemm_store64x128_mxfp4, "gemm64_mxfp4", p, 2,
                               gemm_stage_lds(64, 128, B4, 2), s);
    return launch_gemm_small(f32 ? gemm_store64x128_f32_mxfp8_mxfp4 : gemm_store64x128_mxfp8_mxfp4, "gemm64_mxfp8_mxfp4",
                             p, 2, gemm_stage_lds(64, 128, B8, 3), s);
  }
  if (a4)
    return launch_gemm_small(f32 ? gemm_store64x64_f32_mxfp4 : gemm_store64x64_mxfp4, "gemm64_mxfp4", p, 2,
                             gemm_stage_lds(64, 64, B4, 3), s);
  return launch_gemm_small(f32 ? gemm_store64x64_f32_mxfp8_mxfp4 : gemm_store64x64_mxfp8_mxfp4, "gemm64_mxfp8_mxfp4", p, 2,
                           gemm_stage_lds(64, 64, B8, 4), s);
}

}  // namespace mge
