// The grouped-GEMM kernels with MXFP4 weights (block-scaled 4-bit MFMA), for groups of many
// rows: the tile kernel of gemm_impl.hpp in its 4-bit formats.  mxfp8_mxfp4: rows in MXFP8
// (the expert MLP's activations), mxfp4: rows in MXFP4 too, at twice the matrix rate.
#include "gemm_impl.hpp"

namespace mge {

#define MGE_GEMM_KERNEL(name, FMT, EPI, OUT) \
  __global__ __launch_bounds__(G_THREADS, 1) void name(GemmParams p) { gemm_body<FMT, EPI, RAGGED_M, OUT>(p); }
#define MGE_GEMM_TAIL_KERNEL(name, FMT, OUT) \
  __global__ __launch_bounds__(G_THREADS, 1) void name(GemmParams p) { gemm_body<FMT, EPI_STORE, RAGGED_M, OUT, 1>(p); }

MGE_GEMM_KERNEL(gemm_gateup_swiglu_mxfp8_mxfp4, FMT_MXFP8_MXFP4, EPI_SWIGLU, OUT_NONE)
MGE_GEMM_KERNEL(gemm_store_mxfp8_mxfp4, FMT_MXFP8_MXFP4, EPI_STORE, OUT_BF16)
MGE_GEMM_KERNEL(gemm_store_f32_mxfp8_mxfp4, FMT_MXFP8_MXFP4, EPI_STORE, OUT_F32)
MGE_GEMM_KERNEL(gemm_store_mxfp4, FMT_MXFP4, EPI_STORE, OUT_BF16)
MGE_GEMM_KERNEL(gemm_store_f32_mxfp4, FMT_MXFP4, EPI_STORE, OUT_F32)
MGE_GEMM_TAIL_KERNEL(gemm_store_tail_mxfp8_mxfp4, FMT_MXFP8_MXFP4, OUT_BF16)
MGE_GEMM_TAIL_KERNEL(gemm_store_f32_tail_mxfp8_mxfp4, FMT_MXFP8_MXFP4, OUT_F32)
MGE_GEMM_TAIL_KERNEL(gemm_store_tail_mxfp4, FMT_MXFP4, OUT_BF16)
MGE_GEMM_TAIL_KERNEL(gemm_store_f32_tail_mxfp4, FMT_MXFP4, OUT_F32)

#undef MGE_GEMM_TAIL_KERNEL
#undef MGE_GEMM_KERNEL

mge_status launch_gemm_mxfp4(const GemmParams& p, bool a4, hipStream_t s) {
  if (p.role == GEMM_GATEUP) return launch_gemm_kernel(gemm_gateup_swiglu_mxfp8_mxfp4, "gemm_gateup_swiglu_mxfp4", p, s);
  const bool f32 = p.out_dtype == MGE_DTYPE_F32;
  if (a4)
    return f32 ? launch_gemm_split(gemm_store_f32_mxfp4, gemm_store_f32_tail_mxfp4, "gemm_mxfp4", p, s)
               : launch_gemm_split(gemm_store_mxfp4, gemm_store_tail_mxfp4, "gemm_mxfp4", p, s);
  return f32 ? launch_gemm_split(gemm_store_f32_mxfp8_mxfp4, gemm_store_f32_tail_mxfp8_mxfp4, "gemm_mxfp8_mxfp4", p, s)
             : launch_gemm_split(gemm_store_mxfp8_mxfp4, gemm_store_tail_mxfp8_mxfp4, "gemm_mxfp8_mxfp4", p, s);
}

}  // namespace mge
