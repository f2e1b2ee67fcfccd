// C ABI entry points of the norm and of FP8 with one scale per block of 128: argument checks,
// workspace carving and the launch sequence of each call (as in api.cpp: every check before the
// first launch, nothing synchronizes).
#include <math.h>

#include <algorithm>

#include "mge_common.hpp"
#include "mge_internal.hpp"

#include "fp8b.hpp"

using namespace mge;

namespace mge {

static bool is_dtype(int d) { return d == MGE_DTYPE_BF16 || d == MGE_DTYPE_F32; }
constexpr int64_t kTwoGiB = int64_t(1) << 31;
// Columns of a product and lengths of its sums: 64 rows of fp32 results and a tile's 256 rows of operands stay within a
// buffer's 31-bit offsets
constexpr int kMaxCols = 1 << 22;
constexpr int kTileRows = 256;

static mge_status check_norm(int T, int H, int x_dtype, int w_dtype, int y_dtype, int64_t ld) {
  MGE_REQUIRE(T >= 0, "T must be >= 0 (got %d)", T);
  MGE_REQUIRE(H >= 32 && H % 32 == 0 && H <= kNormMaxH, "H must be a multiple of 32 in [32, %d] (got %d)", kNormMaxH, H);
  MGE_REQUIRE(is_dtype(x_dtype) && is_dtype(w_dtype) && is_dtype(y_dtype), "x_dtype, weight_dtype and y_dtype must be BF16 or F32");
  MGE_REQUIRE(ld >= H && ld % 8 == 0, "row strides must be >= H and multiples of 8 (got %lld)", static_cast<long long>(ld));
  return MGE_OK;
}

// Streaming or tile kernels: estimates of a product's time in microseconds from what both measured on
// MI355X (whole calls, rows an expert of E x [N][K]: streamed, tiled).
//   8 x [4096][14336]: 8 rows 100, 122; 16 rows 118, 123; 32 rows 142, 127; 64 rows 217, 143
//   8 x [2048][4096]: 8 rows 17, 22; 16 rows 20, 22; 32 rows 24, 22; 64 rows 38, 22
//   16 x [1024][2048]: 8 rows 9, 15; 32 rows 13.5, 15.4; 48 rows 20, 16; 128 rows 40, 17
//   [8192][8192]: 8 rows 18, 33; 48 rows 30, 33; 64 rows 34, 33; 128 rows 64, 35
//   [4096][4096]: 8 rows 6.7, 20; 64 rows 19, 20; 128 rows 34, 20
// Streaming reads the weights at about 5 TB/s for every 64 rows, and a row past 8 adds 1/57 of that;
// the tile kernels take a fixed 8 us, 0.75 us for every 256 of K of a round of 128 x 128 tiles, and no less than
// their weights at 4.2 TB/s.
static double stream_us(int64_t E, int64_t N, int64_t K, int64_t total) {
  const double rows = double(total) / double(E), bytes = double(std::min(E, total)) * double(N) * double(K);
  return (4 + bytes / 5.0e6) * (1 + std::max(0.0, rows - 8) / 57) * std::max(1.0, ceil(rows / 64));
}
static double tile_us(int64_t E, int64_t N, int64_t K, int64_t total) {
  const double rows = double(total) / double(E), bytes = double(std::min(E, total)) * double(N) * double(K);
  const double tiles = double(std::min(E, total)) * std::max(1.0, ceil(rows / 128)) * double((N + 127) / 128);
  return 8 + std::max(0.75 * double((K + 255) / 256) * ceil(tiles / 256), bytes / 4.2e6);
}
static bool fb_tile(int64_t E, int64_t N, int64_t K, int64_t total) { return tile_us(E, N, K, total) < stream_us(E, N, K, total); }
static bool fb_tile_mlp(int64_t E, int64_t H, int64_t F, int64_t total) {
  return tile_us(E, 2 * F, H, total) + tile_us(E, H, F, total) < stream_us(E, 2 * F, H, total) + stream_us(E, H, F, total);
}
// SwiGLU in the gate-up product's epilogue needs all of a block of 128 columns, gate and up, in a workgroup: tiles of
// 256 weight rows.  Where those are half a round at most, the product in the plain form, by quadrants, fills more CUs,
// and SwiGLU follows on its own.  Whole MLP, fused and not, us: 250 tokens, one expert 4096 x 4096 (32 tiles) 78, 52;
// 250 tokens, top-2 of 8 experts 2048 x 1408 (88) 51, 47, 1000 tokens 65, 65; 256 tokens, top-2 of 4 experts 4096 x
// 4096 (128) 84, 78; 500 tokens, one expert 4096 x 14336 (224) 128, 147; 128 tokens, top-4 of 16 experts 1024 x 2048
// (256) 44, 51.
static bool fb_fused(int64_t E, int64_t F, int64_t total, bool tile) { return tile && !fb_tail_only(E, 2 * F, total); }

// Rows of all groups at most (without groups: all rows)
static int64_t fb_total(const void* sizes, int64_t total, int64_t rows) { return sizes && total > 0 && total < rows ? total : rows; }

// Few experts' pointers travel in the kernels' arguments, more through a table in the workspace
static bool fb_table(int E) { return E > kFbInline; }

}  // namespace mge

extern "C" {

mge_status rmsnorm_fwd(const mge_rmsnorm_args* a, void* stream) {
  set_error("%s", "");
  MGE_REQUIRE(a != nullptr, "args is NULL");
  MGE_REQUIRE(a->struct_size == sizeof(mge_rmsnorm_args), "struct_size mismatch");
  mge_status st = check_norm(a->T, a->H, a->x_dtype, a->weight_dtype, a->y_dtype, a->x_row_stride);
  if (st != MGE_OK) return st;
  MGE_REQUIRE(isfinite(a->eps) && a->eps >= 0.f, "eps must be finite and >= 0");
  MGE_REQUIRE((a->residual == nullptr) == (a->residual_out == nullptr), "residual and residual_out go together");
  MGE_REQUIRE((a->codes == nullptr) == (a->scales == nullptr), "codes and scales go together");
  if (a->T == 0) return MGE_OK;
  MGE_REQUIRE(a->y || a->codes, "no output asked for (y or codes)");
  MGE_REQUIRE(a->x && aligned16(a->x) && a->weight && aligned16(a->weight), "x / weight NULL or misaligned");
  MGE_REQUIRE(aligned16(a->residual) && aligned16(a->residual_out) && aligned16(a->y) && aligned16(a->codes) && aligned4(a->scales) &&
                  aligned4(a->rstd), "residual / residual_out / y / codes / scales / rstd misaligned");
  NormParams p{};
  p.T = a->T; p.H = a->H; p.x_ld = a->x_row_stride; p.eps = a->eps;
  p.w_f32 = a->weight_dtype == MGE_DTYPE_F32; p.y_f32 = a->y_dtype == MGE_DTYPE_F32;
  p.x = a->x; p.residual = a->residual; p.weight = a->weight; p.res_out = a->residual_out;
  p.y = a->y; p.rstd = a->rstd; p.codes = a->codes; p.scales = a->scales;
  return launch_rmsnorm(p, a->x_dtype == MGE_DTYPE_F32, static_cast<hipStream_t>(stream));
}

size_t mge_rmsnorm_bwd_workspace_bytes(int32_t T, int32_t H) {
  if (T <= 0 || H < 32 || H > kNormMaxH) return 0;
  return up256(size_t(rmsnorm_bwd_parts(T, H)) * H * 4);
}

mge_status rmsnorm_bwd(const mge_rmsnorm_bwd_args* a, void* stream) {
  set_error("%s", "");
  MGE_REQUIRE(a != nullptr, "args is NULL");
  MGE_REQUIRE(a->struct_size == sizeof(mge_rmsnorm_bwd_args), "struct_size mismatch");
  mge_status st = check_norm(a->T, a->H, a->x_dtype, a->weight_dtype, a->dy_dtype, a->x_row_stride);
  if (st != MGE_OK) return st;
  MGE_REQUIRE(a->dy_row_stride >= a->H && a->dy_row_stride % 8 == 0, "row strides must be >= H and multiples of 8 (got %lld)",
              static_cast<long long>(a->dy_row_stride));
  MGE_REQUIRE(a->d_weight == nullptr || aligned16(a->d_weight), "d_weight misaligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a->T == 0) return a->d_weight ? launch_rmsnorm_dw_zero(a->H, a->d_weight, s) : MGE_OK;
  MGE_REQUIRE(a->dy && aligned16(a->dy) && a->x && aligned16(a->x) && a->weight && aligned16(a->weight) && a->rstd && aligned4(a->rstd) &&
                  a->dx && aligned16(a->dx) && aligned16(a->d_residual),
              "dy / x / weight / rstd / dx NULL or misaligned, or d_residual misaligned");
  const size_t need = a->d_weight ? mge_rmsnorm_bwd_workspace_bytes(a->T, a->H) : 0;
  if (need > 0 && (!a->workspace || a->workspace_bytes < need)) {
    set_error("norm backward workspace needs %zu bytes (got %zu)", need, a->workspace_bytes);
    return MGE_ERR_WORKSPACE;
  }
  MGE_REQUIRE(need == 0 || aligned16(a->workspace), "workspace must be 16-byte aligned");
  NormBwdParams p{};
  p.T = a->T; p.H = a->H; p.x_ld = a->x_row_stride; p.dy_ld = a->dy_row_stride;
  p.w_f32 = a->weight_dtype == MGE_DTYPE_F32; p.dy_f32 = a->dy_dtype == MGE_DTYPE_F32;
  p.dy = a->dy; p.x = a->x; p.weight = a->weight; p.rstd = a->rstd; p.d_res = a->d_residual;
  p.dx = a->dx; p.dw = a->d_weight; p.part = static_cast<float*>(a->workspace);
  return launch_rmsnorm_bwd(p, a->x_dtype == MGE_DTYPE_F32, s);
}

mge_status fp8_block_quantize(const mge_quant_fb_args* a, void* stream) {
  set_error("%s", "");
  MGE_REQUIRE(a != nullptr, "args is NULL");
  MGE_REQUIRE(a->struct_size == sizeof(mge_quant_fb_args), "struct_size mismatch");
  MGE_REQUIRE(a->block == MGE_BLOCK_1X128 || a->block == MGE_BLOCK_128X128, "block must be 1X128 or 128X128 (got %d)", a->block);
  MGE_REQUIRE(a->batch >= 0 && a->R >= 0 && a->C >= 0, "negative size");
  MGE_REQUIRE(a->C % 32 == 0 && a->C <= 1 << 24 && a->R <= 0x7fffff00, "C must be a multiple of 32 and at most 2^24, R at most %d (got %d, %d)",
              0x7fffff00, a->C, a->R);
  MGE_REQUIRE(a->orient != 0 && (a->orient & ~3u) == 0, "orient must be ROW, COL or ROW|COL");
  MGE_REQUIRE(!a->rows || (a->batch <= 1 && a->block == MGE_BLOCK_1X128 && a->src_rows >= 0 && aligned4(a->rows)),
              "a row map needs one matrix, 1x128 blocks and src_rows >= 0");
  const int64_t in_rows = a->rows ? a->src_rows : a->R;
  MGE_REQUIRE((a->in || in_rows == 0 || a->R == 0 || a->C == 0 || a->batch == 0) && aligned16(a->in),
              "in must be non-NULL and 16-byte aligned");
  MGE_REQUIRE(a->in_row_stride >= a->C && a->in_row_stride % 8 == 0, "in_row_stride must be >= C and a multiple of 8");
  MGE_REQUIRE(a->batch <= 1 || (a->in_batch_stride % 8 == 0 && a->in_batch_stride >= int64_t(a->R) * a->in_row_stride),
              "in_batch_stride too small or not a multiple of 8");
  if (a->batch == 0 || a->R == 0 || a->C == 0) return MGE_OK;   // no element, no output
  if (a->orient & MGE_ORIENT_ROW)
    MGE_REQUIRE(a->row_codes && a->row_scales && aligned16(a->row_codes) && aligned4(a->row_scales), "row outputs missing or misaligned");
  if (a->orient & MGE_ORIENT_COL)
    MGE_REQUIRE(a->col_codes && a->col_scales && aligned16(a->col_codes) && aligned4(a->col_scales), "column outputs missing or misaligned");
  QuantFbParams q{};
  q.in = a->in; q.in_bstride = a->in_batch_stride; q.in_ld = a->in_row_stride;
  q.map = a->rows; q.src_rows = a->src_rows;
  q.batch = a->batch; q.R = a->R; q.Rp = (int64_t(a->R) + 31) / 32 * 32; q.C = a->C;
  q.tile = a->block == MGE_BLOCK_128X128;
  if (a->orient & MGE_ORIENT_ROW) { q.row_codes = a->row_codes; q.row_scales = a->row_scales; }
  if (a->orient & MGE_ORIENT_COL) { q.col_codes = a->col_codes; q.col_scales = a->col_scales; }
  return launch_quant_fb(q, static_cast<hipStream_t>(stream));
}

mge_status fp8_block_dequantize(const mge_dequant_fb_args* a, void* stream) {
  set_error("%s", "");
  MGE_REQUIRE(a != nullptr, "args is NULL");
  MGE_REQUIRE(a->struct_size == sizeof(mge_dequant_fb_args), "struct_size mismatch");
  MGE_REQUIRE(a->block == MGE_BLOCK_1X128 || a->block == MGE_BLOCK_128X128, "block must be 1X128 or 128X128 (got %d)", a->block);
  MGE_REQUIRE(a->batch >= 0 && a->R >= 0 && a->C >= 0 && a->C % 32 == 0, "sizes must be >= 0 and C a multiple of 32");
  MGE_REQUIRE(a->C <= 0x7fffff00 && a->R <= 0x7fffff00, "C and R must be at most %d (got %d, %d)", 0x7fffff00, a->C, a->R);
  MGE_REQUIRE(is_dtype(a->out_dtype), "out_dtype must be BF16 or F32");
  if (a->batch == 0 || a->R == 0 || a->C == 0) return MGE_OK;
  MGE_REQUIRE(a->codes && aligned16(a->codes) && a->scales && aligned4(a->scales) && a->out && aligned16(a->out),
              "codes / scales / out NULL or misaligned");
  return launch_dequant_fb(a->batch, a->R, a->C, a->block == MGE_BLOCK_128X128, a->codes, a->scales, a->out_dtype, a->out,
                           static_cast<hipStream_t>(stream));
}

size_t mge_gemm_fb_workspace_bytes(const mge_gemm_fb_args* a) {
  if (!a || a->struct_size != sizeof(mge_gemm_fb_args) || a->E < 1 || a->E > 256 || a->N < 32 || a->K < 32 || a->rows < 0 || a->rows >= kTwoGiB / a->K)
    return 0;
  const int64_t total = fb_total(a->split_sizes, a->total_rows, a->rows);
  const bool tile = fb_tile(a->E, a->N, a->K, total);
  return (fb_table(a->E) ? up256(2 * size_t(a->E) * sizeof(void*)) : 0) +
         (tile && !fb_tail_only(a->E, a->N, total) ? fb_scales_bytes(a->rows, a->K) : 0);
}

mge_status fp8_block_grouped_gemm(const mge_gemm_fb_args* a, void* stream) {
  set_error("%s", "");
  MGE_REQUIRE(a != nullptr, "args is NULL");
  MGE_REQUIRE(a->struct_size == sizeof(mge_gemm_fb_args), "struct_size mismatch");
  MGE_REQUIRE(a->E >= 1 && a->E <= 256, "E must be in [1, 256] (got %d)", a->E);
  MGE_REQUIRE(a->N >= 32 && a->N % 32 == 0 && a->N <= kMaxCols && a->K >= 32 && a->K % 32 == 0 && a->K <= kMaxCols,
              "N and K must be positive multiples of 32, at most %d (got N=%d, K=%d)", kMaxCols, a->N, a->K);
  MGE_REQUIRE(a->rows >= 0 && a->rows < kTwoGiB / a->K && a->src_rows >= 0 && a->src_rows < kTwoGiB / a->K,
              "rows and src_rows must be in [0, 2^31 / K) (got %lld, %lld)", static_cast<long long>(a->rows),
              static_cast<long long>(a->src_rows));
  MGE_REQUIRE(a->a_rows || a->src_rows == a->rows, "without a row map src_rows must be rows");
  MGE_REQUIRE(a->total_rows >= 0, "total_rows must be >= 0");
  MGE_REQUIRE(int64_t(a->N) * a->K < kTwoGiB, "an expert's weight must be below 2^31 bytes");
  MGE_REQUIRE((a->split_sizes != nullptr) == (a->group_offsets != nullptr) && (a->split_sizes || a->E == 1),
              "split_sizes and group_offsets go together, and E > 1 needs both");
  MGE_REQUIRE(is_dtype(a->out_dtype), "out_dtype must be BF16 or F32");
  MGE_REQUIRE(a->w && a->w_scale, "weight pointer arrays are NULL");
  for (int e = 0; e < a->E; ++e)
    MGE_REQUIRE(a->w[e] && aligned16(a->w[e]) && a->w_scale[e] && aligned4(a->w_scale[e]),
                "weight of expert %d or its scales NULL or misaligned", e);
  if (a->rows > 0)
    MGE_REQUIRE(((a->a && a->a_scale) || a->src_rows == 0) && aligned16(a->a) && aligned4(a->a_scale) && a->out && aligned16(a->out) &&
                    aligned4(a->a_rows),
                "a / a_scale / out NULL or misaligned, or a_rows misaligned");
  const size_t need = mge_gemm_fb_workspace_bytes(a);
  if (need > 0 && (!a->workspace || a->workspace_bytes < need)) {
    set_error("FP8 block product workspace needs %zu bytes (got %zu)", need, a->workspace_bytes);
    return MGE_ERR_WORKSPACE;
  }
  MGE_REQUIRE(need == 0 || aligned16(a->workspace), "workspace must be 16-byte aligned");
  if (a->rows == 0) return MGE_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Carve ws(a->workspace);
  FbGemm p{};
  p.E = a->E; p.N = a->N; p.K = a->K;
  p.rows = int(a->rows); p.total = int(fb_total(a->split_sizes, a->total_rows, a->rows));
  p.sizes = a->split_sizes; p.offs = a->group_offsets;
  p.map = a->a_rows; p.src_rows = int(a->src_rows);
  p.A = a->a; p.As = a->a_scale;
  p.C = a->out; p.out_f32 = a->out_dtype == MGE_DTYPE_F32;
  if (fb_table(a->E)) {
    void** tab = static_cast<void**>(ws.take(2 * size_t(a->E) * sizeof(void*)));
    const void* const* tabs[4] = {reinterpret_cast<const void* const*>(a->w), reinterpret_cast<const void* const*>(a->w_scale), nullptr, nullptr};
    const mge_status st = launch_upload_tables(tabs, 2, a->E, tab, s);
    if (st != MGE_OK) return st;
    p.W = reinterpret_cast<const uint8_t* const*>(tab);
    p.Ws = reinterpret_cast<const float* const*>(tab + a->E);
  } else {
    for (int e = 0; e < a->E; ++e) {
      p.Wv[e] = a->w[e];
      p.Wsv[e] = a->w_scale[e];
    }
  }
  if (!fb_tile(p.E, p.N, p.K, p.total)) return launch_fb_stream(p, s);
  if (fb_tail_only(p.E, p.N, p.total)) return launch_fb_tile(p, false, s);
  float* ast = static_cast<float*>(ws.take(fb_scales_bytes(a->rows, a->K)));   // (block-major, by row of the groups)
  p.Ast = ast; p.ast_ld = a->rows;
  const FbScaleT t{a->a_scale, a->a_rows, a->src_rows, a->rows, int(fb_blocks(a->K)), ast, a->rows};
  const mge_status st = launch_fb_scale_t(&t, 1, s);
  return st != MGE_OK ? st : launch_fb_tile(p, false, s);
}

// (with block-major scales whatever the tiles: their choice goes by the device's CUs, a size asked for beforehand does not)
size_t mge_wgrad_fb_workspace_bytes(const mge_wgrad_fb_args* a) {
  if (!a || a->struct_size != sizeof(mge_wgrad_fb_args) || a->E < 1 || a->E > 256 || a->N < 32 || a->K < 32 || a->rows < 0 ||
      a->rows >= kTwoGiB / std::max({a->N, a->K, kTileRows}))
    return 0;
  return (fb_table(a->E) ? up256(size_t(a->E) * sizeof(void*)) : 0) + fb_scales_bytes(a->N, a->rows) + fb_scales_bytes(a->K, a->rows);
}

mge_status fp8_block_grouped_wgrad(const mge_wgrad_fb_args* a, void* stream) {
  set_error("%s", "");
  MGE_REQUIRE(a != nullptr, "args is NULL");
  MGE_REQUIRE(a->struct_size == sizeof(mge_wgrad_fb_args), "struct_size mismatch");
  MGE_REQUIRE(a->E >= 1 && a->E <= 256, "E must be in [1, 256] (got %d)", a->E);
  MGE_REQUIRE(a->N >= 32 && a->N % 32 == 0 && a->K >= 32 && a->K % 32 == 0 && a->N <= kMaxCols && a->K <= kMaxCols,
              "N and K must be positive multiples of 32, at most %d (got N=%d, K=%d)", kMaxCols, a->N, a->K);
  MGE_REQUIRE(a->rows >= 0 && a->rows % 32 == 0 && a->rows < kTwoGiB / std::max({a->N, a->K, kTileRows}),
              "rows must be a multiple of 32 in [0, 2^31 / max(N, K, 256)) (got %lld)", static_cast<long long>(a->rows));
  MGE_REQUIRE((a->split_sizes != nullptr) == (a->group_offsets != nullptr) && (a->split_sizes || a->E == 1),
              "split_sizes and group_offsets go together, and E > 1 needs both");
  MGE_REQUIRE(is_dtype(a->out_dtype) && (!a->accumulate || a->out_dtype == MGE_DTYPE_F32), "out_dtype must be BF16 or F32, F32 to accumulate");
  MGE_REQUIRE(a->dw != nullptr, "dw is NULL");
  for (int e = 0; e < a->E; ++e) MGE_REQUIRE(a->dw[e] && aligned16(a->dw[e]), "dw[%d] NULL or misaligned", e);
  if (a->rows > 0)
    MGE_REQUIRE(a->dy && aligned16(a->dy) && a->dy_scale && aligned4(a->dy_scale) && a->x && aligned16(a->x) && a->x_scale &&
                    aligned4(a->x_scale),
                "dy / dy_scale / x / x_scale NULL or misaligned");
  const size_t need = mge_wgrad_fb_workspace_bytes(a);
  if (need > 0 && (!a->workspace || a->workspace_bytes < need)) {
    set_error("FP8 block weight gradient workspace needs %zu bytes (got %zu)", need, a->workspace_bytes);
    return MGE_ERR_WORKSPACE;
  }
  MGE_REQUIRE(need == 0 || aligned16(a->workspace), "workspace must be 16-byte aligned");
  hipStream_t s = static_cast<hipStream_t>(stream);
  Carve ws(a->workspace);
  FbWgrad p{};
  p.E = a->E; p.N = a->N; p.K = a->K; p.rows = int(a->rows);
  p.sizes = a->split_sizes; p.offs = a->group_offsets;
  p.Y = a->dy; p.X = a->x;
  if (fb_table(a->E)) {
    void** tab = static_cast<void**>(ws.take(size_t(a->E) * sizeof(void*)));
    const void* const* tabs[4] = {const_cast<const void* const*>(a->dw), nullptr, nullptr, nullptr};
    const mge_status st = launch_upload_tables(tabs, 1, a->E, tab, s);
    if (st != MGE_OK) return st;
    p.D = tab;
  } else {
    for (int e = 0; e < a->E; ++e) p.Dv[e] = a->dw[e];
  }
  const int nb = int(fb_blocks(a->rows));
  float* yst = static_cast<float*>(ws.take(fb_scales_bytes(a->N, a->rows)));
  float* xst = static_cast<float*>(ws.take(fb_scales_bytes(a->K, a->rows)));
  p.Ys = a->dy_scale; p.Xs = a->x_scale; p.Yst = yst; p.Xst = xst;
  p.out = a->accumulate ? OUT_F32_ACC : (a->out_dtype == MGE_DTYPE_F32 ? OUT_F32 : OUT_BF16);
  if (fb_wgrad_small(p)) return launch_fb_wgrad(p, s);
  const FbScaleT t[2] = {{a->dy_scale, nullptr, a->N, a->N, nb, yst, a->N}, {a->x_scale, nullptr, a->K, a->K, nb, xst, a->K}};
  const mge_status st = launch_fb_scale_t(t, 2, s);
  return st != MGE_OK ? st : launch_fb_wgrad(p, s);
}

size_t mge_fwd_fb_workspace_bytes(const mge_fwd_fb_args* a) {
  if (!a || a->struct_size != sizeof(mge_fwd_fb_args) || a->E < 1 || a->E > 256 || a->H < 32 || a->F < 32 || a->rows < 0 ||
      a->rows >= kTwoGiB / std::max(a->H, a->F))
    return 0;
  const int64_t total = fb_total(a->split_sizes, a->total_rows, a->rows);
  const bool tile = fb_tile_mlp(a->E, a->H, a->F, total);
  return (fb_table(a->E) ? up256(4 * size_t(a->E) * sizeof(void*)) : 0) + up256(size_t(a->rows) * a->F) + fb_scales_bytes(a->rows, a->F) +
         (fb_fused(a->E, a->F, total, tile) ? fb_scales_bytes(a->rows, a->H) : up256(size_t(a->rows) * a->F * 8));
}

mge_status grouped_mlp_fwd_fp8_block(const mge_fwd_fb_args* a, void* stream) {
  set_error("%s", "");
  MGE_REQUIRE(a != nullptr, "args is NULL");
  MGE_REQUIRE(a->struct_size == sizeof(mge_fwd_fb_args), "struct_size mismatch");
  MGE_REQUIRE(a->E >= 1 && a->E <= 256, "E must be in [1, 256] (got %d)", a->E);
  MGE_REQUIRE(a->H >= 32 && a->H % 32 == 0 && a->F >= 32 && a->F % 32 == 0 && a->H <= kMaxCols && a->F <= kMaxCols / 2,
              "H and F must be positive multiples of 32, at most %d and %d (got H=%d, F=%d)", kMaxCols, kMaxCols / 2, a->H, a->F);
  MGE_REQUIRE(a->rows >= 0 && a->rows < kTwoGiB / std::max(a->H, a->F) && a->x_rows >= 0 && a->x_rows < kTwoGiB / a->H,
              "rows must be in [0, 2^31 / max(H, F)) and x_rows in [0, 2^31 / H) (got %lld, %lld)", static_cast<long long>(a->rows),
              static_cast<long long>(a->x_rows));
  MGE_REQUIRE(a->perm_src || a->x_rows == a->rows, "without perm_src x_rows must be rows");
  MGE_REQUIRE(a->total_rows >= 0, "total_rows must be >= 0");
  MGE_REQUIRE(2 * int64_t(a->F) * a->H < kTwoGiB, "an expert's gate-up weight must be below 2^31 bytes");
  MGE_REQUIRE((a->split_sizes != nullptr) == (a->group_offsets != nullptr) && (a->split_sizes || a->E == 1),
              "split_sizes and group_offsets go together, and E > 1 needs both");
  MGE_REQUIRE(is_dtype(a->y_dtype), "y_dtype must be BF16 or F32");
  MGE_REQUIRE(a->w_gate_up && a->w_down && a->w_gate_up_scale && a->w_down_scale, "weight pointer arrays are NULL");
  for (int e = 0; e < a->E; ++e) {
    MGE_REQUIRE(a->w_gate_up[e] && aligned16(a->w_gate_up[e]) && a->w_gate_up_scale[e] && aligned4(a->w_gate_up_scale[e]),
                "w_gate_up[%d] or its scales NULL or misaligned", e);
    MGE_REQUIRE(a->w_down[e] && aligned16(a->w_down[e]) && a->w_down_scale[e] && aligned4(a->w_down_scale[e]),
                "w_down[%d] or its scales NULL or misaligned", e);
  }
  if (a->rows > 0)
    MGE_REQUIRE(((a->x && a->x_scale) || a->x_rows == 0) && aligned16(a->x) && aligned4(a->x_scale) && a->y_perm && aligned16(a->y_perm) &&
                    aligned4(a->perm_src) && aligned4(a->prob_perm),
                "x / x_scale / y_perm NULL or misaligned, or perm_src / prob_perm misaligned");
  const size_t need = mge_fwd_fb_workspace_bytes(a);
  if (need > 0 && (!a->workspace || a->workspace_bytes < need)) {
    set_error("forward workspace needs %zu bytes (got %zu)", need, a->workspace_bytes);
    return MGE_ERR_WORKSPACE;
  }
  MGE_REQUIRE(need == 0 || aligned16(a->workspace), "workspace must be 16-byte aligned");
  if (a->rows == 0) return MGE_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Carve ws(a->workspace);
  const int E = a->E, H = a->H, F = a->F;
  FbGemm g{};
  g.E = E; g.N = 2 * F; g.K = H; g.F = F;
  g.rows = int(a->rows); g.total = int(fb_total(a->split_sizes, a->total_rows, a->rows));
  g.sizes = a->split_sizes; g.offs = a->group_offsets;
  g.map = a->perm_src; g.src_rows = int(a->x_rows);
  g.A = a->x; g.As = a->x_scale; g.prob = a->prob_perm;
  FbGemm d{};
  d.E = E; d.N = H; d.K = F;
  d.rows = g.rows; d.total = g.total; d.sizes = g.sizes; d.offs = g.offs; d.src_rows = g.rows;
  d.C = a->y_perm; d.out_f32 = a->y_dtype == MGE_DTYPE_F32;
  mge_status st = MGE_OK;
  if (fb_table(E)) {
    void** tab = static_cast<void**>(ws.take(4 * size_t(E) * sizeof(void*)));
    const void* const* tabs[4] = {reinterpret_cast<const void* const*>(a->w_gate_up), reinterpret_cast<const void* const*>(a->w_gate_up_scale),
                                  reinterpret_cast<const void* const*>(a->w_down), reinterpret_cast<const void* const*>(a->w_down_scale)};
    st = launch_upload_tables(tabs, 4, E, tab, s);
    if (st != MGE_OK) return st;
    g.W = reinterpret_cast<const uint8_t* const*>(tab);
    g.Ws = reinterpret_cast<const float* const*>(tab + E);
    d.W = reinterpret_cast<const uint8_t* const*>(tab + 2 * E);
    d.Ws = reinterpret_cast<const float* const*>(tab + 3 * E);
  } else {
    for (int e = 0; e < E; ++e) {
      g.Wv[e] = a->w_gate_up[e];
      g.Wsv[e] = a->w_gate_up_scale[e];
      d.Wv[e] = a->w_down[e];
      d.Wsv[e] = a->w_down_scale[e];
    }
  }
  g.h_codes = static_cast<uint8_t*>(ws.take(size_t(a->rows) * F));
  g.h_scales = static_cast<float*>(ws.take(fb_scales_bytes(a->rows, F)));
  d.A = g.h_codes; d.As = g.h_scales; d.Ast = g.h_scales; d.ast_ld = a->rows;
  const bool tile = fb_tile_mlp(E, H, F, g.total);
  const bool fused = fb_fused(E, F, g.total, tile);
  if (fused) {   // (the quadrants take the tokens' scales as they come)
    float* xst = static_cast<float*>(ws.take(fb_scales_bytes(a->rows, H)));
    g.Ast = xst; g.ast_ld = a->rows;
    const FbScaleT t{a->x_scale, a->perm_src, a->x_rows, a->rows, int(fb_blocks(H)), xst, a->rows};
    st = launch_fb_scale_t(&t, 1, s);
    if (st != MGE_OK) return st;
  }
  if (fused) {
    st = launch_fb_tile(g, true, s);
  } else {
    float* gu = static_cast<float*>(ws.take(size_t(a->rows) * F * 8));
    g.C = gu;
    g.out_f32 = 1;
    st = tile ? launch_fb_tile(g, false, s) : launch_fb_stream(g, s);
    if (st == MGE_OK) st = launch_fb_swiglu(g, gu, tile ? a->rows : 0, s);
  }
  if (st != MGE_OK) return st;
  return tile ? launch_fb_tile(d, false, s) : launch_fb_stream(d, s);
}

}  // extern "C"
