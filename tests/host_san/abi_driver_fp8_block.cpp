// Host-side driver of the norm and of the calls on FP8 with one scale per block of 128 for the
// sanitizer build, beside abi_driver.cpp: argument checks, workspace queries and empty calls, with
// inputs at and past the documented limits.  Pointers stand in for device buffers only as values;
// every call here returns before a kernel would be launched.  "abi_driver_fp8_block ok" when every
// call returned the documented status.
#include <math.h>
#include <stdio.h>

#include <vector>

#include "../../include/mge.h"

static int g_fail = 0;

#define EXPECT(expr, code)                                                                      \
  do {                                                                                          \
    const int got_ = int(expr);                                                                 \
    if (got_ != int(code)) {                                                                    \
      fprintf(stderr, "%s:%d: %s returned %d, expected %d (%s)\n", __FILE__, __LINE__, #expr, \
              got_, int(code), mge_last_error());                                               \
      ++g_fail;                                                                                 \
    }                                                                                           \
  } while (0)

static void* const A16 = reinterpret_cast<void*>(uintptr_t(0x10000));
static const int32_t kExtremes[] = {INT32_MIN, -1, 0, 1, 31, 32, 256, 257, 4096, 1 << 21, 1 << 22, 1 << 24, 1 << 30, INT32_MAX / 32 * 32, INT32_MAX};
static const int64_t kRows[] = {INT64_MIN, -1, 0, 1, 32, 1 << 20, int64_t(1) << 31, int64_t(1) << 40, INT64_MAX};

int main() {
  // ------------------------------------------------------------ norm
  EXPECT(rmsnorm_fwd(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  EXPECT(rmsnorm_bwd(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  {
    mge_rmsnorm_args a{};
    a.struct_size = sizeof(a);
    a.H = 16384; a.x_row_stride = int64_t(1) << 40;
    EXPECT(rmsnorm_fwd(&a, nullptr), MGE_OK);
    for (int32_t v : kExtremes) {
      mge_rmsnorm_args b = a;
      b.H = v;
      EXPECT(rmsnorm_fwd(&b, nullptr), v == 32 || v == 256 || v == 4096 ? MGE_OK : MGE_ERR_INVALID_ARG);
      b = a;
      b.T = v;   // above 0: no output
      EXPECT(rmsnorm_fwd(&b, nullptr), v == 0 ? MGE_OK : MGE_ERR_INVALID_ARG);
      for (int32_t u : kExtremes) (void)mge_rmsnorm_bwd_workspace_bytes(u, v);
    }
    for (int64_t v : kRows) {
      mge_rmsnorm_args b = a;
      b.x_row_stride = v;
      EXPECT(rmsnorm_fwd(&b, nullptr), v >= 16384 && v % 8 == 0 ? MGE_OK : MGE_ERR_INVALID_ARG);
    }
    a.eps = NAN;
    EXPECT(rmsnorm_fwd(&a, nullptr), MGE_ERR_INVALID_ARG);
    mge_rmsnorm_bwd_args r{};
    r.struct_size = sizeof(r);
    r.H = 64; r.x_row_stride = 64; r.dy_row_stride = 64;
    EXPECT(rmsnorm_bwd(&r, nullptr), MGE_OK);
    r.T = INT32_MAX;
    r.dy = r.x = r.weight = r.dx = A16;
    r.rstd = static_cast<float*>(A16);
    r.d_weight = static_cast<float*>(A16);
    EXPECT(rmsnorm_bwd(&r, nullptr), MGE_ERR_WORKSPACE);
  }

  // ------------------------------------------------------------ formats
  EXPECT(fp8_block_quantize(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  EXPECT(fp8_block_dequantize(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  {
    mge_quant_fb_args q{};
    q.struct_size = sizeof(q);
    q.batch = INT32_MAX; q.R = 0; q.C = 1 << 24; q.in_row_stride = int64_t(1) << 40; q.in_batch_stride = int64_t(1) << 62;
    q.orient = MGE_ORIENT_ROW | MGE_ORIENT_COL;
    EXPECT(fp8_block_quantize(&q, nullptr), MGE_OK);
    for (int32_t v : kExtremes) {
      mge_quant_fb_args b = q;
      b.R = v;   // above 0: no input
      EXPECT(fp8_block_quantize(&b, nullptr), v == 0 ? MGE_OK : MGE_ERR_INVALID_ARG);
      b = q;
      b.C = v;
      EXPECT(fp8_block_quantize(&b, nullptr), v >= 0 && v % 32 == 0 && v <= 1 << 24 ? MGE_OK : MGE_ERR_INVALID_ARG);
      b = q;
      b.block = v;
      b.batch = 1;
      EXPECT(fp8_block_quantize(&b, nullptr), v == 0 || v == 1 ? MGE_OK : MGE_ERR_INVALID_ARG);
    }
    q.batch = 1;
    q.rows = static_cast<int32_t*>(A16);
    q.src_rows = INT64_MAX;
    EXPECT(fp8_block_quantize(&q, nullptr), MGE_OK);
    q.src_rows = INT64_MIN;
    EXPECT(fp8_block_quantize(&q, nullptr), MGE_ERR_INVALID_ARG);
    mge_dequant_fb_args d{};
    d.struct_size = sizeof(d);
    d.batch = INT32_MAX; d.C = INT32_MAX / 32 * 32 - 256;
    EXPECT(fp8_block_dequantize(&d, nullptr), MGE_OK);
    d.R = INT32_MAX;
    EXPECT(fp8_block_dequantize(&d, nullptr), MGE_ERR_INVALID_ARG);
  }

  // ------------------------------------------------------------ products
  EXPECT(fp8_block_grouped_gemm(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  EXPECT(fp8_block_grouped_wgrad(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  EXPECT(grouped_mlp_fwd_fp8_block(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  for (int E : {3, 64, 65, 256}) {
    const std::vector<const uint8_t*> w(E, static_cast<const uint8_t*>(A16));   // exactly E entries: reads past them show
    const std::vector<const float*> s(E, static_cast<const float*>(A16));
    mge_gemm_fb_args g{};
    g.struct_size = sizeof(g);
    g.E = E; g.N = 64; g.K = 64; g.w = w.data(); g.w_scale = s.data();
    g.split_sizes = static_cast<int32_t*>(A16); g.group_offsets = static_cast<int32_t*>(A16);
    std::vector<uint8_t> ws(mge_gemm_fb_workspace_bytes(&g) + 16);
    if (ws.size() > 16) EXPECT(fp8_block_grouped_gemm(&g, nullptr), MGE_ERR_WORKSPACE);
    g.workspace = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws.data()) + 15) & ~uintptr_t(15));
    g.workspace_bytes = mge_gemm_fb_workspace_bytes(&g);
    EXPECT(fp8_block_grouped_gemm(&g, nullptr), MGE_OK);              // no rows
    mge_fwd_fb_args f{};
    f.struct_size = sizeof(f);
    f.E = E; f.H = 64; f.F = 96;
    f.split_sizes = static_cast<int32_t*>(A16); f.group_offsets = static_cast<int32_t*>(A16);
    f.w_gate_up = w.data(); f.w_down = w.data(); f.w_gate_up_scale = s.data(); f.w_down_scale = s.data();
    f.workspace = A16; f.workspace_bytes = mge_fwd_fb_workspace_bytes(&f);
    EXPECT(grouped_mlp_fwd_fp8_block(&f, nullptr), MGE_OK);
    const std::vector<void*> dw(E, A16);
    mge_wgrad_fb_args d{};
    d.struct_size = sizeof(d);
    d.E = E; d.N = 64; d.K = 64; d.dw = dw.data();
    for (int32_t v : kExtremes)
      for (int32_t u : kExtremes)
        for (int64_t r : kRows) {
          mge_gemm_fb_args b = g;
          b.N = v; b.K = u; b.rows = b.src_rows = r; b.total_rows = r;
          (void)mge_gemm_fb_workspace_bytes(&b);
          b.a = nullptr;   // no product of rows is launched
          const mge_status want = r == 0 && v >= 32 && v % 32 == 0 && v <= 1 << 22 && u >= 32 && u % 32 == 0 && u <= 1 << 22 &&
                                          int64_t(v) * u < int64_t(1) << 31 ? MGE_OK : MGE_ERR_INVALID_ARG;
          EXPECT(fp8_block_grouped_gemm(&b, nullptr), want);
          mge_fwd_fb_args c = f;
          c.H = v; c.F = u; c.rows = c.x_rows = r; c.total_rows = r;
          const size_t need = mge_fwd_fb_workspace_bytes(&c);
          const bool fit = r == 0 && v >= 32 && v % 32 == 0 && v <= 1 << 22 && u >= 32 && u % 32 == 0 && u <= 1 << 21 && 2 * int64_t(v) * u < int64_t(1) << 31;
          c.workspace_bytes = need;
          EXPECT(grouped_mlp_fwd_fp8_block(&c, nullptr), fit ? MGE_OK : MGE_ERR_INVALID_ARG);
          mge_wgrad_fb_args x = d;
          x.N = v; x.K = u; x.rows = r;
          (void)mge_wgrad_fb_workspace_bytes(&x);   // (no rows would write zeros: refused before it, without groups)
          EXPECT(fp8_block_grouped_wgrad(&x, nullptr), MGE_ERR_INVALID_ARG);
        }
    g.E = 257;
    EXPECT(fp8_block_grouped_gemm(&g, nullptr), MGE_ERR_INVALID_ARG);
    f.x_rows = INT64_MAX;
    EXPECT(grouped_mlp_fwd_fp8_block(&f, nullptr), MGE_ERR_INVALID_ARG);
  }

  if (g_fail) {
    fprintf(stderr, "abi_driver_fp8_block: %d failures\n", g_fail);
    return 1;
  }
  printf("abi_driver_fp8_block ok\n");
  return 0;
}
