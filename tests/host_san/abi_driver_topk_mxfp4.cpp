// Host-side driver of the router-choice and MXFP4 calls for the sanitizer build, beside
// abi_driver.cpp: argument checks, workspace queries and empty calls, with inputs at and past
// the documented limits.  Pointers stand in for device buffers only as values; every call here
// returns before a kernel would be launched.  "abi_driver_topk_mxfp4 ok" when every call
// returned the documented status.
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
static const int32_t kExtremes[] = {INT32_MIN, -1, 0, 1, 31, 32, 256, 257, 4096, 1 << 24, 1 << 30, INT32_MAX};

int main() {
  // ------------------------------------------------------------ moe_route_topk and its backward
  EXPECT(moe_route_topk(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  EXPECT(moe_route_topk_bwd(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  {
    mge_route_topk_args a{};
    a.struct_size = sizeof(a) - 8;
    EXPECT(moe_route_topk(&a, nullptr), MGE_ERR_INVALID_ARG);
    a.struct_size = sizeof(a);
    a.T = 0; a.E = 256; a.k = 8; a.score = MGE_SCORE_SIGMOID; a.num_groups = 256; a.topk_groups = 256; a.group_topn = 2;
    a.scale = 2.5f; a.logits_dtype = MGE_DTYPE_F32; a.logits_row_stride = 256;
    EXPECT(moe_route_topk(&a, nullptr), MGE_OK);
    a.scale = INFINITY;
    EXPECT(moe_route_topk(&a, nullptr), MGE_ERR_INVALID_ARG);
    a.scale = 1.f;
    for (int32_t v : kExtremes) {
      mge_route_topk_args b = a;
      b.num_groups = v;   // past E, or not a divisor: refused; a divisor: T = 0
      EXPECT(moe_route_topk(&b, nullptr), v == 256 ? MGE_OK : MGE_ERR_INVALID_ARG);
      b = a;
      b.topk_groups = v;
      EXPECT(moe_route_topk(&b, nullptr), v == 256 || v == 31 || v == 32 ? MGE_OK : MGE_ERR_INVALID_ARG);
      b = a;
      b.E = v;
      EXPECT(moe_route_topk(&b, nullptr), v == 256 ? MGE_OK : MGE_ERR_INVALID_ARG);
      b = a;
      b.k = v;
      EXPECT(moe_route_topk(&b, nullptr), v == 1 ? MGE_OK : MGE_ERR_INVALID_ARG);
    }
    a.T = INT32_MAX;
    EXPECT(moe_route_topk(&a, nullptr), MGE_ERR_INVALID_ARG);   // NULL pointers
    mge_route_topk_bwd_args r{};
    r.struct_size = sizeof(r);
    r.E = 8; r.k = 2; r.logits_dtype = MGE_DTYPE_BF16; r.logits_row_stride = 8;
    EXPECT(moe_route_topk_bwd(&r, nullptr), MGE_OK);
    r.logits_row_stride = INT64_MIN;
    EXPECT(moe_route_topk_bwd(&r, nullptr), MGE_ERR_INVALID_ARG);
    r.logits_row_stride = 8; r.T = 4; r.logits = A16; r.topk_idx = static_cast<int32_t*>(A16);
    EXPECT(moe_route_topk_bwd(&r, nullptr), MGE_ERR_INVALID_ARG);
  }

  // ------------------------------------------------------------ MXFP4 formats
  EXPECT(mxfp4_quantize(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  EXPECT(mxfp4_dequantize(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  {
    mge_quant4_args q{};
    q.struct_size = sizeof(q);
    q.batch = 65535; q.R = 0; q.C = INT32_MAX / 32 * 32; q.in_row_stride = int64_t(1) << 40; q.in_batch_stride = int64_t(1) << 62;
    q.orient = MGE_ORIENT_ROW | MGE_ORIENT_COL;
    EXPECT(mxfp4_quantize(&q, nullptr), MGE_OK);
    for (int32_t v : kExtremes) {
      mge_quant4_args b = q;
      b.R = v;   // above 0: no input
      EXPECT(mxfp4_quantize(&b, nullptr), v == 0 ? MGE_OK : MGE_ERR_INVALID_ARG);
      b = q;
      b.in_row_stride = v;
      EXPECT(mxfp4_quantize(&b, nullptr), MGE_ERR_INVALID_ARG);
    }
    mge_dequant4_args d{};
    d.struct_size = sizeof(d);
    d.codes = static_cast<uint8_t*>(A16); d.scales = static_cast<uint8_t*>(A16); d.out = A16;
    d.C = INT32_MAX / 32 * 32;
    EXPECT(mxfp4_dequantize(&d, nullptr), MGE_OK);
    d.rows = INT64_MAX;
    EXPECT(mxfp4_dequantize(&d, nullptr), MGE_ERR_INVALID_ARG);
  }

  // ------------------------------------------------------------ mxfp4_grouped_gemm
  EXPECT(mxfp4_grouped_gemm(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  {
    const std::vector<const uint8_t*> w(256, static_cast<const uint8_t*>(A16));   // exactly E entries: reads past them show
    mge_gemm4_args g{};
    g.struct_size = sizeof(g);
    g.E = 256; g.N = 64; g.K = 64; g.w = w.data(); g.w_scale = w.data();
    g.split_sizes = static_cast<int32_t*>(A16); g.group_offsets = static_cast<int32_t*>(A16);
    g.a = static_cast<uint8_t*>(A16); g.a_scale = static_cast<uint8_t*>(A16); g.out = A16;
    EXPECT(mxfp4_grouped_gemm(&g, nullptr), MGE_ERR_WORKSPACE);   // more experts than pointers travel with a launch
    std::vector<uint8_t> ws(mge_gemm4_workspace_bytes(&g) + 16);
    g.workspace = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws.data()) + 15) & ~uintptr_t(15));
    g.workspace_bytes = mge_gemm4_workspace_bytes(&g);
    EXPECT(mxfp4_grouped_gemm(&g, nullptr), MGE_OK);              // no rows
    for (int32_t v : kExtremes)
      for (int32_t u : kExtremes) {
        mge_gemm4_args b = g;
        b.N = v; b.K = u; b.rows = INT64_MAX; b.total_rows = INT64_MAX;
        if (mge_gemm4_workspace_bytes(&b) != 0) ++g_fail;
        EXPECT(mxfp4_grouped_gemm(&b, nullptr), MGE_ERR_INVALID_ARG);
        b.rows = 100; b.E = v;
        (void)mge_gemm4_workspace_bytes(&b);
      }
    g.E = 257;
    EXPECT(mxfp4_grouped_gemm(&g, nullptr), MGE_ERR_INVALID_ARG);
  }

  // ------------------------------------------------------------ grouped_mlp_fwd_mxfp4
  EXPECT(grouped_mlp_fwd_mxfp4(nullptr, nullptr), MGE_ERR_INVALID_ARG);
  {
    const std::vector<const void*> w(3, A16);
    const std::vector<const uint8_t*> s(3, static_cast<const uint8_t*>(A16));
    mge_fwd_args f{};
    f.struct_size = sizeof(f);
    f.prec = MGE_PREC_MXFP8; f.E = 3; f.H = 64; f.F = 96; f.T = 0; f.k = 2; f.align = 32;
    f.split_sizes = static_cast<int32_t*>(A16); f.group_offsets = static_cast<int32_t*>(A16);
    f.prob_perm = static_cast<float*>(A16); f.x_perm = A16; f.x_perm_scale = static_cast<uint8_t*>(A16);
    f.w_gate_up = w.data(); f.w_down = w.data(); f.w_gate_up_scale = s.data(); f.w_down_scale = s.data(); f.y_perm = A16;
    EXPECT(grouped_mlp_fwd_mxfp4(&f, nullptr), MGE_ERR_WORKSPACE);
    f.workspace = A16; f.workspace_bytes = mge_fwd_mxfp4_workspace_bytes(&f);
    EXPECT(grouped_mlp_fwd_mxfp4(&f, nullptr), MGE_OK);
    for (int32_t v : kExtremes)
      for (int32_t u : kExtremes) {
        mge_fwd_args b = f;
        b.H = v; b.F = u; b.T = 1 << 20;
        (void)mge_fwd_mxfp4_workspace_bytes(&b);
        b.T = u; b.F = 96;
        (void)mge_fwd_mxfp4_workspace_bytes(&b);
      }
    f.T = 1 << 28; f.k = 2;
    EXPECT(grouped_mlp_fwd_mxfp4(&f, nullptr), MGE_ERR_INVALID_ARG);   // rows past 32-bit offsets
    f.T = 4; f.saved_gu = static_cast<uint16_t*>(A16);
    EXPECT(grouped_mlp_fwd_mxfp4(&f, nullptr), MGE_ERR_UNSUPPORTED);
  }

  if (g_fail) {
    fprintf(stderr, "abi_driver_topk_mxfp4: %d failures\n", g_fail);
    return 1;
  }
  printf("abi_driver_topk_mxfp4 ok\n");
  return 0;
}
