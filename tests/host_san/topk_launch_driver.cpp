// Launches of the router choice and its backward, recorded instead of made: this driver defines the
// runtime's launch functions itself, so that launch_topk and launch_topk_bwd run on the CPU with any
// number of tokens.  For every form it checks that a launch has fewer than 2^32 threads, that its
// workgroups are those of its tokens, and that the launches of a call cover the tokens one after the
// other, each with its own part of every array.  "topk_launch_driver ok" when all hold.
#include <hip/hip_runtime.h>
#include <stdio.h>

#include "../../include/mge.h"
#include "../../moe_grouped_expert_amd/csrc/mge_internal.hpp"

namespace mge {
ProfScope::ProfScope(hipStream_t s, const char*) : stream(s), slot(-1) {}
ProfScope::~ProfScope() {}
mge_status hip_check(const char*) { return MGE_OK; }
}  // namespace mge

static bool g_bwd;
static int g_dtype, g_fail;
static int64_t g_done;
static mge::TopkParams g_f;
static mge::TopkBwdParams g_b;
static dim3 g_grid, g_block;

static void need(bool ok, const char* what, long long v) {
  if (ok) return;
  fprintf(stderr, "%s (%lld) after %lld tokens, %s\n", what, v, static_cast<long long>(g_done), g_bwd ? "backward" : "forward");
  ++g_fail;
}
static bool at(const void* p, const void* base, int64_t bytes) {
  return p == static_cast<const char*>(base) + bytes;
}

extern "C" {
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
  g_grid = grid;
  g_block = block;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
  *grid = g_grid;
  *block = g_block;
  *lds = 0;
  *s = nullptr;
  return hipSuccess;
}
void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, dim3*, dim3*, int*) {}

hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
  const int64_t threads = int64_t(grid.x) * block.x;
  need(threads < (int64_t(1) << 32) && grid.y == 1 && grid.z == 1, "threads of a launch", threads);
  const int64_t es = g_dtype == MGE_DTYPE_F32 ? 4 : 2;
  int64_t T;
  if (g_bwd) {
    const auto& p = *static_cast<const mge::TopkBwdParams*>(args[0]);
    T = p.T;
    need(at(p.logits, g_b.logits, g_done * p.ld * es) && at(p.topk_idx, g_b.topk_idx, g_done * p.k * 4) &&
             at(p.d_prob, g_b.d_prob, g_done * p.k * 4) && at(p.d_logits, g_b.d_logits, g_done * p.E * es),
         "pointers", T);
  } else {
    const auto& p = *static_cast<const mge::TopkParams*>(args[0]);
    T = p.T;
    need(at(p.logits, g_f.logits, g_done * p.ld * es) && at(p.topk_idx, g_f.topk_idx, g_done * p.k * 4) &&
             at(p.topk_prob, g_f.topk_prob, g_done * p.k * 4) && p.bias == g_f.bias,
         "pointers", T);
  }
  // 16 or 64 lanes a token
  need(int64_t(grid.x) == (T * 16 + 255) / 256 || int64_t(grid.x) == (T * 64 + 255) / 256, "workgroups", grid.x);
  g_done += T;
  return hipSuccess;
}
}

int main() {
  static const int64_t kTokens[] = {1, 2048, 2049, 1 << 20, (1 << 25) - 1, 1 << 25, (1 << 25) + 1, (1 << 26) + 3, (1 << 28) + 37, INT32_MAX};
  struct Shape { int E, k, G, topg; };
  static const Shape kShapes[] = {{1, 1, 1, 1}, {8, 2, 1, 1}, {60, 6, 4, 2}, {256, 8, 8, 4}, {255, 8, 17, 4}};   // the last: groups that walk
  for (int64_t T : kTokens)
    for (const Shape& sh : kShapes)
      for (int dtype : {MGE_DTYPE_BF16, MGE_DTYPE_F32}) {
        void* const base = reinterpret_cast<void*>(uintptr_t(1) << 40);
        g_dtype = dtype;
        g_bwd = false;
        g_done = 0;
        g_f = mge::TopkParams{};
        g_f.T = T; g_f.ld = sh.E + 8; g_f.E = sh.E; g_f.k = sh.k; g_f.G = sh.G; g_f.topg = sh.topg; g_f.topn = 2; g_f.scale = 1.f;
        g_f.logits = base; g_f.topk_idx = static_cast<int32_t*>(base); g_f.topk_prob = static_cast<float*>(base);
        mge::launch_topk(g_f, dtype, nullptr);
        need(g_done == T, "tokens", T);
        g_bwd = true;
        g_done = 0;
        g_b = mge::TopkBwdParams{};
        g_b.T = T; g_b.ld = sh.E + 8; g_b.E = sh.E; g_b.k = sh.k; g_b.scale = 1.f;
        g_b.logits = base; g_b.topk_idx = static_cast<int32_t*>(base); g_b.d_prob = static_cast<float*>(base); g_b.d_logits = base;
        mge::launch_topk_bwd(g_b, dtype, nullptr);
        need(g_done == T, "tokens", T);
      }
  if (g_fail) {
    fprintf(stderr, "topk_launch_driver: %d failures\n", g_fail);
    return 1;
  }
  printf("topk_launch_driver ok\n");
  return 0;
}
