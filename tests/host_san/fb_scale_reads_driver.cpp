// Which scales the FP8 block tile kernels read (CPU only): every wave's resource (fb_scale_span), its lanes' offsets and
// its slices' places, over odd numbers of rows, columns and slices, against the table's size: fb_scales_bytes for the
// block-major ones in the workspace, exactly the matrix's scales for those read as they come.  A lane's access counts
// as made if either form of a buffer's range check lets it through: the lane's offset against the resource's bytes, or
// against those less the scalar offset, as an unsigned number.  The same enumeration with a resource that is empty only
// behind the whole table has to fail, so that the check sees what it is for.  "fb_scale_reads ok" when both hold.
#include <stdint.h>
#include <stdio.h>

#include <algorithm>

#include "../../moe_grouped_expert_amd/csrc/mge_common.hpp"
#include "../../moe_grouped_expert_amd/csrc/fp8b.hpp"

using mge::FbSpan;
using mge::fb_blocks;
using mge::fb_scale_span;
using mge::fb_scales_bytes;

static bool g_whole;       // the resource that is empty only behind the whole table
static int64_t g_worst;    // bytes read past a table's end at most
static int64_t g_reads;

static FbSpan span(int64_t row, int64_t rows, int64_t blk, int64_t nb, bool by_row) {
  FbSpan s = fb_scale_span(row, rows, blk, nb, by_row);
  if (g_whole) s.bytes = s.at < rows * nb ? uint32_t(rows * nb - s.at) * 4 : 0;
  return s;
}

// `slices` of a wave: lane l at l * lane_ld bytes, slice k at k * slice_ld bytes, in a table of `size` bytes
static void wave(FbSpan s, int64_t lane_ld, int lanes, int64_t slices, int64_t slice_ld, int64_t size) {
  if (s.bytes == 0) return;
  for (int64_t k : {int64_t(0), int64_t(1), slices / 2, slices - 2, slices - 1}) {
    if (k < 0 || k >= slices) continue;
    const uint32_t soff = uint32_t(k * slice_ld);
    for (int l = 0; l < lanes; ++l) {
      const uint32_t voff = uint32_t(l * lane_ld);
      if (voff < s.bytes || voff < uint32_t(s.bytes - soff)) {
        g_worst = std::max(g_worst, s.at * 4 + int64_t(voff) + soff + 4 - size);
        ++g_reads;
      }
    }
  }
}

// The weight gradient: tiles of nt x nr, one operand's rows n, tile starts every `step` of them, `waves` waves of 64 rows
static void wgrad(int64_t n, int64_t rows, int step, int waves, bool by_row) {
  const int64_t nb = fb_blocks(rows), size = by_row ? n * nb * 4 : int64_t(fb_scales_bytes(n, rows));
  for (int64_t r0 = 0; r0 < n; r0 += step)
    for (int w = 0; w < waves; ++w)
      for (int64_t b0 : {int64_t(0), nb / 2, nb - 1}) {   // (a group's first block)
        const FbSpan s = span(r0 + w * 64, n, b0, nb, by_row);
        wave(s, by_row ? nb * 4 : 4, 64, nb - b0, by_row ? 4 : n * 4, size);
      }
}

// The product: a group at `off` of `size` tokens, tiles of nt tokens from every multiple of `step`
static void gemm(int64_t rows, int64_t K, int64_t off, int64_t count, int nt, int step) {
  const int64_t kb = fb_blocks(K), size = int64_t(fb_scales_bytes(rows, K));
  for (int64_t m0 = 0; m0 < count; m0 += step)
    for (int q = 0; q < step; q += nt)
      for (int w = 0; w < nt / 64; ++w)
        wave(span(off + m0 + q + w * 64, rows, 0, kb, false), 4, 64, kb, rows * 4, size);
}

// Weight scales of the product: the tile's blocks of 128 rows, `lanes` of them
static void weights(int64_t N, int64_t K, int step, int lanes) {
  const int64_t kb = fb_blocks(K), nb = fb_blocks(N);
  for (int64_t n0 = 0; n0 < N; n0 += step) wave(span(n0 / 128, nb, 0, kb, true), kb * 4, lanes, kb, 4, nb * kb * 4);
}

static int64_t worst(bool whole) {
  g_whole = whole;
  g_worst = INT64_MIN;
  g_reads = 0;
  const int64_t sizes[] = {32, 64, 96, 128, 160, 224, 256, 288, 416, 512, 544, 1056, 1184, 2080, 4096, 4128};
  const int64_t counts[] = {1, 2, 31, 32, 63, 64, 65, 127, 128, 129, 191, 193, 255, 256, 257, 300, 511, 513, 700, 1025, 8191};
  for (int64_t n : sizes)
    for (int64_t rows : {int64_t(32), int64_t(128), int64_t(160), int64_t(256), int64_t(544), int64_t(2080), int64_t(8192)})
      for (int waves : {4, 2}) {
        wgrad(n, rows, waves * 64, waves, false);
        wgrad(n, rows, waves * 64, waves, true);
      }
  for (int64_t rows : counts)
    for (int64_t K : sizes)
      for (int64_t off : {int64_t(0), rows / 2, rows - 1}) {
        gemm(rows, K, off, rows - off, 256, 256);
        gemm(rows, K, off, rows - off, 128, 256);   // quadrants
      }
  for (int64_t N : sizes)
    for (int64_t K : sizes) {
      weights(N, K, 256, 2);
      weights(N, K, 128, 5);
    }
  return g_worst;
}

int main() {
  const int64_t now = worst(false);
  const int64_t made = g_reads;
  const int64_t loose = worst(true);
  printf("%lld reads, past a table's end: %lld bytes; with resources of the whole table %lld\n", static_cast<long long>(made),
         static_cast<long long>(now), static_cast<long long>(loose));
  if (made < 1000000 || now > 0 || loose <= 0) return 1;
  puts("fb_scale_reads ok");
  return 0;
}
