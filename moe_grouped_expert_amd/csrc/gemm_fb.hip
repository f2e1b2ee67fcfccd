// Grouped products of FP8 operands with one fp32 scale per block of 128, for groups of many rows:
//   C[r][n]   = sum over blocks b of sa[r][b] sw_e[n / 128][b] (sum over k in b of A[r][k] W_e[n][k])
//   dW_e[n][k] = sum over blocks b of sy[n][b] sx[k][b] (sum over the tokens t in b of dY[t][n] X[t][k])
// The matrix unit has no fp32 scales, so a block's 128 products are summed on it from zero
// (v_mfma_f32_16x16x128_f8f6f4, one instruction a block) and the vector unit adds the partial sum,
// scaled, to the fp32 accumulators: acc += d * s, 4 FMAs for each 32-cycle matrix instruction.
//
// The weights (for dW: X) are the matrix unit's row operand and the tokens (dY) its columns, so a
// lane's results are 4 consecutive columns of one row of C: its token scale is one register, the
// weight scale is the same in all lanes (dW has a scale a column of C too, a second multiply), and
// the results leave as 4 consecutive values.
//
// Tiles of 256 x 256, 8 waves, each 128 x 64 (8 x 4 blocks of 16 x 16, 128 accumulators: they have to
// be vector registers, which only half of the file is for one wave a SIMD, so two waves share one).
// Operands come HBM -> LDS directly in slices of 128 bytes, two stages of 64 KB.  The tokens' fragments
// of a slice (32 registers) are read first and the weights' streamed behind the matrix instructions, so
// the tokens' half of a stage and the first half of the weights' are free at mid-slice and refilled from
// there on (one and a half slices to arrive), the rest at the slice's end.  The next tile's first slices
// are issued before the epilogue (C) or with the last slices of the tile (dW).
//
// What bounds it, on MI355X: a slice of a CU takes 1.8 us (C; 2.4 PFLOP/s) and 1.9 - 2.1 us (dW), where the
// matrix unit needs 1.1 at the 1.7 - 1.9 GHz that the power leaves.  An f8 instruction holds the vector unit's
// port for 16 of its 32 cycles (its 16 operand registers), which leaves room for 4 additions; dW's second
// multiply makes a step 50 cycles.  Without the operands' arrival a slice takes 1.6 and 1.5 us, so a CU's
// intake (33 - 36 bytes a ns) is the rest.  A tile's start and epilogue, 600 vector instructions a wave, is 3 - 5 us.
// Measured: 8191 uneven rows over 8 x [4096][14336] 475 us (2.0 PFLOP/s), its weight gradient in bf16 620 us,
// the gate-up product with SwiGLU of 16384 rows over 8 x [28672][4096] 1.8 ms (2.1 PFLOP/s).
//
// C's tiles past the last whole round of the CUs run as quadrants of 128 x 128, whose 8 waves are two groups
// that take the slices in turn and add their sums at the end: 64 tiles left of 8191 rows take 100 us that way,
// one 256 x 256 tile more 200.
#include "gemm_impl.hpp"

#include "fp8b.hpp"

#include <algorithm>

namespace mge {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A kernel's tile: WN x WT waves of RB x TB blocks of 16 x 16 (weight rows x tokens), NST LDS stages.  KG groups of
// such waves take the slices in turn, each through stages of its own, and add their sums at the tile's end.
template <int WN_, int WT_, int RB_, int TB_, int NST_, int KG_>
struct FbTile {
  static constexpr int WN = WN_, WT = WT_, RB = RB_, TB = TB_, NST = NST_, KG = KG_;
  static constexpr int WAVES = WN * WT, THREADS = 64 * WAVES * KG;   // WAVES: of a group
  static constexpr int NR = WN * RB * 16, NT = WT * TB * 16;   // weight rows, tokens
  static constexpr int H = RB / 2;                             // a wave's blocks in each half of the weight rows
  static constexpr int OPT = NT * 128, OPW = NR * 128;         // bytes of the operands in a stage: tokens, then weights
  static constexpr int STAGE = OPT + OPW;
  static constexpr int SCALES = NST * STAGE;                   // then a ring of 2 NST slices' scales, 64 a wave:
  static constexpr int RING = WAVES * 256;                     // the tokens' (first waves), then the row operand's
  static constexpr int GROUP = SCALES + 2 * NST * RING, LDS = KG * GROUP;
  static constexpr int DT = NT / 8 / WAVES, DW = NR / 16 / WAVES;   // DMAs of a wave: tokens, each half of the weights
  static_assert((NST & (NST - 1)) == 0 && RB % 2 == 0 && NT % (8 * WAVES) == 0 && NR % (16 * WAVES) == 0, "whole DMAs");
  static_assert(NT / 64 + (NR + 63) / 64 <= WAVES && NT % 64 == 0, "64 scales a wave");
};
typedef FbTile<2, 4, 8, 4, 2, 1> FbMain;   // 256 x 256
typedef FbTile<2, 2, 4, 4, 2, 2> FbQuad;   // 128 x 128
typedef FbTile<2, 2, 4, 4, 2, 1> FbSmall;  // 128 x 128, two workgroups a CU (dW)

// Lanes 2j and 2j + 1 trade their b and a: the even lane then has its own a and the odd lane's a, the odd one
// the even lane's b and its own b.  Where a lane's a and b are neighbouring 16 bytes of its row of the output,
// stores of `a` then write the even lanes' rows and those of `b` the odd lanes', in twice as long runs.
__device__ __forceinline__ void pair_rows(u32x4& a, u32x4& b, bool odd) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t got = dpp_u<0xB1>(odd ? a[k] : b[k]);
    const uint32_t x = a[k];
    a[k] = odd ? got : x;
    b[k] = odd ? b[k] : got;
  }
}

// vm_barrier<A> where n > 0 (the same in every lane), else vm_barrier<B>.  The choice is made inside the asm: a
// branch of the compiler's would cut the K loop's body into blocks, across which it moves the additions.
template <int A, int B>
__device__ __forceinline__ void vm_barrier_if(int n) {
  asm volatile(
      "s_cmp_gt_i32 %0, 0\n\ts_cbranch_scc0 .Lfb_b%=\n\ts_waitcnt vmcnt(%1) lgkmcnt(0)\n\ts_branch .Lfb_m%=\n"
      ".Lfb_b%=:\n\ts_waitcnt vmcnt(%2) lgkmcnt(0)\n.Lfb_m%=:\n\ts_barrier" ::"s"(n), "n"(A), "n"(B)
      : "memory", "scc");
}

// 4 x 4 transpose over the lanes 16 apart: lane 16q + i gives v[j] for j = 0..3 and gets v[q] of the
// lanes 16p + i in v[p]
__device__ __forceinline__ void transpose4(uint32_t* v) {
  const U32Pair a = permlane32_swap(v[0], v[2]), b = permlane32_swap(v[1], v[3]);
  const U32Pair c = permlane16_swap(a.a, b.a), d = permlane16_swap(a.b, b.b);
  v[0] = c.a; v[1] = c.b; v[2] = d.a; v[3] = d.b;
}

// 4 bytes per lane from buffer offset voff + soff (soff the same in every lane) straight into LDS at
// lds_addr + 4 * lane
__device__ __forceinline__ void dma4(i32x4 rsrc, uint32_t lds_addr, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}

// 16 bytes per lane in the same way, at lds_addr + 16 * lane
__device__ __forceinline__ void dma16s(i32x4 rsrc, uint32_t lds_addr, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}

struct FtTile {
  int valid, e, off, m_valid, m0, n0, nkt, kbase, khi;
};

// What a tile's DMAs need beside offsets that all tiles share
struct FtOps {
  i32x4 rT, rW[2], rS;
  uint32_t toff[4];   // C (the rows of A may be gathered)
  uint32_t soff;      // TAIL
};

// KR: dW (FbWgrad), else C (FbGemm).  SW: the SwiGLU epilogue.  TAIL: the tiles past the main launch's last
// whole round, in quarters (their 128 x 128 quadrants).
template <typename TL, bool KR, bool SW, int OUT, bool TAIL, typename P>
__device__ __forceinline__ void fb_tile_body(const P& p) {
  constexpr int WN = TL::WN, RB = TL::RB, TB = TL::TB, H = TL::H, NST = TL::NST, KG = TL::KG;
  constexpr int HR = TL::NR / 2;               // weight rows of a half
  static_assert(!SW || HR == FB, "a block of h is a tile's columns");
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int32_t s_prefix[G_MAXE + 1];
  __shared__ int32_t s_mtiles[G_MAXE];
  __shared__ uint32_t s_amax[SW ? WN * TL::NT : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = KG == 1 ? uniform(tid >> 6) : uniform((tid >> 6) % TL::WAVES);   // of the group
  const int kg = KG == 1 ? 0 : uniform((tid >> 6) / TL::WAVES);
  uint8_t* const gmem = smem + kg * TL::GROUP;                                      // the group's stages
  const uint32_t lds_base = uniform(int(uint32_t(reinterpret_cast<uintptr_t>(gmem))));
  const int wn = wave % WN, wt = wave / WN;    // the wave's share of each half of the weight rows, its tokens
  // derived again from an opaque copy of the lane at the top of every tile and after its K loop, so
  // that one phase's addresses are not kept in registers through the other
  int i16 = lane & 15, q = lane >> 4;
  auto rederive_lane = [&]() {
    int v = lane;
    asm volatile("" : "+v"(v));
    i16 = v & 15;
    q = v >> 4;
  };

  // tiles of 256 x 256 for C whatever the kernel's own (SwiGLU: 128 columns of gate and of up, the kernel's tokens)
  constexpr int TM = SW || KR ? TL::NT : 256, TN = SW ? FB : (KR ? TL::NR : 256);
  int ncols = KR ? p.K : p.N;                              // columns of C
  if constexpr (SW) ncols = p.F;
  const int ntiles = (ncols + TN - 1) / TN;
  auto group_off = [&](int off) { return off < 0 ? 0 : (off > p.rows ? p.rows : off); };
  auto group_size = [&](int size, int off) { return size < 0 ? 0 : (size > p.rows - off ? p.rows - off : size); };
  if constexpr (!KR) {
    for (int e = tid; e < p.E; e += TL::THREADS)
      s_mtiles[e] = ((p.sizes ? group_size(p.sizes[e], group_off(p.offs[e])) : p.rows) + TM - 1) / TM;
    __syncthreads();
    if (tid == 0) {
      int acc = 0;
      for (int e = 0; e < p.E; ++e) {
        s_prefix[e] = acc;
        acc += s_mtiles[e] * ntiles;
      }
      s_prefix[p.E] = acc;
    }
    __syncthreads();
  }
  const int ymt = KR ? (p.N + TM - 1) / TM : 0;
  const int total = KR ? p.E * ymt * ntiles : uniform(s_prefix[p.E]);
  const int nwg = gridDim.x;
  int vid = blockIdx.x;
  if ((nwg & 7) == 0) vid = (blockIdx.x & 7) * (nwg >> 3) + (blockIdx.x >> 3);
  // The tiles past the main launch's last whole round run as quadrants where those are at most two a
  // workgroup; both launches decide from the same numbers.  (Without a main launch a round has no end.)
  int items = total, t_full = 0;
  if constexpr (!KR && !SW) {
    const int full = total / p.grid_main * p.grid_main, left = total - full;
    const bool split = 2 * left <= p.grid_main;
    t_full = uniform(full);
    items = uniform(TAIL ? (split ? 4 * left : 0) : (split ? full : total));
    if constexpr (TAIL) {
      // an equal run of the items for each XCD (further ones at nwg on)
      const int n = items < nwg ? items : nwg, run = (n + 7) >> 3;
      if ((nwg & 7) == 0) vid = int(blockIdx.x >> 3) < run ? int(blockIdx.x & 7) * run + int(blockIdx.x >> 3) : items;
    }
  }

  auto decode = [&](int item) {
    FtTile t{};
    t.valid = item < items;
    if (!t.valid) return t;
    const int tile = TAIL ? t_full + item / 4 : item;
    int local, mtn;
    if constexpr (KR) {
      t.e = tile / (ymt * ntiles);
      local = tile - t.e * ymt * ntiles;
      mtn = ymt;
    } else {
      int lo = 0, hi = p.E - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_prefix[mid] <= tile) lo = mid; else hi = mid - 1;
      }
      t.e = uniform(lo);
      local = tile - uniform(s_prefix[t.e]);
      mtn = uniform(s_mtiles[t.e]);
    }
    // bands of 8 token tiles, walked across the columns, tokens fastest (as in the MX kernels)
    const int nband = (mtn + 7) / 8;
    const int band = min(local / (8 * ntiles), nband - 1);
    const int within = local - band * 8 * ntiles;
    const int gm = band == nband - 1 ? mtn - band * 8 : 8;
    t.m0 = (band * 8 + within % gm) * TM;
    t.n0 = (within / gm) * TN;
    if constexpr (TAIL) {
      t.m0 += (item & 2) ? 128 : 0;
      t.n0 += (item & 1) ? 128 : 0;
    }
    t.off = p.sizes ? uniform(group_off(ld_uniform(p.offs, t.e))) : 0;
    const int size = p.sizes ? uniform(group_size(ld_uniform(p.sizes, t.e), t.off)) : p.rows;
    if constexpr (KR) {
      // the group's tokens; its last 32 may hold padding, which is zero
      const int span = group_size((size + 31) / 32 * 32, t.off);
      t.m_valid = p.N;
      t.kbase = t.off & ~127;
      t.khi = t.off + span;
      t.nkt = size > 0 ? (t.khi - t.kbase + 127) / 128 : 0;
    } else {
      t.m_valid = size;
      t.khi = p.K;
      t.nkt = TAIL && (t.m0 >= size || t.n0 >= ncols) ? 0 : (p.K + 127) / 128;   // (a quadrant of nothing)
    }
    return t;
  };

  // LDS rows of a DMA instruction: 8, lane l row l / 8, chunk l % 8; the lane loads the chunk that the
  // swizzle puts there: (l % 8) ^ (l / 16), that ^ 4 in odd instructions
  const int lchunk = ((lane & 7) ^ (lane >> 4)) * 16;
  const uint32_t ldw = KR ? uint32_t(p.rows) : uint32_t(p.K);   // bytes of an operand row
  const int KB = KR ? 0 : (p.K + 127) / 128;
  constexpr int DT = TL::DT, DW = TL::DW;
  static_assert(DT <= 4 && DW <= 2, "offsets of a lane");
  constexpr int SWV = TL::NT / 64;             // the first wave that brings the row operand's scales

  const bool of_t = wave < SWV;                // (the wave brings the tokens' scales)
  bool direct = false;                         // C's quadrants without a main launch read the tokens' scales as they come
  if constexpr (TAIL) direct = p.Ast == nullptr;

  // Rows of A of the lane's DMAs (TAIL: and of its scale)
  auto rows_of = [&](const FtTile& t, int* src) {
    if constexpr (TAIL) {
      const int m = t.m0 + wave * 64 + lane;
      src[DT] = direct && of_t && t.valid && m < t.m_valid ? t.off + m : -1;
      if (src[DT] >= 0 && p.map) src[DT] = p.map[src[DT]];
    }
#pragma unroll
    for (int i = 0; i < DT; ++i) {
      const int m = t.m0 + wave * (DT * 8) + i * 8 + (lane >> 3);
      src[i] = t.valid && m < t.m_valid ? t.off + m : -1;
      if constexpr (!KR) {
        if (src[i] >= 0 && p.map) src[i] = p.map[src[i]];
      }
    }
  };
  // The lane's offsets hold its row and chunk, the slice's place in K is the same in all lanes.
  uint32_t krow[4], woff[2];
#pragma unroll
  for (int i = 0; i < DT; ++i) krow[i] = uint32_t(wave * (DT * 8) + i * 8 + (lane >> 3)) * ldw + (lchunk ^ ((i & 1) * 64));   // (dW: rows of dY)
  woff[0] = uint32_t(wave * (DW * 8) + (lane >> 3)) * ldw + uint32_t(lchunk);
  woff[1] = uint32_t(wave * (DW * 8) + 8 + (lane >> 3)) * ldw + uint32_t(lchunk ^ 64);
  // Scales: the tokens' (dW: of dY), 64 a wave; in the other waves for dW those of X, for C in the first lanes those of
  // the weights, of the tile's halves or with SwiGLU of the gate rows and of every 32 up rows.  (Lanes past the rows or
  // the group read other rows' scales or zeros; what they scale is zero or not stored.)
  uint32_t s_ld, soff = uint32_t(lane) * 4;   // bytes of a slice; the lane's
  constexpr bool ROWS = KR && TL::NR < 256;    // dW's small tiles: the scales as they come, a line a row
  if constexpr (ROWS) {
    s_ld = 4;
    soff *= uint32_t((p.rows + 127) / 128);
  } else if constexpr (KR) {
    s_ld = uint32_t(of_t ? p.N : p.K) * 4;
  } else {
    s_ld = of_t && !direct ? uint32_t(p.ast_ld) * 4 : 4u;
    const int blk = SW ? (lane == 0 ? 0 : (p.F + (lane - 1) * 32) / FB) : lane * HR / FB;
    if (!of_t) soff = lane < (SW ? 5 : 2) ? uint32_t(blk * KB) * 4 : kInvalid;
  }
  auto setup = [&](const FtTile& t, const int* src) {
    FtOps o;
    auto left = [](int n, int cap) { return n < 0 ? 0 : (n > cap ? cap : n); };
    if constexpr (KR) {
      o.rT = make_rsrc_n(p.Y + int64_t(t.m0) * p.rows, uint32_t(left(p.N - t.m0, TL::NT)) * ldw);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        o.rW[h] = make_rsrc_n(p.X + int64_t(t.n0 + HR * h) * p.rows, uint32_t(left(p.K - t.n0 - HR * h, HR)) * ldw);
      const FbSpan sp = fb_scale_span(of_t ? t.m0 + wave * 64 : t.n0 + (wave - SWV) * 64, of_t ? p.N : p.K, t.kbase / 128, (p.rows + 127) / 128, ROWS);
      o.rS = make_rsrc_n((ROWS ? (of_t ? p.Ys : p.Xs) : (of_t ? p.Yst : p.Xst)) + sp.at, sp.bytes);
    } else {
      o.rT = make_rsrc_n(p.A, uint32_t(p.src_rows) * ldw);
#pragma unroll
      for (int i = 0; i < DT; ++i)
        o.toff[i] = src[i] >= 0 && src[i] < p.src_rows ? uint32_t(src[i]) * ldw + (lchunk ^ ((i & 1) * 64)) : kInvalid;
      const uint8_t* w = p.W ? ld_uniform(p.W, t.e) : p.Wv[t.e];
      const float* ws = p.W ? ld_uniform(p.Ws, t.e) : p.Wsv[t.e];
      const int nrows = SW ? ncols : p.N;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r0 = SW ? t.n0 : t.n0 + HR * h;          // (SwiGLU: gate, then up rows of the same columns)
        o.rW[h] = make_rsrc_n(w + (int64_t(r0) + (SW ? h * ncols : 0)) * p.K, uint32_t(left(nrows - r0, HR)) * ldw);
      }
      const FbSpan sp = of_t ? fb_scale_span(int64_t(t.off) + t.m0 + wave * 64, p.ast_ld, 0, KB, false)
                             : fb_scale_span(t.n0 / FB, ((SW ? 2 * ncols : p.N) + FB - 1) / FB, 0, KB, true);
      o.rS = make_rsrc_n((of_t ? p.Ast : ws) + sp.at, sp.bytes);
      o.soff = soff;
      if constexpr (TAIL) {
        if (direct && of_t) {
          o.rS = make_rsrc_n(p.As, uint32_t(p.src_rows) * uint32_t(KB) * 4);
          o.soff = src[DT] >= 0 && src[DT] < p.src_rows ? uint32_t(src[DT]) * uint32_t(KB) * 4 : kInvalid;
        }
      }
    }
    return o;
  };
  // (a wave's first LDS row is a multiple of 16, so that its even and odd instructions are those of the swizzle)
  static_assert(DT % 2 == 0 && DW % 2 == 0, "even instructions start at even groups of 8 rows");
  // (from here on kt counts the group's own slices: slice KG kt + kg of the tile)
  auto at_slice = [&](i32x4 r, const FtTile& t, int kt) {
    r[2] = KG * kt + kg < t.nkt ? r[2] : 0;
    return r;
  };
  // (no offset beside a resource without records, so that no form of the range check takes one from the other)
  auto place = [](const i32x4& r, uint32_t k) { return r[2] != 0 ? k : 0u; };
  // A slice past the last has a resource without records; in the last one, where it is not a whole 128 bytes, the
  // chunks past its end get the top bit.  Both read zeros.
  auto off_at = [&](const FtTile& t, uint32_t off, int kt, int odd) {
    const int tail = (t.khi - t.kbase) & 127;      // bytes of the last slice, 0: whole
    const int end = tail != 0 && KG * kt + kg == t.nkt - 1 ? tail : 128;
    return (lchunk ^ (odd * 64)) < end ? off : kInvalid;
  };
  // AHEAD: the last NST slices of a tile bring the first NST of the next one, so that operands arrive without a
  // pause; the stages are taken in turn over all tiles (gd: slices before those of the tile that is brought in).
  constexpr bool AHEAD = KR && KG == 1;
  int gd = 0;
  auto dma_t = [&](const FtOps& o, const FtTile& t, int kt, int i) {
    const i32x4 r = at_slice(o.rT, t, kt);
    dma16s(r, lds_base + ((gd + kt) & (NST - 1)) * TL::STAGE + (wave * (DT * 8) + i * 8) * 128, off_at(t, KR ? krow[i] : o.toff[i], kt, i & 1),
           place(r, uint32_t(t.kbase + (KG * kt + kg) * 128)));
  };
  auto dma_w = [&](const FtOps& o, const FtTile& t, int kt, int h, int i) {
    const i32x4 r = at_slice(o.rW[h], t, kt);
    dma16s(r, lds_base + ((gd + kt) & (NST - 1)) * TL::STAGE + TL::OPT + (h * HR + wave * (DW * 8) + i * 8) * 128,
           off_at(t, woff[i], kt, i), place(r, uint32_t(t.kbase + (KG * kt + kg) * 128)));
  };
  auto dma_s = [&](const FtOps& o, const FtTile& t, int kt) {
    const i32x4 r = at_slice(o.rS, t, kt);
    dma4(r, lds_base + TL::SCALES + ((gd + kt) & (2 * NST - 1)) * TL::RING + wave * 256, TAIL ? o.soff : soff, place(r, uint32_t(KG * kt + kg) * s_ld));
  };
  // The early part of a slice (its tokens, scales and the first half of the weight rows) and the late one
  constexpr int EARLY = 1 + DT + DW, LATE = DW;
  auto issue_late = [&](const FtOps& o, const FtTile& t, int kt) {
#pragma unroll
    for (int i = 0; i < DW; ++i) dma_w(o, t, kt, 1, i);
  };
  auto issue_early = [&](const FtOps& o, const FtTile& t, int kt) {
    dma_s(o, t, kt);
#pragma unroll
    for (int i = 0; i < DT; ++i) dma_t(o, t, kt, i);
#pragma unroll
    for (int i = 0; i < DW; ++i) dma_w(o, t, kt, 0, i);
  };
  auto prologue = [&](const FtOps& o, const FtTile& t) {
#pragma unroll
    for (int k = 0; k < NST; ++k) {
      issue_early(o, t, k);
      issue_late(o, t, k);
    }
  };
  // Stores that every wave's epilogue issues at least: the next tile's first DMAs are issued before
  // them, and its first waits leave them in flight
  constexpr int STORES = OUT == OUT_BF16 ? TB * 2 * 2 : (OUT == OUT_F32 ? TB * RB : (SW ? TB : 0));
  static_assert(NST * (EARLY + LATE) + STORES < 64, "vmcnt");

  FtTile t = decode(vid);
  FtOps o{};
  int stores = 0;   // 1: the wave has stores in flight that are newer than this tile's first DMAs
  bool ahead = false;   // the tile's first slices came with the tile before
  int src[DT + (TAIL ? 1 : 0)];
  rows_of(t, src);
  if (t.valid) {
    o = setup(t, src);
    if (t.nkt > 0) prologue(o, t);
  }
  for (int item = vid; item < items; item += nwg) {
    rederive_lane();
    // loads whose latency the K loop hides: the next tile's rows, the probabilities of this one's
    const FtTile nxt = decode(item + nwg);
    rows_of(nxt, src);
    float pr[TB];
    if constexpr (SW) {
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
        const int m = t.m0 + wt * (TB * 16) + tb * 16 + i16;
        pr[tb] = p.prob == nullptr ? 1.f : (m < t.m_valid ? p.prob[int64_t(t.off) + m] : 0.f);
      }
    }
    const int tread = (wt * (TB * 16) + i16) * 128 + ((q ^ ((i16 >> 1) & 7)) << 4);
    const int wread = (wn * (H * 16) + i16) * 128 + ((q ^ ((i16 >> 1) & 7)) << 4);
    f32x4 acc[RB][TB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) acc[rb][tb] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (t.nkt > 0) {
      // ---- K loop.  Step rb of a slice multiplies weight block rb by the token blocks, adds the partial
      // sums of the step before (so that no addition waits for its matrix instruction) and reads the next
      // weight block; the last step also reads the next slice's tokens, each as soon as its last product is
      // issued, so that the matrix unit runs on across slices.  Two barriers a slice, at each of which one
      // part of the stage has been read by every wave and is filled again with slice kt + NST, and the part
      // read next, issued NST - 1/2 slices ago, is resident:
      //   before step H - 1 (which reads the late part)   the early part is free
      //   before the last step (which reads the early part of kt + 1)   the late part is free
      constexpr int BP = H - 1, BQ = RB - 1;
      constexpr int FLY = (NST - 1) * (EARLY + LATE);   // DMAs newer than the part waited for, at both
      // the early part of slice 0 is resident (ahead: since the last barrier of the tile before)
      if (!AHEAD || !ahead) vm_barrier_if<FLY + LATE + STORES, FLY + LATE>(stores);
      const int g0 = gd;
      // (the two chunks of a fragment are 64 bytes apart in the row, either way round: a base each, so that the
      // rows' distances fit the instructions' offsets)
      auto frag = [&](const uint8_t* p0, const uint8_t* p1, int at) {
        const uint4 a = *reinterpret_cast<const uint4*>(p0 + at);
        const uint4 b = *reinterpret_cast<const uint4*>(p1 + at);
        return i32x8{int(a.x), int(a.y), int(a.z), int(a.w), int(b.x), int(b.y), int(b.z), int(b.w)};
      };
      auto scales_of = [&](int kt) { return reinterpret_cast<const float*>(gmem + TL::SCALES + ((g0 + kt) & (2 * NST - 1)) * TL::RING); };
      constexpr int RS = SWV * 64;        // the row operand's scales in a slice's ring entry
      const int s0 = (g0 & (NST - 1)) * TL::STAGE;
      i32x8 tf[TB], wf[2];
      float ts[TB], tn[TB], sc[TB];       // token scales, those of the next slice, times the weights'
      float ws = 0.f;
      f32x4 d[2][TB], xs[2];
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
        tf[tb] = frag(gmem + s0 + tread, gmem + s0 + (tread ^ 64), tb * 2048);
        tn[tb] = scales_of(0)[wt * (TB * 16) + tb * 16 + i16];
        ts[tb] = sc[tb] = 0.f;
        d[1][tb] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      xs[1] = f32x4{0.f, 0.f, 0.f, 0.f};
      wf[0] = frag(gmem + s0 + wread, gmem + s0 + (wread ^ 64), TL::OPT);
      // (AHEAD: at least NST slices, those past the end are zeros)
      const int nit = AHEAD ? max(t.nkt, NST) : (t.nkt + KG - 1) / KG;
      int fresh = stores ? NST : 0;       // slices whose parts are older than the stores
      FtTile in = t;                      // the tile that is brought in, and its slice beside slice kt: kt + di
      int kt = 0, di = NST;
#pragma clang loop unroll(disable)
      for (int end = AHEAD ? nit - NST : nit;; end = nit) {
#pragma clang loop unroll(disable)
      for (; kt < end; ++kt) {
        const int st = ((g0 + kt) & (NST - 1)) * TL::STAGE, sn = ((g0 + kt + 1) & (NST - 1)) * TL::STAGE;   // this slice's stage, the next one's
        const uint8_t *w0 = gmem + st + wread, *w1 = gmem + st + (wread ^ 64);
        const float* sS = scales_of(kt) + RS;
        static_for<0, RB>([&](auto rbc) {
          constexpr int rb = decltype(rbc)::value;
          constexpr int pb = (rb + RB - 1) % RB;   // the block whose sums are added
          if constexpr (rb == BP) {
            vm_barrier_if<FLY + STORES, FLY>(fresh);
            dma_s(o, in, kt + di);
          }
          if constexpr (rb == BQ) {
            --fresh;
            vm_barrier_if<FLY + STORES, FLY>(fresh);
          }
          if constexpr (rb < RB - 1) wf[(rb + 1) & 1] = frag(w0, w1, TL::OPT + (rb + 1 < H ? (rb + 1) * 2048 : HR * 128 + (rb + 1 - H) * 2048));
          else wf[0] = frag(gmem + sn + wread, gmem + sn + (wread ^ 64), TL::OPT);
          if constexpr (KR) xs[rb & 1] = *reinterpret_cast<const f32x4*>(sS + (rb < H ? 0 : HR) + wn * (H * 16) + (rb % H) * 16 + 4 * q);
          if constexpr (KR && rb == 1) {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) ts[tb] = tn[tb];
          }
          // the scales of the sums that this step adds (SwiGLU: an up half's rows are in one or two scales' rows), the
          // weights' read a step before
          constexpr auto fresh_scale = [](int b) { return b == 1 || b == H + 1 || (SW && b > H && (b - 1 - H) * 16 % 32 == 0); };
          if constexpr (!KR && fresh_scale(rb)) {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
              if constexpr (rb == 1) ts[tb] = tn[tb];
              sc[tb] = ts[tb] * ws;
            }
          }
          if constexpr (!KR && fresh_scale(rb + 1)) ws = sS[rb == 0 ? 0 : (SW ? 1 + (wn * H + rb - H) / 2 : 1)];
          __builtin_amdgcn_sched_barrier(0);
          static_for<0, TB>([&](auto tbc) {
            constexpr int tb = decltype(tbc)::value;
            const f32x4 z = {0.f, 0.f, 0.f, 0.f};
            d[rb & 1][tb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[rb & 1], tf[tb], z, 0, 0, 0, 0, 0, 0);
            if constexpr (rb == RB - 1) {
              tf[tb] = frag(gmem + sn + tread, gmem + sn + (tread ^ 64), tb * 2048);
              tn[tb] = scales_of(kt + 1)[wt * (TB * 16) + tb * 16 + i16];
            }
            // the parts of kt + NST, at most one DMA a matrix instruction
            if constexpr (rb >= BP && rb < BQ) {
              constexpr int n = (BQ - BP) * TB, i = (rb - BP) * TB + tb, k0 = (DT + DW) * i / n, k1 = (DT + DW) * (i + 1) / n;
              if constexpr (k1 > k0) {
                if constexpr (k0 < DT) dma_t(o, in, kt + di, k0);
                else dma_w(o, in, kt + di, 0, k0 - DT);
              }
            }
            if constexpr (rb == BQ && tb < DW) dma_w(o, in, kt + di, 1, tb);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if constexpr (KR) acc[pb][tb][r] = fmaf(d[(rb + 1) & 1][tb][r] * ts[tb], xs[(rb + 1) & 1][r], acc[pb][tb][r]);
              else acc[pb][tb][r] = fmaf(d[(rb + 1) & 1][tb][r], sc[tb], acc[pb][tb][r]);
            }
            __builtin_amdgcn_sched_barrier(0);
          });
          static_assert((BQ - BP) * TB >= DT + DW && TB >= DW, "a part is issued before the next barrier");
        });
      }
        if (end == nit) break;
        o = setup(nxt, src);
        in = nxt;
        gd = g0 + nit;
        di = NST - nit;
      }
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (KR) acc[RB - 1][tb][r] = fmaf(d[1][tb][r] * ts[tb], xs[1][r], acc[RB - 1][tb][r]);
          else acc[RB - 1][tb][r] = fmaf(d[1][tb][r], sc[tb], acc[RB - 1][tb][r]);
        }
    }
    const FtTile cur = t;
    t = nxt;
    ahead = AHEAD && cur.nkt > 0 && t.nkt > 0;
    if (!ahead) {
      __builtin_amdgcn_s_waitcnt(0);    // the slices past the end (zeros) have landed
      if (t.valid) o = setup(t, src);
      lds_barrier();                    // every wave is done with the stages
    }
    if constexpr (KG > 1) {
      // the second group's sums through LDS (16 bytes a lane and block, whole wave after wave)
      static_assert(KG == 2 && TL::WAVES * 64 * RB * TB * 16 <= TL::LDS, "sums of a group");
      f32x4* sum = reinterpret_cast<f32x4*>(smem) + wave * (RB * TB * 64) + lane;
      if (kg == 1) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
          for (int tb = 0; tb < TB; ++tb) sum[(rb * TB + tb) * 64] = acc[rb][tb];
      }
      lds_barrier();
      if (kg == 0) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
          for (int tb = 0; tb < TB; ++tb) acc[rb][tb] += sum[(rb * TB + tb) * 64];
      }
      lds_barrier();
    }
    if (!ahead && t.valid && t.nkt > 0) prologue(o, t);
    if (KG > 1 && kg > 0) continue;     // (no stores)
    stores = STORES > 0 ? 1 : 0;
    rederive_lane();

    // ---- epilogues.  acc[rb][tb][r]: column n0 + (rb < H ? 0 : HR) + wn * 16 H + (rb % H) * 16 + 4q + r,
    // token m0 + wt * 16 TB + tb * 16 + i16.  Stores go through resources that end at the last valid row.
    const int wrow0 = cur.m0 + wt * (TB * 16);
    int vr = cur.m_valid - wrow0;
    vr = uniform(vr < 0 ? 0 : (vr > TB * 16 ? TB * 16 : vr));
    if constexpr (!SW) {
      constexpr int ESZ = OUT == OUT_BF16 ? 2 : 4;
      uint8_t* base;
      if constexpr (KR) base = static_cast<uint8_t*>(p.D ? ld_uniform(p.D, cur.e) : p.Dv[cur.e]) + int64_t(wrow0) * ncols * ESZ;
      else base = static_cast<uint8_t*>(p.C) + (int64_t(cur.off) + wrow0) * ncols * ESZ;
      const uint32_t rowb = uint32_t(ncols) * ESZ;
      const __amdgpu_buffer_rsrc_t rC = __builtin_amdgcn_make_buffer_rsrc(base, 0, int(uint32_t(vr) * rowb), kRsrcFlags);
      // whole lines of 128 bytes: lanes 2j and 2j + 1 store row 2j, then row 2j + 1, 16 bytes each
      constexpr int pol = KR ? kNonTemporal : 0;   // gradients: written once, read by no workgroup
      const bool odd = (i16 & 1) != 0;
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
        const uint32_t row = uint32_t(tb * 16 + (i16 & ~1)) * rowb;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c0 = cur.n0 + h * HR + wn * (H * 16);
          if constexpr (OUT == OUT_BF16) {
            static_assert(H == 4 || H == 2, "blocks of a half");
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f32x4 v = acc[H * h + j % H][tb];
              lo[j] = bf16x2(v[0], v[1]);
              hi[j] = bf16x2(v[2], v[3]);
            }
            transpose4(lo);
            transpose4(hi);
            // the lane has columns c .. c + 15 of block q now (two blocks: q and q + 2 have the same one,
            // and the lanes q >= 2 store nothing)
            u32x4 a = {lo[0], hi[0], lo[1], hi[1]}, b = {lo[2], hi[2], lo[3], hi[3]};
            pair_rows(a, b, odd);
            const int c = c0 + q * 16;
            const uint32_t off = c < ncols && q < H ? row + uint32_t(c) * ESZ + (odd ? 16 : 0) : kInvalid;
            __builtin_amdgcn_raw_buffer_store_b128(a, rC, int(off), 0, pol);
            __builtin_amdgcn_raw_buffer_store_b128(b, rC, int(off + rowb), 0, pol);
          } else {
#pragma unroll
            for (int j = 0; j < H; j += 2) {
              u32x4 a = __builtin_bit_cast(u32x4, acc[H * h + j][tb]), b = __builtin_bit_cast(u32x4, acc[H * h + j + 1][tb]);
              pair_rows(a, b, odd);
              const int c = c0 + (j + (odd ? 1 : 0)) * 16 + 4 * q;
              const uint32_t off = c < ncols ? row + uint32_t(c) * ESZ : kInvalid;
              if constexpr (OUT == OUT_F32_ACC) {
                const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(rC, int(off), 0, pol);
                const u32x4 y = __builtin_amdgcn_raw_buffer_load_b128(rC, int(off + rowb), 0, pol);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  a[r] = __float_as_uint(__uint_as_float(a[r]) + __uint_as_float(x[r]));
                  b[r] = __float_as_uint(__uint_as_float(b[r]) + __uint_as_float(y[r]));
                }
              }
              __builtin_amdgcn_raw_buffer_store_b128(a, rC, int(off), 0, pol);
              __builtin_amdgcn_raw_buffer_store_b128(b, rC, int(off + rowb), 0, pol);
            }
          }
        }
      }
    } else {
      // h = p silu(G) U of the tile's 128 columns, one block of 128 a token: its largest magnitude over
      // the lane's columns, the lanes 16 apart and the waves that share the tokens
      const int64_t grow0 = int64_t(cur.off) + wrow0;
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
        uint32_t am = 0;
#pragma unroll
        for (int j = 0; j < H; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float G = acc[j][tb][r], U = acc[H + j][tb][r];
            const float h = pr[tb] * (G * __builtin_amdgcn_rcpf(1.f + __expf(-G))) * U;
            acc[j][tb][r] = h;
            am = umax(am, __float_as_uint(h) & 0x7fffffffu);
          }
        const U32Pair a = permlane16_swap(am, am);
        am = umax(a.a, a.b);
        const U32Pair b = permlane32_swap(am, am);
        am = umax(b.a, b.b);
        if (q == 0) s_amax[wn * TL::NT + wt * (TB * 16) + tb * 16 + i16] = am;
      }
      lds_barrier();
      const __amdgpu_buffer_rsrc_t rH =
          __builtin_amdgcn_make_buffer_rsrc(p.h_codes + grow0 * p.F, 0, int(uint32_t(vr) * uint32_t(p.F)), kRsrcFlags);
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
        const int m = wt * (TB * 16) + tb * 16 + i16;
        uint32_t am = s_amax[m];
#pragma unroll
        for (int w = 1; w < WN; ++w) am = umax(am, s_amax[w * TL::NT + m]);
        const FbScale sc = fb_scale(am);
        const int c0 = cur.n0 + wn * (H * 16);
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 x = acc[j % H][tb];
          v[j] = fb_codes4(x[0] * sc.inv, x[1] * sc.inv, x[2] * sc.inv, x[3] * sc.inv);
        }
        transpose4(v);
        const int c = c0 + (q % H) * 16;
        const uint32_t off = c < p.F && q < H ? uint32_t(tb * 16 + i16) * uint32_t(p.F) + uint32_t(c) : kInvalid;
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{v[0], v[1], v[2], v[3]}, rH, int(off), 0, 0);
        if (wn == 0 && q == 0 && tb * 16 + i16 < vr) p.h_scales[int64_t(cur.n0 / FB) * p.ast_ld + grow0 + tb * 16 + i16] = sc.s;
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(0);   // no LDS DMA outlives the workgroup
}

#define FB_KERNEL(name, TL, PER_SIMD, KR, SW, OUT, TAIL, P) \
  __global__ __launch_bounds__(TL::THREADS, PER_SIMD) void name(P p) { fb_tile_body<TL, KR, SW, OUT, TAIL>(p); }
FB_KERNEL(gemm_fb_store, FbMain, 2, false, false, OUT_BF16, false, FbGemm)
FB_KERNEL(gemm_fb_store_f32, FbMain, 2, false, false, OUT_F32, false, FbGemm)
FB_KERNEL(gemm_fb_store_tail, FbQuad, 2, false, false, OUT_BF16, true, FbGemm)
FB_KERNEL(gemm_fb_store_f32_tail, FbQuad, 2, false, false, OUT_F32, true, FbGemm)
FB_KERNEL(gemm_fb_swiglu, FbMain, 2, false, true, OUT_NONE, false, FbGemm)
FB_KERNEL(gemm_fb_wgrad, FbMain, 2, true, false, OUT_BF16, false, FbWgrad)
FB_KERNEL(gemm_fb_wgrad_f32, FbMain, 2, true, false, OUT_F32, false, FbWgrad)
FB_KERNEL(gemm_fb_wgrad_f32_acc, FbMain, 2, true, false, OUT_F32_ACC, false, FbWgrad)
FB_KERNEL(gemm_fb_wgrad_small, FbSmall, 2, true, false, OUT_BF16, false, FbWgrad)
FB_KERNEL(gemm_fb_wgrad_f32_small, FbSmall, 2, true, false, OUT_F32, false, FbWgrad)
FB_KERNEL(gemm_fb_wgrad_f32_acc_small, FbSmall, 2, true, false, OUT_F32_ACC, false, FbWgrad)
#undef FB_KERNEL

// A persistent launch of at most `grid` workgroups
template <typename TL, typename Kern, typename P>
static mge_status launch_fb(Kern kern, const char* name, const P& p, int64_t grid, hipStream_t s) {
  hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, TL::LDS);
  if (grid <= 0) return MGE_OK;
  ProfScope prof(s, name);
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(TL::THREADS), TL::LDS, s, p);
  return hip_check(name);
}

static int64_t fb_token_tiles(const FbGemm& p) { return (int64_t(p.total) + 255) / 256 + (p.sizes ? p.E : 0); }
// With tiles for half a round at most, were the groups even, all tiles are the tail's, however many there are; it takes
// the tokens' scales in either form, which saves the launch that makes them block-major
bool fb_tail_only(int64_t E, int64_t N, int64_t total) {
  const int64_t groups = std::max<int64_t>(1, std::min(E, total)), each = (total + groups - 1) / groups;
  return 2 * groups * ((each + 255) / 256) * ((N + 255) / 256) <= 256;   // (CUs of a whole chip: workspaces go by it)
}
mge_status launch_fb_tile(const FbGemm& p0, bool swiglu, hipStream_t s) {
  FbGemm p = p0;
  const int64_t mt = fb_token_tiles(p);
  const int cus = device_cus();
  if (swiglu) return launch_fb<FbMain>(gemm_fb_swiglu, "gemm_fp8_block_swiglu", p, std::min<int64_t>(cus, mt * ((p.F + 127) / 128)), s);
  const int64_t tiles = mt * ((p.N + 255) / 256);
  const bool only = fb_tail_only(p.E, p.N, p.total);
  p.grid_main = only ? 1 << 30 : cus;
  mge_status st = MGE_OK;
  if (!only) {
    const int64_t grid = std::min<int64_t>(cus, tiles);
    st = p.out_f32 ? launch_fb<FbMain>(gemm_fb_store_f32, "gemm_fp8_block", p, grid, s)
                   : launch_fb<FbMain>(gemm_fb_store, "gemm_fp8_block", p, grid, s);
    if (st != MGE_OK) return st;
  }
  const int64_t tail = std::min<int64_t>(cus, 4 * tiles);
  return p.out_f32 ? launch_fb<FbQuad>(gemm_fb_store_f32_tail, "gemm_fp8_block_tail", p, tail, s)
                   : launch_fb<FbQuad>(gemm_fb_store_tail, "gemm_fp8_block_tail", p, tail, s);
}

// dW's tiles: 256 x 256, or 128 x 128 with two workgroups a CU, which take in twice the bytes, but fill the CUs with
// few tiles, overlap one's epilogue with the other's slices and read the scales as they come (the pass that makes them
// block-major is a launch of its own).  By estimates of the time in us from what both measured on MI355X (bf16, 256 and
// 128; slices: an expert's tokens / 128): 8 x [1024][1024], 1 slice 16.4, 9.6, 8 26.9, 17.5, 32 66, 49; [4096][4096], 3
// slices 21.9, 17.8, 8 31.9, 28.5, 32 78, 94; 8 x [2048][2048], 1 slice 27.9, 25.1, 8 52, 56; 8 x [4096][14336] (scales
// block-major for both), 1 slice 219, 293, 8 556, 709.
bool fb_wgrad_small(const FbWgrad& p) {
  const int64_t cus = device_cus();
  const double slices = std::max(1.0, double(p.rows) / 128 / p.E);
  auto rounds = [&](int n, int64_t per) { return double((int64_t(p.E) * ((p.N + n - 1) / n) * ((p.K + n - 1) / n) + per - 1) / per); };
  return 5 + rounds(128, 2 * cus) * (3 + 1.3 * slices) < 11 + rounds(256, cus) * (5.5 + 1.85 * slices);
}
template <typename TL, typename Kern>
static mge_status launch_wgrad(Kern kern, int per_cu, const FbWgrad& p, hipStream_t s) {
  const int64_t tiles = int64_t(p.E) * ((p.N + TL::NT - 1) / TL::NT) * ((p.K + TL::NR - 1) / TL::NR);
  return launch_fb<TL>(kern, "wgrad_fp8_block", p, std::min<int64_t>(int64_t(per_cu) * device_cus(), tiles), s);
}
mge_status launch_fb_wgrad(const FbWgrad& p, hipStream_t s) {
  if (fb_wgrad_small(p)) {
    if (p.out == OUT_BF16) return launch_wgrad<FbSmall>(gemm_fb_wgrad_small, 2, p, s);
    if (p.out == OUT_F32) return launch_wgrad<FbSmall>(gemm_fb_wgrad_f32_small, 2, p, s);
    return launch_wgrad<FbSmall>(gemm_fb_wgrad_f32_acc_small, 2, p, s);
  }
  if (p.out == OUT_BF16) return launch_wgrad<FbMain>(gemm_fb_wgrad, 1, p, s);
  if (p.out == OUT_F32) return launch_wgrad<FbMain>(gemm_fb_wgrad_f32, 1, p, s);
  return launch_wgrad<FbMain>(gemm_fb_wgrad_f32_acc, 1, p, s);
}

// Scales made block-major, 64 x 64 a workgroup through LDS; every matrix of the launch has its own range of workgroups
struct FbScaleTArgs {
  FbScaleT m[2];
  int64_t first[2];
  int n;
};
__global__ __launch_bounds__(256) void fb_scale_t_kernel(FbScaleTArgs a) {
  __shared__ float tile[64][65];
  const int which = a.n > 1 && int64_t(blockIdx.x) >= a.first[1] ? 1 : 0;
  const FbScaleT& m = a.m[which];
  const int nj = (m.kb + 63) / 64;
  const int64_t blk = int64_t(blockIdx.x) - a.first[which];
  const int64_t r0 = blk / nj * 64;
  const int j0 = int(blk % nj) * 64;
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  // (all 16 loads of a thread in flight, the map's first)
  int64_t src[16];
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t r = r0 + 4 * i + y;
    src[i] = r >= m.rows ? -1 : (m.map ? int64_t(m.map[r]) : r);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = src[i] >= 0 && src[i] < m.src_rows && j0 + x < m.kb ? m.in[src[i] * m.kb + j0 + x] : 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) tile[4 * i + y][x] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = y; i < 64; i += 4)
    if (j0 + i < m.kb && r0 + x < m.rows) m.out[int64_t(j0 + i) * m.ld + r0 + x] = tile[x][i];
}
mge_status launch_fb_scale_t(const FbScaleT* list, int n, hipStream_t s) {
  FbScaleTArgs a{};
  int64_t blocks = 0;
  for (int i = 0; i < n; ++i) {
    a.m[i] = list[i];
    a.first[i] = blocks;
    blocks += (list[i].rows + 63) / 64 * ((list[i].kb + 63) / 64);
  }
  a.n = n;
  if (blocks == 0) return MGE_OK;
  ProfScope prof(s, "fp8_block_scales");
  hipLaunchKernelGGL(fb_scale_t_kernel, dim3(unsigned(blocks)), dim3(256), 0, s, a);
  return hip_check("fp8_block_scales");
}

}  // namespace mge
