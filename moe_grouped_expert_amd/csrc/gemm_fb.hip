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
// there on (one and a half slices to arrive), the rest at the slice's end.
#include "gemm_impl.hpp"

#include "fp8b.hpp"

namespace mge {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int FT = 256;                       // rows of a tile on both sides
constexpr int FT_THREADS = 512;
constexpr int FT_OP = FT * 128;               // bytes of an operand in a stage
constexpr int FT_STAGE = 2 * FT_OP;           // tokens, then weights
constexpr int FT_SCALES = 2 * FT_STAGE;       // then a ring of 4 slices' scales: the tokens' and (dW) the row operand's
constexpr int FT_LDS = FT_SCALES + 4 * 2 * FT * 4;

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

// KR: dW (FbWgrad), else C (FbGemm).  SW: the SwiGLU epilogue.
template <bool KR, bool SW, int OUT, typename P>
__device__ __forceinline__ void fb_tile_body(const P& p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int32_t s_prefix[G_MAXE + 1];
  __shared__ int32_t s_mtiles[G_MAXE];
  __shared__ uint32_t s_amax[SW ? 2 * FT : 1];
  const uint32_t lds_base = uniform(int(uint32_t(reinterpret_cast<uintptr_t>(smem))));
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int wn = wave & 1, wt = wave >> 1;    // the wave's half of each 128 weight rows, its 64 tokens
  // derived again from an opaque copy of the lane at the top of every tile and after its K loop, so
  // that one phase's addresses are not kept in registers through the other
  int i16 = lane & 15, q = lane >> 4;
  auto rederive_lane = [&]() {
    int v = lane;
    asm volatile("" : "+v"(v));
    i16 = v & 15;
    q = v >> 4;
  };

  int ncols = KR ? p.K : p.N;                              // columns of C
  if constexpr (SW) ncols = p.F;
  const int per = SW ? FT / 2 : FT;
  const int ntiles = (ncols + per - 1) / per;
  auto group_off = [&](int off) { return off < 0 ? 0 : (off > p.rows ? p.rows : off); };
  auto group_size = [&](int size, int off) { return size < 0 ? 0 : (size > p.rows - off ? p.rows - off : size); };
  if constexpr (!KR) {
    for (int e = tid; e < p.E; e += FT_THREADS)
      s_mtiles[e] = ((p.sizes ? group_size(p.sizes[e], group_off(p.offs[e])) : p.rows) + FT - 1) / FT;
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
  const int ymt = KR ? (p.N + FT - 1) / FT : 0;
  const int total = KR ? p.E * ymt * ntiles : uniform(s_prefix[p.E]);
  const int nwg = gridDim.x;
  int vid = blockIdx.x;
  if ((nwg & 7) == 0) vid = (blockIdx.x & 7) * (nwg >> 3) + (blockIdx.x >> 3);

  auto decode = [&](int tile) {
    FtTile t{};
    t.valid = tile < total;
    if (!t.valid) return t;
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
    t.m0 = (band * 8 + within % gm) * FT;
    t.n0 = (within / gm) * per;
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
      t.nkt = (p.K + 127) / 128;
    }
    return t;
  };

  // LDS rows of a DMA instruction: 8, lane l row l / 8, chunk l % 8; the lane loads the chunk that the
  // swizzle puts there: (l % 8) ^ (l / 16), that ^ 4 in odd instructions
  const int lchunk = ((lane & 7) ^ (lane >> 4)) * 16;
  const uint32_t ldw = KR ? uint32_t(p.rows) : uint32_t(p.K);   // bytes of an operand row

  for (int item = vid; item < total; item += nwg) {
    const FtTile t = decode(item);
    rederive_lane();
    const int tread = (wt * 64 + i16) * 128 + ((q ^ ((i16 >> 1) & 7)) << 4);
    const int wread = (wn * 64 + i16) * 128 + ((q ^ ((i16 >> 1) & 7)) << 4);
    // ---- the tile's operands
    i32x4 rT, rW[2], rS;
    uint32_t toff[4], soff, s_ld;
    const float* wsc[3] = {nullptr, nullptr, nullptr};   // the weights' scales: rows rb 0..3, 4..5, 6..7
    const int KB = KR ? 0 : (p.K + 127) / 128;
    if constexpr (KR) {
      auto left = [](int n, int cap) { return n < 0 ? 0 : (n > cap ? cap : n); };
      rT = make_rsrc_n(p.Y + int64_t(t.m0) * p.rows, uint32_t(left(p.N - t.m0, FT)) * ldw);
#pragma unroll
      for (int i = 0; i < 4; ++i) toff[i] = uint32_t(wave * 32 + i * 8 + (lane >> 3)) * ldw + (lchunk ^ ((i & 1) * 64));
#pragma unroll
      for (int h = 0; h < 2; ++h)
        rW[h] = make_rsrc_n(p.X + int64_t(t.n0 + 128 * h) * p.rows, uint32_t(left(p.K - t.n0 - 128 * h, 128)) * ldw);
      // waves 0..3 bring the scales of 64 rows of dY each, waves 4..7 those of X
      const uint32_t nb = uint32_t((p.rows + 127) / 128);
      const int n = wave < 4 ? p.N : p.K;
      rS = make_rsrc_n(wave < 4 ? p.Yst : p.Xst, nb * uint32_t(n) * 4);
      s_ld = uint32_t(n) * 4;
      soff = uint32_t(t.kbase / 128) * s_ld + uint32_t((wave < 4 ? t.m0 : t.n0) + (wave & 3) * 64 + lane) * 4;
    } else {
      rT = make_rsrc_n(p.A, uint32_t(p.src_rows) * ldw);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = t.m0 + wave * 32 + i * 8 + (lane >> 3);
        int src = t.off + m;
        if (m < t.m_valid && p.map) src = p.map[src];
        const bool in = m < t.m_valid && src >= 0 && src < p.src_rows;
        toff[i] = in ? uint32_t(src) * ldw + (lchunk ^ ((i & 1) * 64)) : kInvalid;
      }
      const uint8_t* w = p.W ? ld_uniform(p.W, t.e) : p.Wv[t.e];
      const float* ws = p.W ? ld_uniform(p.Ws, t.e) : p.Wsv[t.e];
      const int nrows = SW ? p.F : p.N;
      auto left = [](int n, int cap) { return n < 0 ? 0 : (n > cap ? cap : n); };
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r0 = SW ? t.n0 : t.n0 + 128 * h;          // (SwiGLU: gate, then up rows of the same columns)
        rW[h] = make_rsrc_n(w + (int64_t(r0) + (SW ? h * p.F : 0)) * p.K, uint32_t(left(nrows - r0, 128)) * ldw);
      }
      const int last = (SW ? 2 * p.F : p.N) - 1;
      const int up = SW ? p.F + t.n0 + wn * 64 : t.n0 + 128;
      wsc[0] = ws + int64_t(t.n0 / 128) * KB;
      wsc[1] = ws + int64_t(min(up, last) / 128) * KB;
      wsc[2] = ws + int64_t(min(SW ? up + 32 : up, last) / 128) * KB;
      // (waves 4..7 bring the same scales as waves 0..3: every wave then has the same count to wait for)
      rS = make_rsrc_n(p.Ast, uint32_t(KB) * uint32_t(p.ast_ld) * 4);
      s_ld = uint32_t(p.ast_ld) * 4;
      soff = uint32_t(t.off + t.m0 + (wave & 3) * 64 + lane) * 4;
    }
    // ---- DMA of one slice: the tokens, their scales and the first 128 weight rows; the other 128
    // The lane's offsets hold its row and chunk, the slice's place in K is the same in all lanes.  A slice
    // past the last has a resource without records; in the last one, where it is not a whole 128 bytes, the
    // chunks past its end get the top bit.  Both read zeros.
    const int tail = (t.khi - t.kbase) & 127;      // bytes of the last slice, 0: whole
    const uint32_t past0 = tail != 0 && lchunk >= tail ? kInvalid : 0u, past1 = tail != 0 && (lchunk ^ 64) >= tail ? kInvalid : 0u;
    const uint32_t woff = uint32_t(wave * 16 + (lane >> 3)) * ldw + uint32_t(lchunk);
    const uint32_t woff1 = uint32_t(wave * 16 + 8 + (lane >> 3)) * ldw + uint32_t(lchunk ^ 64);
    auto at_slice = [&](i32x4 r, int kt) {
      r[2] = kt < t.nkt ? r[2] : 0;
      return r;
    };
    auto off_at = [&](uint32_t off, int kt, int odd) { return ((odd ? past1 : past0) & (kt == t.nkt - 1 ? kInvalid : 0u)) | off; };
    auto dma_t = [&](int kt, int i) {
      dma16s(at_slice(rT, kt), lds_base + (kt & 1) * FT_STAGE + (wave * 32 + i * 8) * 128, off_at(toff[i], kt, i & 1),
             uint32_t(t.kbase + kt * 128));
    };
    auto dma_w = [&](int kt, int h, int i) {
      dma16s(at_slice(rW[h], kt), lds_base + (kt & 1) * FT_STAGE + FT_OP + (h * 128 + wave * 16 + i * 8) * 128,
             off_at(i ? woff1 : woff, kt, i), uint32_t(t.kbase + kt * 128));
    };
    auto dma_s = [&](int kt) {
      dma4(at_slice(rS, kt), lds_base + FT_SCALES + (kt & 3) * (2 * FT * 4) + (KR ? wave : wave & 3) * 256, soff, uint32_t(kt) * s_ld);
    };
    // The early part of a slice (its tokens, scales and first 128 weight rows: 7 DMAs) and the late one
    // (the other weight rows: 2).
    constexpr int EARLY = 7, LATE = 2;
    auto issue_late = [&](int kt) {
      dma_w(kt, 1, 0);
      dma_w(kt, 1, 1);
    };
    auto issue_early = [&](int kt) {
      dma_s(kt);
      for (int i = 0; i < 4; ++i) dma_t(kt, i);
      for (int i = 0; i < 2; ++i) dma_w(kt, 0, i);
    };

    f32x4 acc[8][4];
#pragma unroll
    for (int rb = 0; rb < 8; ++rb)
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) acc[rb][tb] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (t.nkt > 0) {
      // ---- K loop.  Step rb of a slice multiplies weight block rb by the 4 token blocks, adds the partial
      // sums of the step before (so that no addition waits for its matrix instruction) and reads the next
      // weight block; step 7 also reads the next slice's tokens, each as soon as its last product is issued,
      // so that the matrix unit runs on across slices.  Two barriers a slice:
      //   step 2   every wave has left slice kt - 1: the late part of kt + 1 is issued into its place; the
      //            late part of kt, issued a slice ago, is resident (read from step 3 on)
      //   step 5   every wave has read the early part of kt: that of kt + 2 is issued into its place; that of
      //            kt + 1, issued a slice ago, is resident (read in step 7)
      float swv[3] = {0.f, 0.f, 0.f};     // lane l: the weight scale of slice (kt & ~63) + l
      auto load_swv = [&](int kt) {
        const int kb = min(kt + lane, KB - 1);
#pragma unroll
        for (int h = 0; h < (SW ? 3 : 2); ++h) swv[h] = wsc[h][kb];
        // (here, once in 64 slices: the compiler would otherwise wait for it, and with it for every
        // DMA in flight, where the scales are used)
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
      };
      if constexpr (!KR) load_swv(0);
      lds_barrier();   // every wave is done with the previous tile's slices
      issue_early(0);
      issue_late(0);
      issue_early(1);
      vm_barrier<EARLY + LATE>();        // the early part of slice 0 is resident
      // (the two chunks of a fragment are 64 bytes apart in the row, either way round: a base each, so that the
      // rows' distances fit the instructions' offsets)
      auto frag = [&](const uint8_t* p0, const uint8_t* p1, int at) {
        const uint4 a = *reinterpret_cast<const uint4*>(p0 + at);
        const uint4 b = *reinterpret_cast<const uint4*>(p1 + at);
        return i32x8{int(a.x), int(a.y), int(a.z), int(a.w), int(b.x), int(b.y), int(b.z), int(b.w)};
      };
      auto scales_of = [&](int kt) { return reinterpret_cast<const float*>(smem + FT_SCALES + (kt & 3) * (2 * FT * 4)); };
      i32x8 tf[4], wf[2];
      float ts[4], tn[4], sc[4];          // token scales, those of the next slice, times the weights'
      f32x4 d[2][4], xs[2];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        tf[tb] = frag(smem + tread, smem + (tread ^ 64), tb * 2048);
        tn[tb] = scales_of(0)[wt * 64 + tb * 16 + i16];
        ts[tb] = sc[tb] = 0.f;
        d[1][tb] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      xs[1] = f32x4{0.f, 0.f, 0.f, 0.f};
      wf[0] = frag(smem + wread, smem + (wread ^ 64), FT_OP);
      for (int kt = 0; kt < t.nkt; ++kt) {
        if constexpr (!KR) {
          if ((kt & 63) == 0 && kt > 0) load_swv(kt);
        }
        const int st = (kt & 1) * FT_STAGE, sn = FT_STAGE - st;   // this slice's stage, the next one's
        const uint8_t *w0 = smem + st + wread, *w1 = smem + st + (wread ^ 64);
        static_for<0, 8>([&](auto rbc) {
          constexpr int rb = decltype(rbc)::value;
          constexpr int pb = (rb + 7) & 7;   // the block whose sums are added
          if constexpr (rb == 2) {
            vm_barrier<EARLY>();
            issue_late(kt + 1);
          }
          if constexpr (rb == 5) {
            vm_barrier<LATE>();
            dma_s(kt + 2);
          }
          if constexpr (rb < 7) wf[(rb + 1) & 1] = frag(w0, w1, FT_OP + (rb + 1 < 4 ? (rb + 1) * 2048 : 128 * 128 + (rb + 1 - 4) * 2048));
          else wf[0] = frag(smem + sn + wread, smem + sn + (wread ^ 64), FT_OP);
          if constexpr (KR) xs[rb & 1] = *reinterpret_cast<const f32x4*>(scales_of(kt) + FT + (rb < 4 ? 0 : 128) + wn * 64 + (rb & 3) * 16 + 4 * q);
          if constexpr (KR && rb == 1) {
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) ts[tb] = tn[tb];
          }
          // the scales of the sums that this step adds
          if constexpr (!KR && (rb == 1 || rb == 5 || (SW && rb == 7))) {
            const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(swv[rb == 1 ? 0 : (rb == 5 ? 1 : 2)]), kt & 63));
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
              if constexpr (rb == 1) ts[tb] = tn[tb];
              sc[tb] = ts[tb] * w;
            }
          }
          __builtin_amdgcn_sched_barrier(0);
          static_for<0, 4>([&](auto tbc) {
            constexpr int tb = decltype(tbc)::value;
            const f32x4 z = {0.f, 0.f, 0.f, 0.f};
            d[rb & 1][tb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[rb & 1], tf[tb], z, 0, 0, 0, 0, 0, 0);
            if constexpr (rb == 7) {
              tf[tb] = frag(smem + sn + tread, smem + sn + (tread ^ 64), tb * 2048);
              tn[tb] = scales_of(kt + 1)[wt * 64 + tb * 16 + i16];
            }
            if constexpr (rb == 5 || rb == 6) {
              constexpr int i = (rb - 5) * 4 + tb;   // the early part of kt + 2, one DMA a matrix instruction
              if constexpr (i < 4) dma_t(kt + 2, i);
              else if constexpr (i < 6) dma_w(kt + 2, 0, i - 4);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if constexpr (KR) acc[pb][tb][r] = fmaf(d[(rb + 1) & 1][tb][r] * ts[tb], xs[(rb + 1) & 1][r], acc[pb][tb][r]);
              else acc[pb][tb][r] = fmaf(d[(rb + 1) & 1][tb][r], sc[tb], acc[pb][tb][r]);
            }
            __builtin_amdgcn_sched_barrier(0);
          });
        });
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (KR) acc[7][tb][r] = fmaf(d[1][tb][r] * ts[tb], xs[1][r], acc[7][tb][r]);
          else acc[7][tb][r] = fmaf(d[1][tb][r], sc[tb], acc[7][tb][r]);
        }
    }
    __builtin_amdgcn_s_waitcnt(0);      // the slices past the end (zeros) have landed
    rederive_lane();

    // ---- epilogues.  acc[rb][tb][r]: column n0 + (rb < 4 ? 0 : 128) + wn * 64 + (rb % 4) * 16 + 4q + r,
    // token m0 + wt * 64 + tb * 16 + i16
    const int wrow0 = t.m0 + wt * 64;
    int vr = t.m_valid - wrow0;
    vr = uniform(vr < 0 ? 0 : (vr > 64 ? 64 : vr));
    if constexpr (!SW) {
      constexpr int ESZ = OUT == OUT_BF16 ? 2 : 4;
      uint8_t* base;
      if constexpr (KR) base = static_cast<uint8_t*>(p.D ? ld_uniform(p.D, t.e) : p.Dv[t.e]) + int64_t(wrow0) * ncols * ESZ;
      else base = static_cast<uint8_t*>(p.C) + (int64_t(t.off) + wrow0) * ncols * ESZ;
      const uint32_t rowb = uint32_t(ncols) * ESZ;
      const __amdgpu_buffer_rsrc_t rC = __builtin_amdgcn_make_buffer_rsrc(base, 0, int(uint32_t(vr) * rowb), kRsrcFlags);
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      if (vr > 0) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          const uint32_t row = uint32_t(tb * 16 + i16) * rowb;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c0 = t.n0 + h * 128 + wn * 64;
            if constexpr (OUT == OUT_BF16) {
              uint32_t lo[4], hi[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                lo[j] = bf16x2(acc[4 * h + j][tb][0], acc[4 * h + j][tb][1]);
                hi[j] = bf16x2(acc[4 * h + j][tb][2], acc[4 * h + j][tb][3]);
              }
              transpose4(lo);
              transpose4(hi);
              const int c = c0 + q * 16;   // the lane has columns c .. c + 15 now
              const uint32_t o = c < ncols ? row + uint32_t(c) * ESZ : kInvalid;
              __builtin_amdgcn_raw_buffer_store_b128(u32x4{lo[0], hi[0], lo[1], hi[1]}, rC, int(o), 0, 0);
              __builtin_amdgcn_raw_buffer_store_b128(u32x4{lo[2], hi[2], lo[3], hi[3]}, rC, int(o + 16), 0, 0);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int c = c0 + j * 16 + 4 * q;
                const uint32_t o = c < ncols ? row + uint32_t(c) * ESZ : kInvalid;
                f32x4 v = acc[4 * h + j][tb];
                if constexpr (OUT == OUT_F32_ACC) {
                  const u32x4 old = __builtin_amdgcn_raw_buffer_load_b128(rC, int(o), 0, 0);
#pragma unroll
                  for (int r = 0; r < 4; ++r) v[r] += __uint_as_float(old[r]);
                }
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rC, int(o), 0, 0);
              }
            }
          }
        }
      }
    } else {
      // h = p silu(G) U of the tile's 128 columns, one block of 128 a token: its largest magnitude over
      // the lane's 16 columns, the lanes 16 apart and the two waves of the columns' halves
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      const int64_t grow0 = int64_t(t.off) + wrow0;
      uint32_t am[4];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const bool in = tb * 16 + i16 < vr;
        const float pr = p.prob == nullptr ? 1.f : (in ? p.prob[grow0 + tb * 16 + i16] : 0.f);
        am[tb] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float G = acc[j][tb][r], U = acc[4 + j][tb][r];
            const float h = pr * (G * __builtin_amdgcn_rcpf(1.f + __expf(-G))) * U;
            acc[j][tb][r] = h;
            am[tb] = umax(am[tb], __float_as_uint(h) & 0x7fffffffu);
          }
        const U32Pair a = permlane16_swap(am[tb], am[tb]);
        am[tb] = umax(a.a, a.b);
        const U32Pair b = permlane32_swap(am[tb], am[tb]);
        am[tb] = umax(b.a, b.b);
        if (q == 0) s_amax[wn * FT + wt * 64 + tb * 16 + i16] = am[tb];
      }
      lds_barrier();
      const __amdgpu_buffer_rsrc_t rH =
          __builtin_amdgcn_make_buffer_rsrc(p.h_codes + grow0 * p.F, 0, int(uint32_t(vr) * uint32_t(p.F)), kRsrcFlags);
      if (vr > 0) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          const int m = wt * 64 + tb * 16 + i16;
          const FbScale sc = fb_scale(umax(s_amax[m], s_amax[FT + m]));
          uint32_t v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[j] = e4m3x4(acc[j][tb][0] * sc.inv, acc[j][tb][1] * sc.inv, acc[j][tb][2] * sc.inv, acc[j][tb][3] * sc.inv);
          transpose4(v);
          const int c = t.n0 + wn * 64 + q * 16;
          const uint32_t o = c < p.F ? uint32_t(tb * 16 + i16) * uint32_t(p.F) + uint32_t(c) : kInvalid;
          __builtin_amdgcn_raw_buffer_store_b128(u32x4{v[0], v[1], v[2], v[3]}, rH, int(o), 0, 0);
          if (wn == 0 && q == 0 && tb * 16 + i16 < vr) p.h_scales[int64_t(t.n0 / 128) * p.ast_ld + grow0 + tb * 16 + i16] = sc.s;
        }
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(0);   // no LDS DMA outlives the workgroup
}

#define FB_KERNEL(name, KR, SW, OUT, P) \
  __global__ __launch_bounds__(FT_THREADS, 2) void name(P p) { fb_tile_body<KR, SW, OUT>(p); }
FB_KERNEL(gemm_fb_store, false, false, OUT_BF16, FbGemm)
FB_KERNEL(gemm_fb_store_f32, false, false, OUT_F32, FbGemm)
FB_KERNEL(gemm_fb_swiglu, false, true, OUT_NONE, FbGemm)
FB_KERNEL(gemm_fb_wgrad, true, false, OUT_BF16, FbWgrad)
FB_KERNEL(gemm_fb_wgrad_f32, true, false, OUT_F32, FbWgrad)
FB_KERNEL(gemm_fb_wgrad_f32_acc, true, false, OUT_F32_ACC, FbWgrad)
#undef FB_KERNEL

// One workgroup a CU (its LDS), fewer where there are fewer tiles
template <typename Kern, typename P>
static mge_status launch_fb(Kern kern, const char* name, const P& p, int64_t tiles, hipStream_t s) {
  hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, FT_LDS);
  int64_t grid = device_cus();
  if (tiles < grid) grid = tiles;
  if (grid <= 0) return MGE_OK;
  ProfScope prof(s, name);
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(FT_THREADS), FT_LDS, s, p);
  return hip_check(name);
}

mge_status launch_fb_tile(const FbGemm& p, bool swiglu, hipStream_t s) {
  const int64_t mt = (int64_t(p.total) + FT - 1) / FT + (p.sizes ? p.E : 0);
  if (swiglu) return launch_fb(gemm_fb_swiglu, "gemm_fp8_block_swiglu", p, mt * ((p.F + 127) / 128), s);
  const int64_t tiles = mt * ((p.N + FT - 1) / FT);
  return p.out_f32 ? launch_fb(gemm_fb_store_f32, "gemm_fp8_block", p, tiles, s) : launch_fb(gemm_fb_store, "gemm_fp8_block", p, tiles, s);
}

mge_status launch_fb_wgrad(const FbWgrad& p, hipStream_t s) {
  const int64_t tiles = int64_t(p.E) * ((p.N + FT - 1) / FT) * ((p.K + FT - 1) / FT);
  if (p.out == OUT_BF16) return launch_fb(gemm_fb_wgrad, "wgrad_fp8_block", p, tiles, s);
  if (p.out == OUT_F32) return launch_fb(gemm_fb_wgrad_f32, "wgrad_fp8_block", p, tiles, s);
  return launch_fb(gemm_fb_wgrad_f32_acc, "wgrad_fp8_block", p, tiles, s);
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
