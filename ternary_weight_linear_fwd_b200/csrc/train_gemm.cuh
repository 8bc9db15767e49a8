// train_gemm.cuh -- the two matrix products of BitLinear's straight-through
// gradient.  With y = x~ (alpha W_t)^T, x~ the activation that the 8-bit codes
// stand for, W_t the packed ternary matrix:
//   dx = alpha dy W_t            [M, K]   (backward_input)
//   dW = dy^T x~                 [N, K]   (backward_weight)
//
// Both contract dy (bf16) with an operand that lies compressed in memory with
// the OUTPUT columns contiguous: rows of 2-bit codes (W_t, one per output
// feature n) or of 8-bit codes (x~, one per token m).  On the tensor cores:
//
//   D[256 rows, 256 cols] (fp32, TMEM) += A * B over the reduction, where
//   A = dy.  dx: rows are tokens, the reduction (n) contiguous (K-major);
//       dW: rows are features n, contiguous, the reduction is the tokens.
//   B = the compressed rows expanded to bf16 in shared memory, one 128-byte
//       line per step of the reduction and 64 columns (N-contiguous operand),
//       exactly where the packed row's codes already stand side by side, so
//       that nothing is transposed.
// W_t's values and the 8-bit codes are exact in bf16, dy is bf16: every product
// is exact and the sums are fp32.  x~ = RNb(RN(q RN(gamma / 127))) carries the
// token's scale, which cannot leave the sum over tokens; that rounding to bf16
// is the restored activation's own type (dequant_act gives the same values).
//
// Expanding costs the MMAs' shared-memory bandwidth (a k-block of 256 x 256 x 64
// takes 0.43 us with 2-bit rows and 0.53 with 8-bit codes, 0.37 without) and is
// done again for every 256 rows of the result.  Large products therefore restore
// B once, as bf16 in the workspace, and run with kDense (see gg_dense).
//
// Two CTAs of a cluster share one MMA of 256 x 256 x 16 (cta_group::2): each
// holds its own 128 rows of A and expands its own 128 columns of B, so each
// column is expanded once per 256 rows and the shared-memory reads per MMA
// halve.  Rings as in gemm_tc2.cuh: S copy stages of 64 steps of the reduction
// (A's tile by TMA, the compressed rows), R operand slots (expanded B).  Roles:
// warp 0 copies, warp 1 (rank 0) issues the MMAs, warp 2 owns TMEM, warps 4 ..
// 11 expand (two groups, alternate stages), the last eight store.
//
// Measured (us; fp32 library product of the plain form / bf16 library product
// of operands restored beforehand): dx 2048 x 6912 x 2560 58 (1529 / 47), 8192 x
// 11008 x 2048 230 (- / 235); dW 2048 x 6912 x 2560 62 (1270 / 48), 8192 x 11008 x
// 2048 273 (6120 / 255).  Large ones run at the power-limited rate of the tensor
// cores; in small ones set-up (0.7 us), the first stage (1.4), the epilogue (2 to
// 3) and, with parts, the second launch count as much as the k-blocks.
//
// Persistent: one pair per two SMs walks a static list of units.  The tiles
// that fill whole rounds of pairs run over their whole reduction; the rest are
// cut into `split` parts of the reduction, each part's fp32 tile goes to a slab
// of the workspace, and grad_reduce_kernel adds the parts in order and
// finishes the tile: no atomics, the same bits every time.
#pragma once
#include "nm_decode.cuh"
#include "train_rows.cuh"

namespace bl {

constexpr int kGgRows = 256;      // rows of a pair tile (128 a CTA)
constexpr int kGgCols = 256;      // columns of a pair tile (128 of B a CTA)
constexpr int kGgRed = 64;        // steps of the reduction per stage
constexpr int kGgStoring = 8;      // storing warps, two for each 32 rows: one waits for memory while the other computes
constexpr int kGgGroups = 2;       // groups of four expanding warps, taking the stages in turn
// dW: k-blocks that are summed in TMEM.  The tensor cores cut every addition off below its last place, always towards
// zero, so the error of a sum grows with its length: of a 512 x 9472 result's norm (terms of both signs) 2.1e-7 with 4
// k-blocks, 4.5e-7 with 8, 6.9e-7 with 12, 7.4e-7 with 13, 8.1e-7 with 14, 8.9e-7 with 15, 1.5e-6 with 24, 8.9e-6 with 128.
// Allowed is less than the fp32 library product has at 8192 tokens, 8.9e-7: one sum may have 14 k-blocks (896 tokens).
// Longer ones are added up from pieces in registers, rounded to nearest, whose length leaves room for that: of 12, 6.3e-7
// to 6.9e-7 at any number of tokens.  (Terms of one sign: 2.7e-6 of the sum with one of 14, 2.0e-6 with pieces of 12.)
constexpr int kGgChunk = 12;
constexpr int kGgOneSum = 14;  // up to here the kernel with expansion, which has no registers to add up pieces
constexpr int kGgSlab = kGgRows * kGgCols;  // fp32 of one part of a split tile

struct GradArgs {
  int rows, cols, red;    // output rows and columns, length of the reduction
  int col_tiles;          // tiles: column tile fastest
  int kblocks;            // ceil(red / kGgRed)
  int full;               // tiles run over the whole reduction; the others in `split` parts of `per` k-blocks
  int units;              // full + (tiles - full) * split
  int split, per;
  const float* alpha;     // dx
  const uint16_t* add;    // dx: bf16 [rows, cols] or null
  uint16_t* dx;           // dx: bf16 [rows, cols]
  const float* gamma;     // dW: [red]
  float* dw;              // dW: fp32 [rows, cols]
  int accumulate;         // dW: add to it
  int vec;                // output (and add) rows are 32-byte aligned
  int tma;                // dW: stored (or added) by TMA
  float* slab;            // [(tiles - full) * split][32 groups of 8 columns][256 rows][8]: a warp's store is contiguous
  uint32_t* done;         // [(tiles - full) * split][2 CTAs][kGgStoring]: 1 where the warp stored its share of the part
  int32_t* status;
};

template <bool kWeight, bool kDense>
struct GG {
  static constexpr int A_STAGE = 128 * kGgRed * 2;  // 16 KB
  static constexpr int OP = 128 * kGgRed * 2;       // 16 KB of B: [2 blocks of 64 columns][64 lines][128 B]
  // what lands of B: the operand itself, or compressed rows of 128 codes, 1 or 1/4 byte each
  static constexpr int RAW = kDense ? OP : kWeight ? kGgRed * 128 : kGgRed * 32;
  static constexpr int S = kWeight && !kDense ? 5 : 6;
  static constexpr int R = kDense ? S : 4;          // S >= R: an operand slot's wait is on the stage that filled it
  static constexpr int GROUPS = kDense ? 0 : kGgGroups;
  // k-blocks of one sum in TMEM; dW without kDense is given at most kGgOneSum, and dx is rounded to bf16
  static constexpr int CHUNK = kWeight && kDense ? kGgChunk : 1 << 30;
  static constexpr int THREADS = 32 * (4 + 4 * GROUPS + kGgStoring);
  static constexpr int OUT = kGgStoring * 4096;     // a 32 x 32 tile of results for each storing warp
  static constexpr int FIXED = OUT + 512;
  static constexpr int SMEM = S * (A_STAGE + RAW) + (kDense ? 0 : R * OP) + FIXED;
  static constexpr uint32_t IDESC = idesc_bf16(kGgRows, kGgCols, kWeight, true);
  static_assert(SMEM <= kTcSmemMax, "shared memory");
  static_assert(RAW % 1024 == 0, "stages keep the swizzle's alignment");
};

// 16 ternary codes (2 bits each, k from bit 0) as bf16 weights: word i holds
// those of k = i (low half) and k = i + 8.  A code c at bit 2 j (j = 0, 1, 2) of
// a half-word, ORed into the bf16 128, is 128 + 4^j c; one fused multiply-add
// by 4^-j and -(128 4^-j + 1) leaves c - 1, exactly.
__device__ __forceinline__ void ternary16_bf16(uint32_t w, uint32_t (&o)[8]) {
  const uint32_t t[3] = {w, w >> 6, w >> 12};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = i % 3;
    const uint32_t mask = 0x00030003u << (2 * j);
    const uint32_t v = (t[i / 3] & mask) | 0x43004300u;
    const float mul = j == 0 ? 1.0f : j == 1 ? 0.25f : 0.0625f;
    const __nv_bfloat162 m = __floats2bfloat162_rn(mul, mul);
    const __nv_bfloat162 s = __floats2bfloat162_rn(-(128.0f * mul + 1.0f), -(128.0f * mul + 1.0f));
    const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v), m, s);
    o[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
}

// What is added to one thread's W columns of dx (bf16 pairs), or to dW (fp32), where they are whole; loaded ahead of
// the sums.
template <bool kWeight, int W>
__device__ __forceinline__ void grad_addend(const GradArgs& a, int64_t row, int col, uint32_t (&s)[kWeight ? W : W / 2]) {
  if (!(a.vec && col + W <= a.cols && row < a.rows)) return;
  const int64_t at = row * a.cols + col;
  if (kWeight) {
    if (a.accumulate)
#pragma unroll
      for (int i = 0; i < W; i += 8) ld_global_v8(a.dw + at + i, s + i);
  } else {
    if (a.add)
#pragma unroll
      for (int i = 0; i < W; i += 16) ld_global_v8(a.add + at + i, s + i / 2);
  }
}

// Stores one thread's W consecutive columns (from col) of output row `row`,
// fp32 sums v in natural column order; s: grad_addend's.
template <bool kWeight, int W>
__device__ __forceinline__ void grad_store(const GradArgs& a, int64_t row, int col, const float (&v)[W],
                                           const uint32_t (&s)[kWeight ? W : W / 2], float alpha) {
  const int64_t at = row * a.cols + col;
  const bool whole = a.vec && col + W <= a.cols;
  if (kWeight) {
    float* p = a.dw + at;
    if (whole) {
#pragma unroll
      for (int i = 0; i < W; i += 8) {
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          o[e] = __float_as_uint(a.accumulate ? __fadd_rn(__uint_as_float(s[i + e]), v[i + e]) : v[i + e]);
        st_global_v8(p + i, o);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (col + i < a.cols) p[i] = a.accumulate ? __fadd_rn(p[i], v[i]) : v[i];
    }
  } else {
    uint16_t* p = a.dx + at;
    const uint16_t* q = a.add ? a.add + at : nullptr;
    if (whole) {
#pragma unroll
      for (int i = 0; i < W; i += 16) {
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float lo = __fmul_rn(v[i + 2 * e], alpha), hi = __fmul_rn(v[i + 2 * e + 1], alpha);
          if (q) {
            lo = __fadd_rn(lo, bf16_lo(s[i / 2 + e]));
            hi = __fadd_rn(hi, bf16_hi(s[i / 2 + e]));
          }
          o[e] = pack_bf16x2(lo, hi);
        }
        st_global_v8(p + i, o);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (col + i < a.cols) {
          float f = __fmul_rn(v[i], alpha);
          if (q) f = __fadd_rn(f, bf16_bits_to_f32(q[i]));
          p[i] = static_cast<uint16_t>(pack_bf16x2(f, 0.0f));
        }
    }
  }
}

// A warp's 32 x 32 tile of results in shared memory, rows of 128 bytes with the 128-byte swizzle (which TMA undoes).
__device__ __forceinline__ void grad_tile_put(float* tile, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(tile + lane * 32 + 4 * (c ^ (lane & 7))) =
        make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
__device__ __forceinline__ float grad_tile_get(const float* tile, int r, int c) {
  return tile[r * 32 + (((c >> 2) ^ (r & 7)) << 2) + (c & 3)];
}

// Such a tile (rows from row0, columns from col) to rows that neither TMA nor 32-byte stores can take: a row a step,
// lanes side by side (1000 x 2561 x 2559, dW: 42 us; element by element from each lane's own row 83).
template <bool kWeight>
__device__ __forceinline__ void grad_store_tile(const GradArgs& a, int64_t row0, int col, const float* tile,
                                                float alpha) {
  const int lane = threadIdx.x & 31;
  if (col + lane >= a.cols) return;
#pragma unroll 8
  for (int r = 0; r < 32; ++r) {
    if (row0 + r >= a.rows) break;
    const int64_t at = (row0 + r) * a.cols + col + lane;
    float v = grad_tile_get(tile, r, lane);
    if (kWeight) {
      a.dw[at] = a.accumulate ? __fadd_rn(a.dw[at], v) : v;
    } else {
      v = __fmul_rn(v, alpha);
      if (a.add) v = __fadd_rn(v, bf16_bits_to_f32(a.add[at]));
      a.dx[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f));
    }
  }
}

// The mark of a storing warp's share of part g - a.full (none for tiles that are not split): every warp of every launch
// writes its marks, 0 for what it gave up on, so that grad_reduce_kernel adds up no slab that an earlier call left.
__device__ __forceinline__ void grad_mark(const GradArgs& a, int g, uint32_t rank, int sw, uint32_t v) {
  if (g >= a.full && a.split > 1) a.done[static_cast<size_t>(g - a.full) * (2 * kGgStoring) + rank * kGgStoring + sw] = v;
}

// mapA: dy; box 128 bytes x 128 rows (dx) or 128 bytes x 64 rows (dW), landed 128-byte-swizzled.
// mapB: the compressed rows; box 32 bytes (2-bit) or 128 bytes (8-bit) x 64 rows, landed as they are; with kDense the
// bf16 rows, box 128 bytes x 64 rows, landed 128-byte-swizzled.  mapC (dW, a.tma): fp32, box 32 x 32, 128-byte-swizzled.
template <bool kWeight, bool kDense>
__global__ void __launch_bounds__(GG<kWeight, kDense>::THREADS, 1)
    grad_gemm_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                     const __grid_constant__ CUtensorMap mapC, const GradArgs a) {
  using C = GG<kWeight, kDense>;
  constexpr int S = C::S, R = C::R, G = C::GROUPS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // both CTAs see the same offset, so both leave here together (before any cluster barrier)
  if ((smem_u32(smem_raw) & 1023u) != 0u) {
    if (threadIdx.x == 0) *a.status = kDevBadSmemAlign;
    pdl_wait_primary();
    if (threadIdx.x < kGgStoring)
      for (int g = blockIdx.x >> 1; g < a.units; g += gridDim.x >> 1)
        grad_mark(a, g, cluster_ctarank(), static_cast<int>(threadIdx.x), 0u);
    return;
  }
  uint8_t* sA = smem_raw;                   // [S][16 KB]
  uint8_t* sOp = sA + S * C::A_STAGE;       // [R][OP]
  uint8_t* sRaw = sOp + (kDense ? 0 : R * C::OP);  // [S][RAW]; kDense: the operand slots themselves
  float* sOut = reinterpret_cast<float*>(sRaw + S * C::RAW);  // [kGgStoring][32][32]
  uint64_t* full = reinterpret_cast<uint64_t*>(sRaw + S * C::RAW + C::OUT);
  uint64_t* empty = full + S;
  uint64_t* opready = empty + S;     // [R] rank 0's: both CTAs' expanding warps (kDense: their forwarding threads)
  uint64_t* accfull = opready + R;   // [2]
  uint64_t* accempty = accfull + 2;  // [2] rank 0's: both CTAs' storing warps
  uint64_t* drain = accempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  // unit g -> its tile's first row and column, first k-block and number of k-blocks
  auto unit_of = [&](int g, int& row0, int& col0, int& kb0) {
    int tile = g, n = a.kblocks;
    kb0 = 0;
    if (g >= a.full) {
      const int h = g - a.full;
      tile = a.full + h / a.split;
      kb0 = (h - (tile - a.full) * a.split) * a.per;
      n = min(a.per, a.kblocks - kb0);
    }
    const int rt = tile / a.col_tiles;
    row0 = rt * kGgRows;
    col0 = (tile - rt * a.col_tiles) * kGgCols;
    return n;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int j = 0; j < R; ++j) mbar_init(&opready[j], kDense ? 2 : 8);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], 2 * kGgStoring);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&mapA);
    tma_prefetch_desc(&mapB);
    if (kWeight && a.tma) tma_prefetch_desc(&mapC);
  }
  if (warp == 2) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers exist before any remote arrive or multicast commit
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t opready0 = mapa_shared(smem_u32(opready), 0);
  const uint32_t accempty0 = mapa_shared(smem_u32(accempty), 0);
  pdl_wait_primary();

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ copies (both CTAs)
      bool ok = true;
      int i = 0;
      for (int g = pair; g < a.units && ok; g += npairs) {
        int row0, col0, kb0;
        const int n = unit_of(g, row0, col0, kb0);
        row0 += static_cast<int>(rank) * 128;
        col0 += static_cast<int>(rank) * 128;
        for (int kb = kb0; kb < kb0 + n; ++kb, ++i) {
          const int s = i % S;
          if (i >= S && !mbar_wait(&empty[s], ((i / S) - 1) & 1)) {
            *a.status = kDevTimeoutProducer;
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], C::A_STAGE + C::RAW + test_extra_tx());
          uint8_t* dA = sA + s * C::A_STAGE;
          if (kWeight) {
            tma_load_2d(dA, &mapA, 2 * row0, kb * kGgRed, &full[s]);
            tma_load_2d(dA + 8192, &mapA, 2 * row0 + 128, kb * kGgRed, &full[s]);
          } else {
            tma_load_2d(dA, &mapA, kb * kGgRed * 2, row0, &full[s]);
          }
          uint8_t* dB = sRaw + s * C::RAW;
          if (kDense) {
            tma_load_2d(dB, &mapB, 2 * col0, kb * kGgRed, &full[s]);
            tma_load_2d(dB + 8192, &mapB, 2 * col0 + 128, kb * kGgRed, &full[s]);
          } else {
            tma_load_2d(dB, &mapB, kWeight ? col0 : col0 / 4, kb * kGgRed, &full[s]);
          }
        }
      }
      if (!ok) {  // copies in flight land before the CTA may leave
        for (int j = (i - S > 0 ? i - S : 0); j < i; ++j)
          if (!mbar_wait(&full[j % S], (j / S) & 1)) *a.status = kDevTimeoutDrain;
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      // ------------------------------------------------------------ MMAs (rank 0 only)
      bool issued = false, ok = true;
      int i = 0, t = 0;
      for (int g = pair; g < a.units && ok; g += npairs) {
        int row0, col0, kb0;
        const int n = unit_of(g, row0, col0, kb0);
        for (int k0 = 0; k0 < n && ok; k0 += C::CHUNK, ++t) {
          const int buf = t & 1;
          if (t >= 2 && !mbar_wait_cluster(&accempty[buf], ((t >> 1) - 1) & 1)) {
            *a.status = kDevTimeoutMma;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t dcol = tmem + buf * kGgCols;
          for (int kb = k0; kb < min(n, k0 + C::CHUNK); ++kb, ++i) {
            const int s = i % S, j = i % R;
            // both CTAs' expanding warps arrived: both copies landed and both operands are written
            if (!mbar_wait_cluster(&opready[j], (i / R) & 1)) {
              *a.status = kDevTimeoutMma;
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t ua = smem_u32(sA + s * C::A_STAGE), ub = smem_u32(sOp + j * C::OP);
#pragma unroll
            for (int kk = 0; kk < kGgRed / 16; ++kk) {
              const uint64_t ad = kWeight ? smem_desc_sw128_mnmajor(ua + kk * 2048, 8192)
                                          : smem_desc_sw128_kmajor(ua) + static_cast<uint64_t>(kk * 2);
              tc_mma_f16_ss_pair(dcol, ad, smem_desc_sw128_mnmajor(ub + kk * 2048, 8192), C::IDESC,
                                 kb != k0 || kk != 0 ? 1u : 0u);
            }
            tc_commit_pair_mc(&empty[s], 0x3);  // frees copy stage s, and operand slot j for k-block i + R
            issued = true;
          }
          if (ok) tc_commit_pair_mc(&accfull[buf], 0x3);
        }
      }
      if (!ok && issued) {
        tc_commit_pair(drain);
        if (!mbar_wait(drain, 0)) *a.status = kDevTimeoutDrain;
      }
    }
  } else if (kDense && warp == 3) {
    // -------------------------------------------------------------- both CTAs: this one's copies have landed
    if (lane == 0) {
      int i = 0;
      bool ok = true;
      for (int g = pair; g < a.units && ok; g += npairs) {
        int row0, col0, kb0;
        const int n = unit_of(g, row0, col0, kb0);
        for (int kb = 0; kb < n; ++kb, ++i) {
          const int s = i % S;
          if (!mbar_wait(&full[s], (i / S) & 1)) {
            *a.status = kDevTimeoutUnpack;
            ok = false;
            break;
          }
          mbar_arrive_remote_cta(opready0 + static_cast<uint32_t>(s * 8));
        }
      }
    }
  } else if (!kDense && warp >= 4 && warp < 4 + 4 * G) {
    // -------------------------------------------------------------- expansion (both CTAs)
    // Eight lanes take a line's 128 columns, 16 each; lanes 4 .. 7 (the second
    // block of 64) store their odd chunk first, so the eight 16-byte stores of a
    // line fall into eight bank groups.
    const int grp = (warp - 4) >> 2;
    const int tid = (warp & 3) * 32 + lane;
    const int jc = tid & 7, line0 = tid >> 3;  // lines line0 + 16 u
    const int c0 = 2 * (jc & 3) + (jc >> 2), c1 = 2 * (jc & 3) + 1 - (jc >> 2);
    int i = 0;
    bool ok = true;
    for (int g = pair; g < a.units && ok; g += npairs) {
      int row0, col0, kb0;
      const int n = unit_of(g, row0, col0, kb0);
      for (int kb = kb0; kb < kb0 + n; ++kb, ++i) {
        if (i % kGgGroups != grp) continue;
        const int s = i % S, j = i % R;
        float sc[4];
        if (kWeight) {  // the tokens' scales, read while the copy is in flight
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int m = kb * kGgRed + line0 + 16 * u;
            sc[u] = m < a.red ? a.gamma[m] : 0.0f;
          }
        }
        if (!mbar_wait(&full[s], (i / S) & 1) || (i >= R && !mbar_wait(&empty[(i - R) % S], ((i - R) / S) & 1))) {
          *a.status = kDevTimeoutUnpack;
          ok = false;
          break;
        }
        const uint8_t* raw = sRaw + s * C::RAW;
        uint8_t* op = sOp + j * C::OP + (jc >> 2) * 8192;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int line = line0 + 16 * u;
          uint32_t o[8];
          if (kWeight) {
            const uint4 q = *reinterpret_cast<const uint4*>(raw + line * 128 + jc * 16);
            const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
            const float sv = __fdiv_rn(sc[u], kQb);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float2 f[2];
              codes4_f32(qw[e], f);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                f[h] = __fmul2_rn(f[h], splat2(sv));
                o[2 * e + h] = pack_bf16x2(f[h].x, f[h].y);
              }
            }
          } else {
            ternary16_bf16(*reinterpret_cast<const uint32_t*>(raw + line * 32 + jc * 4), o);
          }
          uint8_t* dst = op + line * 128;
          const bool odd = jc >= 4;
          *reinterpret_cast<uint4*>(dst + ((c0 ^ (line & 7)) << 4)) =
              odd ? make_uint4(o[4], o[5], o[6], o[7]) : make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(dst + ((c1 ^ (line & 7)) << 4)) =
              odd ? make_uint4(o[0], o[1], o[2], o[3]) : make_uint4(o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_cta(opready0 + static_cast<uint32_t>(j * 8));
      }
    }
  } else if (warp >= 4 + 4 * G) {
    // -------------------------------------------------------------- stores (both CTAs, own rows)
    const int sw = warp - 4 - 4 * G;
    const int q = sw & 3, first = (sw >> 2) * 32;  // 32 rows, every other 32 columns
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const float alpha = kWeight ? 1.0f : *a.alpha;
    // 32 columns of a row a lane, from c0 of the tile: to their slab, or finished
    auto finish = [&](int g, int row0, int col0, int wrow, int c0, const float (&v)[32], const uint32_t (&s0)[16]) {
      const bool part = g >= a.full && a.split > 1;
      float* out = sOut + sw * 1024;
      if (row0 + wrow < a.rows && col0 + c0 < a.cols) {
        if (part) {
          float* p = a.slab + static_cast<size_t>(g - a.full) * kGgSlab + (c0 / 8 * kGgRows + wrow + lane) * 8;
#pragma unroll
          for (int c = 0; c < 4; ++c) st_global_v8(p + c * 8 * kGgRows, reinterpret_cast<const uint32_t*>(v + 8 * c));
        } else if (!kWeight && a.vec && col0 + c0 + 32 <= a.cols) {
          if (row0 + wrow + lane < a.rows)
            grad_store<false, 32>(a, row0 + wrow + lane, col0 + c0, v, s0, alpha);
        } else if (kWeight && a.tma) {
          if (lane == 0) bulk_wait_read<0>();  // the last store has read the tile
          __syncwarp();
          grad_tile_put(out, v);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (a.accumulate)
              tma_add_2d(&mapC, col0 + c0, row0 + wrow, out);
            else
              tma_store_2d(&mapC, col0 + c0, row0 + wrow, out);
            bulk_commit();
          }
        } else {
          grad_tile_put(out, v);
          __syncwarp();
          grad_store_tile<kWeight>(a, row0 + wrow, col0 + c0, out, alpha);
          __syncwarp();
        }
      }
    };
    int t = 0, g = pair;
    for (; g < a.units; g += npairs) {
      int row0, col0, kb0;
      const int n = unit_of(g, row0, col0, kb0);
      const int wrow = static_cast<int>(rank) * 128 + q * 32;  // the warp's first row of the tile
      if constexpr (C::CHUNK < 1 << 30) {
        // the warp's 32 rows of 4 x 32 columns are summed up in registers, then stored while the next tile is computed
        float acc[4][32];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int c = 0; c < 32; ++c) acc[u][c] = 0.0f;
        bool ok = true;
        for (int k0 = 0; k0 < n; k0 += C::CHUNK, ++t) {
          const int buf = t & 1;
          if (!mbar_wait(&accfull[buf], (t >> 1) & 1)) {
            *a.status = kDevTimeoutEpilogue;
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            uint32_t w[16];
            tc_ld_32x32b_x16(tmem + lane_base + buf * kGgCols + first + 64 * (u / 2) + 16 * (u % 2), w);
            tc_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c)
              acc[u / 2][16 * (u % 2) + c] = __fadd_rn(acc[u / 2][16 * (u % 2) + c], __uint_as_float(w[c]));
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote_cta(accempty0 + static_cast<uint32_t>(buf * 8));
        }
        if (!ok) break;
        const uint32_t none[16] = {};
#pragma unroll
        for (int u = 0; u < 4; ++u) finish(g, row0, col0, wrow, first + 64 * u, acc[u], none);
      } else {
        const int buf = t & 1;
        const bool part = g >= a.full && a.split > 1;
        uint32_t s0[16], s1[16];
        if (!kWeight && !part) grad_addend<false, 32>(a, row0 + wrow + lane, col0 + first, s0);
        if (!mbar_wait(&accfull[buf], (t >> 1) & 1)) {
          *a.status = kDevTimeoutEpilogue;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int c0 = first; c0 < kGgCols; c0 += 64) {
          uint32_t w[32];
          tc_ld_32x32b_x32(tmem + lane_base + buf * kGgCols + c0, w);
          if (!kWeight && !part && c0 + 64 < kGgCols)
            grad_addend<false, 32>(a, row0 + wrow + lane, col0 + c0 + 64, s1);
          tc_wait_ld();
          float v[32];
#pragma unroll
          for (int c = 0; c < 32; ++c)  // 2-bit rows: accumulator column 2 i + h of a 16-group is output column i + 8 h
            v[kWeight || kDense ? c : (c & 16) + ((c & 15) >> 1) + 8 * (c & 1)] = __uint_as_float(w[c]);
          finish(g, row0, col0, wrow, c0, v, s0);
          if (!kWeight)
#pragma unroll
            for (int i = 0; i < 16; ++i) s0[i] = s1[i];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_cta(accempty0 + static_cast<uint32_t>(buf * 8));
        ++t;
      }
      if (lane == 0) grad_mark(a, g, rank, sw, 1u);
    }
    for (; g < a.units; g += npairs)  // given up
      if (lane == 0) grad_mark(a, g, rank, sw, 0u);
    if (kWeight && lane == 0) bulk_wait_read<0>();  // the stores have read the tiles before the CTA ends
  }
  tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();
  cluster_sync_all();  // no remote arrive or multicast commit is left in flight towards either CTA
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// The split tiles: adds each tile's parts in order and finishes it, but for what
// has a part that was given up on.  A thread takes 16 columns of a row, four
// parts' loads in flight.
constexpr int kGgReduceCtas = kGgRows * kGgCols / 16 / 256;  // of a tile
template <bool kWeight>
__global__ void __launch_bounds__(256) grad_reduce_kernel(const GradArgs a) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int unit = blockIdx.x / kGgReduceCtas;                              // split tile
  const int lrow = threadIdx.x, lc = (blockIdx.x % kGgReduceCtas) * 16;     // 256 rows a CTA
  const int tile = a.full + unit;
  const int rt = tile / a.col_tiles;
  const int64_t row = static_cast<int64_t>(rt) * kGgRows + lrow;
  const int col = (tile - rt * a.col_tiles) * kGgCols + lc;
  if (row >= a.rows || col >= a.cols) return;
  const float* p = a.slab + static_cast<size_t>(unit) * a.split * kGgSlab + (lc / 8 * kGgRows + lrow) * 8;
  uint32_t add[kWeight ? 16 : 8];
  grad_addend<kWeight, 16>(a, row, col, add);
  const uint32_t* done = a.done + static_cast<size_t>(unit) * a.split * (2 * kGgStoring) + (lrow >> 7) * kGgStoring +
                         ((lc >> 5) & 1) * 4 + ((lrow >> 5) & 3);  // of the warp that stored these
  uint32_t all = 1u;
  float v[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) v[c] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < a.split; ++s) {
    all &= done[s * (2 * kGgStoring)];
    uint32_t w[16];
    ld_global_v8(p + static_cast<size_t>(s) * kGgSlab, w);
    ld_global_v8(p + static_cast<size_t>(s) * kGgSlab + 8 * kGgRows, w + 8);
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] = __fadd_rn(v[c], __uint_as_float(w[c]));
  }
  if (all) grad_store<kWeight, 16>(a, row, col, v, add, kWeight ? 1.0f : *a.alpha);
}

// ----------------------------------------------------------------- operands put in order
// Rows whose stride TMA cannot step (not a multiple of 16 bytes), copied to rows that it can, zero behind their ends:
// of dy, of the codes, or of both in one launch (the first dy_blocks CTAs take dy, 8 values a thread; the others the
// codes, 16 a thread).
struct PadArgs {
  const uint16_t* dy;
  int64_t lddy, ldd;      // of the source, of the copy
  uint16_t* dy_out;
  const int8_t* q;
  int64_t ldq, ldqd;
  int8_t* q_out;
  int M, N, K;
  unsigned dy_blocks;     // 0: dy is not copied
};
__global__ void __launch_bounds__(256) pad_rows_kernel(const PadArgs a) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const bool dy = blockIdx.x < a.dy_blocks;
  const unsigned per = static_cast<unsigned>(dy ? a.ldd / 8 : a.ldqd / 16);  // chunks of a row
  const int64_t at = static_cast<int64_t>(dy ? blockIdx.x : blockIdx.x - a.dy_blocks) * 256 + threadIdx.x;
  const int64_t row = at / per;
  const int c = static_cast<int>(at - row * per);
  if (row >= a.M) return;
  uint32_t w[4];
  if (dy) {
    load8_any(a.dy + row * a.lddy, 8 * c, a.N, a.dy, a.dy + (a.M - 1) * a.lddy + a.N, w);
    *reinterpret_cast<uint4*>(a.dy_out + row * a.ldd + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    load16_codes_any(a.q + row * a.ldq, 16 * c, a.K, a.q, a.q + (a.M - 1) * a.ldq + a.K, w);
    *reinterpret_cast<uint4*>(a.q_out + row * a.ldqd + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// N:M rows expanded to dense codes (16 weights a thread), the layout of the
// dense matrix of the same size; positions past K hold code 1.
__global__ void __launch_bounds__(256) nm_expand_kernel(const ExpandArgs a) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int words = static_cast<int>(a.ldd / 4);
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= static_cast<int64_t>(a.N) * words) return;
  const int64_t n = at / words;
  a.out[at] = nm_codes16(a, n, static_cast<int>(at - n * words) * 16);
}

// Dense or N:M rows as bf16 values, rows of a multiple of 16 columns (those past K are never read).
__global__ void __launch_bounds__(256) ternary_bf16_kernel(const ExpandArgs a) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int words = static_cast<int>(a.ldd / 16);
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= static_cast<int64_t>(a.N) * words) return;
  const int64_t n = at / words;
  const int w = static_cast<int>(at - n * words);
  const uint32_t c = a.nm_m ? nm_codes16(a, n, 16 * w) : *reinterpret_cast<const uint32_t*>(a.codes + n * a.ldc + 4 * w);
  uint32_t v[8], o[8];
  ternary16_bf16(c, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] = __byte_perm(v[2 * i], v[2 * i + 1], 0x5410);
    o[4 + i] = __byte_perm(v[2 * i], v[2 * i + 1], 0x7632);
  }
  st_global_v8(reinterpret_cast<uint16_t*>(a.out) + at * 16, o);
}

}  // namespace bl
