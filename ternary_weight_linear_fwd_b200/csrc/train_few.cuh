// train_few.cuh -- dx = alpha dy W_t (+ add) for a few tokens, in one launch.
//
// With few tokens the pair GEMM of train_gemm.cuh spends its time on what it
// sets up: rows of its 256-row tile are empty, its parts go through slabs of
// memory and a second launch adds them (18 us for 16 tokens, N = 2560, K =
// 6912).  The product itself only reads the packed matrix (4.4 MB there: 0.7
// us), so here each warp expands packed words in registers and multiplies with
// mma.sync.m16n8k16 (bf16, fp32 sums): no tile is staged, no operand waits for
// another warp, and the packed words are used where they land.
//
// A warp takes 64 output columns (8 of the 16 codes of each of 8 words a row)
// and 64 steps n of the reduction at a time.  The order of n inside the 64 is
// free as long as both operands follow it: lane 4 g + t reads word g of the
// rows n = 16 t .. 16 t + 15 and 16 consecutive dy of the tokens g and g + 8, and
// MMA step s takes n = 16 t + 4 s .. + 3.  A word's 8 columns go to 8 MMAs:
// column j of the eight words is one n8 tile, and two rows' codes of one column
// lie side by side after one byte permutation, which is what the operand wants.
// The sixteen warps of a CTA take the n in turn; their sums are added in shared
// memory in order of the warps, those of a cluster's CTAs (each with its part
// of n) in order of their ranks: no atomics, the same bits every time.
#pragma once
#include "train_gemm.cuh"

namespace bl {

constexpr int kFewWarps = 16;
constexpr int kFewSpan = 128;   // output columns of eight words; a CTA computes every other eight of them
constexpr int kFewRed = 64;     // steps of the reduction a warp takes at a time
constexpr int kFewRow = 72;     // floats of a row of sums: 4 rows apart fall into different banks
constexpr int kFewSmem = kFewWarps * 16 * kFewRow * 4;

struct FewArgs {
  const uint8_t* codes;  // dense rows (an N:M matrix's are expanded before)
  int64_t ldc;
  int N, K;
  const uint16_t* dy;
  int64_t lddy;
  int M;
  int chunks, per;       // 64-wide pieces of N; those of one CTA
  int cs;                // CTAs of a cluster: 1, 2, 4 or 8
  const float* alpha;
  const uint16_t* add;   // bf16 [M, K] or null
  uint16_t* dx;
};

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// blockIdx.x = (2 * span of columns + half of its words) * cs + rank in the cluster, blockIdx.y = 16 tokens.
__global__ void __launch_bounds__(32 * kFewWarps, 1) few_input_kernel(const FewArgs a) {
  extern __shared__ __align__(16) float s_few[];  // [warp][16 tokens][kFewRow]: position 8 j + g is column 16 g + 8 half + j
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = a.cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / a.cs, half = unit & 1;
  const int col0 = (unit >> 1) * kFewSpan, m0 = blockIdx.y * 16;
  const int N = a.N, K = a.K;
  const int end = min((rank + 1) * a.per, a.chunks);
  const bool vec = (a.lddy % 8) == 0 && (reinterpret_cast<uintptr_t>(a.dy) & 15u) == 0;
  // columns past K and tokens past M read the last ones: what they give is not stored
  const int word = min(col0 / 16 + g, (K - 1) / 16);
  const uint16_t* yr[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) yr[h] = a.dy + static_cast<int64_t>(min(m0 + g + 8 * h, a.M - 1)) * a.lddy;
  pdl_wait_primary();
  pdl_launch_dependents();

  const uint32_t sel = half ? 0x7632 : 0x5410;
  float d[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) d[j][i] = 0.0f;
  for (int ch = rank * a.per + warp; ch < end; ch += kFewWarps) {
    const int n0 = ch * kFewRed + 16 * t;
    uint32_t y[2][8], w[16];  // dy of tokens g, g + 8; packed words of 16 rows
    const bool whole = ch * kFewRed + kFewRed <= N;
    if (whole) {
      const uint8_t* p = a.codes + static_cast<int64_t>(n0) * a.ldc + 4 * word;
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p + i * a.ldc));
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        w[i] = 0x55555555u;
        if (n0 + i < N) w[i] = __ldg(reinterpret_cast<const uint32_t*>(a.codes + (n0 + i) * a.ldc + 4 * word));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t r[4];
        if (vec && whole) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(yr[h] + n0 + 8 * q));
          r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
        } else {
          load8_raw(yr[h], n0 + 8 * q, N, vec, r);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y[h][4 * q + i] = r[i];
      }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t av[4] = {y[0][2 * s], y[1][2 * s], y[0][2 * s + 1], y[1][2 * s + 1]};
      uint32_t b0[8], b1[8];
      ternary16_bf16(__byte_perm(w[4 * s], w[4 * s + 1], sel), b0);
      ternary16_bf16(__byte_perm(w[4 * s + 2], w[4 * s + 3], sel), b1);
#pragma unroll
      for (int j = 0; j < 8; ++j) mma_bf16_16816(d[j], av, b0[j], b1[j]);
    }
  }

  // this warp's sums; then the CTA's, into the first warp's place
  float* mine = s_few + warp * 16 * kFewRow;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    *reinterpret_cast<float2*>(mine + g * kFewRow + 8 * j + 2 * t) = make_float2(d[j][0], d[j][1]);
    *reinterpret_cast<float2*>(mine + (g + 8) * kFewRow + 8 * j + 2 * t) = make_float2(d[j][2], d[j][3]);
  }
  __syncthreads();
  if (threadIdx.x < 16 * 64 / 4) {
    float4* p = reinterpret_cast<float4*>(s_few + (threadIdx.x >> 4) * kFewRow + 4 * (threadIdx.x & 15));
    float4 v = p[0];
#pragma unroll
    for (int k = 1; k < kFewWarps; ++k) {
      const float4 u = p[k * 16 * kFewRow / 4];
      v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
    }
    p[0] = v;
  }
  if (a.cs > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // each CTA finishes 8 / cs of the eight words' columns
  const int words = 8 / a.cs;
  const float alpha = *a.alpha;
  const uint32_t s0 = smem_u32(s_few);
  for (int i = threadIdx.x; i < 16 * 8 * words; i += 32 * kFewWarps) {
    const int j = i & 7, row = (i >> 3) & 15, wd = rank * words + (i >> 7);
    const int at = row * kFewRow + 8 * j + wd;
    float v = s_few[at];
    if (a.cs > 1) {
      v = 0.0f;
      for (int r = 0; r < a.cs; ++r)
        v += __uint_as_float(ld_cluster_u32(mapa_shared(s0 + 4 * at, static_cast<uint32_t>(r))));
    }
    const int col = col0 + 16 * wd + 8 * half + j;
    if (m0 + row < a.M && col < K) {
      const int64_t o = static_cast<int64_t>(m0 + row) * K + col;
      v = __fmul_rn(v, alpha);
      if (a.add) v = __fadd_rn(v, bf16_bits_to_f32(a.add[o]));
      a.dx[o] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f));
    }
  }
  if (a.cs > 1) cluster_sync_all();  // no CTA leaves while another reads its sums
}

}  // namespace bl
