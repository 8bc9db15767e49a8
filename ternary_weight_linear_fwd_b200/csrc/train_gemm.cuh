// train_gemm.cuh -- the two matrix products of BitLinear's straight-through
// gradient.  With y = x~ (alpha W_t)^T, x~ the activation that the 8-bit codes
// stand for, W_t the packed ternary matrix:
//   dx = alpha dy W_t            [M, K]   (backward_input)
//   dW = dy^T x~                 [N, K]   (backward_weight)
#pragma once
#include "train_rows.cuh"

namespace bl {

struct GradArgs {
  int M, N, K;
  const uint16_t* dy;  // bf16 [M, lddy]
  int64_t lddy;
  // backward_input
  const uint8_t* codes;
  const uint8_t* meta;
  int64_t ldc, ldm;
  int nm_n, nm_m;
  const float* alpha;
  const uint16_t* add;  // bf16 [M, K] or null
  uint16_t* dx;         // bf16 [M, K]
  // backward_weight
  const int8_t* q;      // [M, ldq]
  int64_t ldq;
  const float* gamma;
  float* dw;            // [N, K]
  int accumulate;
};

// One weight of a packed matrix, any pattern.
__device__ __forceinline__ float packed_weight(const GradArgs& a, int n, int k) {
  const uint8_t* c = a.codes + static_cast<int64_t>(n) * a.ldc;
  int pos = k;
  if (a.nm_m == 4) {
    const int b = k >> 2;
    const uint32_t nib = (a.meta[static_cast<int64_t>(n) * a.ldm + (b >> 1)] >> (4 * (b & 1))) & 15u;
    const uint32_t j = k & 3;
    if ((nib & 3u) == j)
      pos = 2 * b;
    else if ((nib >> 2) == j)
      pos = 2 * b + 1;
    else
      return 0.0f;
  } else if (a.nm_m == 8) {
    const uint32_t mask = a.meta[static_cast<int64_t>(n) * a.ldm + (k >> 3)], j = k & 7;
    if (!((mask >> j) & 1u)) return 0.0f;
    pos = (k >> 3) * a.nm_n + __popc(mask & ((1u << j) - 1u));
  }
  return static_cast<float>(static_cast<int>((c[pos >> 2] >> (2 * (pos & 3))) & 3u) - 1);
}

// Plain tiles of 64 x 64 outputs, 16 of the reduction a step, 4 x 4 outputs a
// thread, fp32.
template <bool kWeight>
__global__ void __launch_bounds__(256) grad_plain_kernel(const GradArgs a) {
  __shared__ float sA[16][65], sB[16][65];
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const int rows = kWeight ? a.N : a.M, cols = a.K, red = kWeight ? a.M : a.N;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int d0 = 0; d0 < red; d0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      {
        const int d = kWeight ? i >> 6 : i & 15, r = kWeight ? i & 63 : i >> 4;
        float v = 0.0f;
        if (d0 + d < red && r0 + r < rows) {
          const int64_t m = kWeight ? d0 + d : r0 + r, n = kWeight ? r0 + r : d0 + d;
          v = bf16_bits_to_f32(a.dy[m * a.lddy + n]);
        }
        sA[d][r] = v;
      }
      {
        const int d = i >> 6, c = i & 63;
        float v = 0.0f;
        if (d0 + d < red && c0 + c < cols) {
          if (kWeight) {
            const int64_t m = d0 + d;
            v = __fmul_rn(static_cast<float>(a.q[m * a.ldq + c0 + c]), __fdiv_rn(a.gamma[m], kQb));
            v = __bfloat162float(__float2bfloat16_rn(v));
          } else {
            v = packed_weight(a, d0 + d, c0 + c);
          }
        }
        sB[d][c] = v;
      }
    }
    __syncthreads();
#pragma unroll
    for (int d = 0; d < 16; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sA[d][ty * 4 + i], sB[d][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  const float alpha = kWeight ? 1.0f : *a.alpha;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + ty * 4 + i, c = c0 + tx + 16 * j;
      if (r >= rows || c >= cols) continue;
      const int64_t at = static_cast<int64_t>(r) * cols + c;
      if (kWeight) {
        a.dw[at] = acc[i][j] + (a.accumulate ? a.dw[at] : 0.0f);
      } else {
        float v = __fmul_rn(acc[i][j], alpha);
        if (a.add) v = __fadd_rn(v, bf16_bits_to_f32(a.add[at]));
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        a.dx[at] = *reinterpret_cast<const uint16_t*>(&h);
      }
    }
}

}  // namespace bl
