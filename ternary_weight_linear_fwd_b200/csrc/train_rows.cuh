// train_rows.cuh -- row-wise kernels of BitLinear's training side: layer norm
// forward (to bf16 or to the 8-bit codes a BitLinear reads), the backward
// passes of layer norm and RMSNorm, the 8-bit checkpoint of the squared-ReLU
// gated FFN with the backward pass that reads it, and the restored activation.
//
// All of them are bound by memory: a few operations per element, every input
// read once and every output written once.
#pragma once
#include "gemv.cuh"

namespace bl {

// ----------------------------------------------------------------- helpers
// 16 fp32 parameters from k0 (zero past K).
__device__ __forceinline__ void load16_f32(const float* p, int k0, int K, float (&v)[16]) {
  if (k0 + 16 <= K && (reinterpret_cast<uintptr_t>(p + k0) & 15u) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = reinterpret_cast<const float4*>(p + k0)[i];
      v[4 * i] = t.x; v[4 * i + 1] = t.y; v[4 * i + 2] = t.z; v[4 * i + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = k0 + i < K ? p[k0 + i] : 0.0f;
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 8 bf16 values at row[k0 ..], those past K left out.
__device__ __forceinline__ void store8_bf16(uint16_t* row, int k0, int K, bool vec, const uint32_t* o) {
  if (vec && k0 + 8 <= K) {
    *reinterpret_cast<uint4*>(row + k0) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k0 + i < K) row[k0 + i] = static_cast<uint16_t>(o[i >> 1] >> (16 * (i & 1)));
  }
}

// 16 codes at row[k0 ..], those past K left out.
__device__ __forceinline__ void store16_codes(int8_t* row, int k0, int K, bool vec, const uint4 w) {
  if (vec && k0 + 16 <= K) {
    *reinterpret_cast<uint4*>(row + k0) = w;
  } else {
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (k0 + i < K) row[k0 + i] = static_cast<int8_t>(ww[i >> 2] >> (8 * (i & 3)));
  }
}

// 16 codes from row[k0 ..] (zero past K).
__device__ __forceinline__ void load16_codes(const int8_t* row, int k0, int K, bool vec, uint32_t (&w)[4]) {
  if (vec && k0 + 16 <= K) {
    const uint4 t = *reinterpret_cast<const uint4*>(row + k0);
    w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k0 + 4 * i + j < K) w[i] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k0 + 4 * i + j])) << (8 * j);
    }
  }
}

// 8 fp32 values of shared memory (16-byte aligned).
__device__ __forceinline__ void load8_smem(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Four int8 codes as fp32, exactly: the code plus 128 goes into the low byte
// of 2^23, whose last place is 1.
__device__ __forceinline__ void codes4_f32(uint32_t w, float (&f)[4]) {
  const uint32_t u = w ^ 0x80808080u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    f[j] = __fsub_rn(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + j)), 8388736.0f);
}

// ----------------------------------------------------------------- layer norm
// Per row: s1 = sum x, s2 = sum x^2 in fp64 (the squares of bf16 values are
// exact there, so the one-pass variance s2 - s1^2 / K loses nothing a two-pass
// one would keep: 53 bits against the 24 of its result even at a mean of a
// thousand deviations); mean = RN32(s1 / K), var = RN32(max(0, (s2 - s1^2 / K) /
// K)), rstd = RN32(1 / sqrt(var + eps)) with root and quotient in fp64, and
//   xn = RN(RN(RN(x - mean) * rstd) * w) (+ RN b)
// every operation one fp32 rounding, so that the codes are defined to the bit.
struct LnArgs {
  const uint16_t* x;
  int64_t ldx;
  int M, K;
  const float* w;
  const float* b;  // or null
  float eps;
  uint16_t* y;     // bf16 out [M, K] (kCodes = false)
  int8_t* q;       // codes out [M, K] (kCodes = true)
  float* gamma;
  int32_t* rowsum;
  float* mean;     // or null
  float* rstd;     // or null
  int wpr;         // warps per row
};

// A row belongs to wpr warps of a 256-thread CTA; a lane owns the 16-wide
// groups g = sub * 32 + lane + j * 32 * wpr.  Rows of up to 16 G lanes * wpr
// elements stay in registers between the three passes (moments, maximum,
// output); longer or unaligned rows are read again, from L2.
template <bool kCodes, int G>
__global__ void __launch_bounds__(32 * kQuantWarps, G <= 3 ? 3 : 2) layernorm_kernel(const LnArgs a) {
  __shared__ double s_s1[kQuantWarps], s_s2[kQuantWarps];
  __shared__ float s_mx[kQuantWarps];
  __shared__ int32_t s_sum[kQuantWarps];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = a.wpr, K = a.K;
  const int rloc = warp / wpr, sub = warp - rloc * wpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kQuantWarps / wpr) + rloc;
  const bool active = row < a.M;  // inactive warps still reach the CTA barriers
  const uint16_t* xr = a.x + (active ? row : 0) * a.ldx;
  const bool vec_ok = (a.ldx % 8) == 0 && (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0;
  const int groups = (K + 15) / 16;
  const int gstride = 32 * wpr;
  const int g0 = sub * 32 + lane;
  const bool in_regs = groups <= G * gstride;

  uint32_t v[G][8];
  if (active && in_regs) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int g = g0 + j * gstride;
      if (g < groups) {
        uint32_t r0[4], r1[4];
        load8_raw(xr, 16 * g, K, vec_ok, r0);
        load8_raw(xr, 16 * g + 8, K, vec_ok, r1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[j][i] = r0[i];
          v[j][4 + i] = r1[i];
        }
      }
    }
  }
  auto for_groups = [&](auto&& f) {
    if (!active) return;
    if (in_regs) {
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (g0 + j * gstride < groups) f(g0 + j * gstride, v[j]);
    } else {
      for (int g = g0; g < groups; g += gstride) {
        uint32_t r0[4], r1[4];
        load8_raw(xr, 16 * g, K, vec_ok, r0);
        load8_raw(xr, 16 * g + 8, K, vec_ok, r1);
        const uint32_t r[8] = {r0[0], r0[1], r0[2], r0[3], r1[0], r1[1], r1[2], r1[3]};
        f(g, r);
      }
    }
  };

  double s1 = 0.0, s2 = 0.0;
  for_groups([&](int, const uint32_t (&r)[8]) {  // zero past K
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double lo = static_cast<double>(__uint_as_float(r[i] << 16));
      const double hi = static_cast<double>(__uint_as_float(r[i] & 0xFFFF0000u));
      s1 += lo;
      s2 = __fma_rn(lo, lo, s2);
      s1 += hi;
      s2 = __fma_rn(hi, hi, s2);
    }
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    s2 += __shfl_xor_sync(0xffffffffu, s2, o);
  }
  if (wpr > 1) {
    if (lane == 0) {
      s_s1[warp] = s1;
      s_s2[warp] = s2;
    }
    __syncthreads();
    s1 = s2 = 0.0;
    for (int i = 0; i < wpr; ++i) {
      s1 += s_s1[rloc * wpr + i];
      s2 += s_s2[rloc * wpr + i];
    }
  }
  const double kd = static_cast<double>(K);
  const float mean = __double2float_rn(__ddiv_rn(s1, kd));
  const double vard = __ddiv_rn(s2 - __ddiv_rn(s1 * s1, kd), kd);
  const float var = __double2float_rn(vard < 0.0 ? 0.0 : vard);  // NaN stays NaN
  const float rstd =
      __double2float_rn(__ddiv_rn(1.0, __dsqrt_rn(static_cast<double>(var) + static_cast<double>(a.eps))));
  if (active && sub == 0 && lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }

  // the group's normalised values; past K they are zero
  auto normed = [&](int g, const uint32_t (&r)[8], float (&xn)[16]) {
    float w[16], b[16];
    load16_f32(a.w, 16 * g, K, w);
    if (a.b) load16_f32(a.b, 16 * g, K, b);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float x = __uint_as_float((e & 1) ? (r[e >> 1] & 0xFFFF0000u) : (r[e >> 1] << 16));
      xn[e] = __fmul_rn(__fmul_rn(__fsub_rn(x, mean), rstd), w[e]);
      if (a.b) xn[e] = __fadd_rn(xn[e], b[e]);
    }
  };

  if (!kCodes) {
    uint16_t* yr = a.y + (active ? row : 0) * K;
    const bool yvec = (K % 8) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15u) == 0;
    for_groups([&](int g, const uint32_t (&r)[8]) {
      float xn[16];
      normed(g, r, xn);
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = pack_bf16x2(xn[2 * i], xn[2 * i + 1]);
      store8_bf16(yr, 16 * g, K, yvec, o);
      store8_bf16(yr, 16 * g + 8, K, yvec, o + 4);
    });
    return;
  }

  float mx = 0.0f;
  for_groups([&](int g, const uint32_t (&r)[8]) {
    float xn[16];
    normed(g, r, xn);
#pragma unroll
    for (int e = 0; e < 16; ++e) mx = fmaxf(mx, fabsf(xn[e]));
  });
  mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
  if (wpr > 1) {
    if (lane == 0) s_mx[warp] = mx;
    __syncthreads();
    for (int i = 0; i < wpr; ++i) mx = fmaxf(mx, s_mx[rloc * wpr + i]);
  }
  const float d = __fadd_rn(mx, kEps);
  const float c = __fmul_rn(kQb, __frcp_rn(d));
  int32_t sum = 0;
  int8_t* qr = a.q + (active ? row : 0) * K;
  const bool qvec = (K % 16) == 0 && (reinterpret_cast<uintptr_t>(a.q) & 15u) == 0;
  for_groups([&](int g, const uint32_t (&r)[8]) {
    float xn[16];
    normed(g, r, xn);
    uint32_t b0[8], b1[8];
    codes8f(xn, c, d, b0);
    codes8f(xn + 8, c, d, b1);
    store16_codes(qr, 16 * g, K, qvec, pack_group<false>(b0, b1, sum));
  });
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (wpr > 1) {
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    sum = 0;
    for (int i = 0; i < wpr; ++i) sum += s_sum[rloc * wpr + i];
  }
  if (active && sub == 0 && lane == 0) {
    a.gamma[row] = mx;
    if (a.rowsum) a.rowsum[row] = sum;
  }
}

// ----------------------------------------------------------------- norm backward
// Layer norm, per row, with xh = (x - mean) rstd and a = dy w:
//   dx = rstd (a - mean_k(a) - xh mean_k(a xh)),  dw = sum_m dy xh,  db = sum_m dy
// RMSNorm (xh = x r, r = 1 / sqrt(mean_k(x^2) + eps), recomputed here since the
// row is read anyway):
//   dx = r (a - xh mean_k(a xh)),  dg = sum_m dy xh.
// A CTA holds rg groups of T threads; a group walks rows, each of its threads
// owning the 8-wide column chunks t + j T (j < G) of every row, so that the
// column sums of dw and db stay in its registers (fp32) until the end: x and
// dy are read once.  Each CTA adds its groups' sums in order and writes one
// partial row; norm_reduce_kernel adds the partial rows in a fixed order.
struct NbArgs {
  const uint16_t* dy;
  int64_t lddy;
  const uint16_t* x;
  int64_t ldx;
  int M, K;
  const float* w;
  const float* mean;   // layer norm
  const float* rstd;   // layer norm
  float eps;           // RMSNorm
  uint16_t* dx;        // [M, K]
  float* part;         // [CTAs][2 or 1][K]
  int T, rg;
};

constexpr int kNbMaxThreads = 768;
constexpr int kNbMaxGroups = 8;                       // one named barrier each
constexpr int kNbMaxK = 2 * 8 * kNbMaxThreads;        // two chunks a thread; longer rows take the split kernels

template <bool kLayer, int G>
__global__ void __launch_bounds__(kNbMaxThreads, 1) norm_backward_kernel(const NbArgs a) {
  extern __shared__ float s_nb[];  // [8 G T] the weight, zero past K; then [K] column sums handed from group to group
  __shared__ float2 s_red[2][kNbMaxThreads / 32];
  const int T = a.T, K = a.K;
  float* s_w = s_nb;
  float* s_acc = s_nb + 8 * G * T;
  for (int k = threadIdx.x; k < 8 * G * T; k += blockDim.x) s_w[k] = k < K ? a.w[k] : 0.0f;
  const int grp = threadIdx.x / T, t = threadIdx.x - grp * T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w0 = grp * (T / 32), nw = T / 32;
  const int chunks = (K + 7) / 8;
  const bool vx = (a.ldx % 8) == 0 && (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0;
  const bool vdy = (a.lddy % 8) == 0 && (reinterpret_cast<uintptr_t>(a.dy) & 15u) == 0;
  const bool vdx = (K % 8) == 0 && (reinterpret_cast<uintptr_t>(a.dx) & 15u) == 0;
  const float kf = static_cast<float>(K);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * a.rg;

  float dwv[G][8], dbv[G][8];
#pragma unroll
  for (int j = 0; j < G; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) dwv[j][e] = dbv[j][e] = 0.0f;
  uint32_t xw[G][4], yw[G][4], nx[G][4], ny[G][4];  // this row's words and the next one's
  auto load = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int c = t + j * T;
      if (c < chunks) {
        load8_raw(a.x + row * a.ldx, 8 * c, K, vx, nx[j]);
        load8_raw(a.dy + row * a.lddy, 8 * c, K, vdy, ny[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) nx[j][i] = ny[j][i] = 0u;
      }
    }
  };
  auto el = [](const uint32_t (&w)[4], int e) { return (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]); };
  __syncthreads();
  int64_t row = static_cast<int64_t>(blockIdx.x) * a.rg + grp;
  if (row < a.M) load(row);
  for (int it = 0; row < a.M; row += stride, it ^= 1) {
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xw[j][i] = nx[j][i];
        yw[j][i] = ny[j][i];
      }
    if (row + stride < a.M) load(row + stride);  // in flight while this row's sums go round
    float mean = 0.0f, rstd = 1.0f;
    if (kLayer) {
      mean = a.mean[row];
      rstd = a.rstd[row];
    }
    float c1 = 0.0f, c2 = 0.0f;  // layer: sum a, sum a xh; RMS: sum x^2, sum a x
#pragma unroll
    for (int j = 0; j < G; ++j) {
      float w[8];
      load8_smem(s_w + 8 * (t + j * T), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // past K the weight and dy are zero: nothing of such a column reaches a sum or is stored
        const float x = el(xw[j], e), av = el(yw[j], e) * w[e];
        c1 += kLayer ? av : x * x;
        c2 = fmaf(av, kLayer ? (x - mean) * rstd : x, c2);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      c1 += __shfl_xor_sync(0xffffffffu, c1, o);
      c2 += __shfl_xor_sync(0xffffffffu, c2, o);
    }
    if (lane == 0) s_red[it][warp] = make_float2(c1, c2);
    bar_sync_n(1 + grp, T);  // one barrier a row: s_red[it] is written again only after the next row's barrier
    c1 = c2 = 0.0f;
    for (int i = 0; i < nw; ++i) {
      const float2 v = s_red[it][w0 + i];
      c1 += v.x;
      c2 += v.y;
    }
    c1 = __fdiv_rn(c1, kf);
    c2 = __fdiv_rn(c2, kf);
    if (!kLayer) {
      rstd = __fdiv_rn(1.0f, __fsqrt_rn(c1 + a.eps));
      c2 *= rstd;
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int c = t + j * T;
      float w[8];
      load8_smem(s_w + 8 * c, w);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int e = 2 * i + h;
          const float xn = (el(xw[j], e) - mean) * rstd, dy = el(yw[j], e);  // RMS: mean = 0
          float s = fmaf(dy, w[e], -xn * c2);
          if (kLayer) s -= c1;
          v[h] = s * rstd;
          dwv[j][e] = fmaf(dy, xn, dwv[j][e]);
          if (kLayer) dbv[j][e] += dy;
        }
        o[i] = pack_bf16x2(v[0], v[1]);
      }
      if (c < chunks) store8_bf16(a.dx + row * K, 8 * c, K, vdx, o);
    }
  }
  pdl_launch_dependents();
  // the groups' column sums, added in order of the groups; the last writes the CTA's partial row
#pragma unroll
  for (int p = 0; p < (kLayer ? 2 : 1); ++p) {
    for (int g = 0; g < a.rg; ++g) {
      __syncthreads();
      if (g != grp) continue;
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int k = 8 * (t + j * T) + e;
          if (k >= K) continue;
          const float v = (p ? dbv[j][e] : dwv[j][e]) + (g > 0 ? s_acc[k] : 0.0f);
          if (g + 1 < a.rg)
            s_acc[k] = v;
          else
            a.part[(static_cast<size_t>(blockIdx.x) * (kLayer ? 2 : 1) + p) * K + k] = v;
        }
    }
  }
}

// Rows longer than kNbMaxK, in two kernels.  First dx: a CTA per row, which it
// reads twice; the row's rstd is left for the second (RMSNorm).
template <bool kLayer>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const NbArgs a, float* __restrict__ rstd_out) {
  __shared__ float2 s_red[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = a.K;
  const int64_t row = blockIdx.x;
  const uint16_t* xr = a.x + row * a.ldx;
  const uint16_t* dyr = a.dy + row * a.lddy;
  float mean = 0.0f, rstd = 1.0f;
  if (kLayer) {
    mean = a.mean[row];
    rstd = a.rstd[row];
  }
  float c1 = 0.0f, c2 = 0.0f;
  for (int k = threadIdx.x; k < K; k += 1024) {
    const float x = bf16_bits_to_f32(xr[k]), av = bf16_bits_to_f32(dyr[k]) * a.w[k];
    c1 += kLayer ? av : x * x;
    c2 = fmaf(av, kLayer ? (x - mean) * rstd : x, c2);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    c1 += __shfl_xor_sync(0xffffffffu, c1, o);
    c2 += __shfl_xor_sync(0xffffffffu, c2, o);
  }
  if (lane == 0) s_red[warp] = make_float2(c1, c2);
  __syncthreads();
  c1 = c2 = 0.0f;
  for (int i = 0; i < 32; ++i) {
    c1 += s_red[i].x;
    c2 += s_red[i].y;
  }
  c1 = __fdiv_rn(c1, static_cast<float>(K));
  c2 = __fdiv_rn(c2, static_cast<float>(K));
  if (!kLayer) {
    rstd = __fdiv_rn(1.0f, __fsqrt_rn(c1 + a.eps));
    c2 *= rstd;
    if (threadIdx.x == 0) rstd_out[row] = rstd;
  }
  for (int k = threadIdx.x; k < K; k += 1024) {
    const float xn = (bf16_bits_to_f32(xr[k]) - mean) * rstd;
    float s = fmaf(bf16_bits_to_f32(dyr[k]), a.w[k], -xn * c2);
    if (kLayer) s -= c1;
    const __nv_bfloat16 h = __float2bfloat16_rn(s * rstd);
    a.dx[row * K + k] = *reinterpret_cast<const uint16_t*>(&h);
  }
}

// Then the column sums: a thread per column, gridDim.y slabs of rows.
template <bool kLayer>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NbArgs a, const float* __restrict__ rstd) {
  const int k = blockIdx.x * 256 + threadIdx.x;
  if (k >= a.K) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y) {
    const float dy = bf16_bits_to_f32(a.dy[row * a.lddy + k]);
    const float xn = (bf16_bits_to_f32(a.x[row * a.ldx + k]) - (kLayer ? a.mean[row] : 0.0f)) * rstd[row];
    dw = fmaf(dy, xn, dw);
    db += dy;
  }
  const size_t at = static_cast<size_t>(blockIdx.y) * (kLayer ? 2 : 1) * a.K + k;
  a.part[at] = dw;
  if (kLayer) a.part[at + a.K] = db;
}

// Column sums of part [P][cols]: out[c] for c < split to o0, the others to o1.
// 32 columns a CTA; its 32 warps take the rows w, w + 32, ... and their sums
// are added in order of the warps.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* __restrict__ part, int P, int64_t cols,
                                                           int64_t split, float* __restrict__ o0,
                                                           float* __restrict__ o1) {
  __shared__ float s[32][33];
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float v = 0.0f;
  if (c < cols)
    for (int p = warp; p < P; p += 32) v += part[static_cast<size_t>(p) * cols + c];
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < cols) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][lane];
    if (c < split)
      o0[c] = v;
    else if (o1)
      o1[c - split] = v;
  }
}

// ----------------------------------------------------------------- 8-bit checkpoints
// The value a code stands for: RN(q * RN(gamma / 127)).

// y = RNbf16 of it: the activation, restored in its own type.  A CTA of 256
// threads takes 256 / lanes rows, `lanes` threads a row, 16 codes each a step.
__global__ void __launch_bounds__(256) dequant_act_kernel(const int8_t* __restrict__ q, int64_t ldq,
                                                          const float* __restrict__ gamma, int M, int K,
                                                          uint16_t* __restrict__ y, int lanes) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int r = threadIdx.x / lanes, t = threadIdx.x - r * lanes;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / lanes) + r;
  if (row >= M) return;
  const float s = __fdiv_rn(gamma[row], kQb);
  const bool qv = (ldq % 16) == 0 && (reinterpret_cast<uintptr_t>(q) & 15u) == 0;
  const bool yv = (K % 8) == 0 && (reinterpret_cast<uintptr_t>(y) & 15u) == 0;
  for (int k0 = 16 * t; k0 < K; k0 += 16 * lanes) {
    uint32_t w[4], o[8];
    load16_codes(q + row * ldq, k0, K, qv, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[4];
      codes4_f32(w[i], f);
      o[2 * i] = pack_bf16x2(__fmul_rn(f[0], s), __fmul_rn(f[1], s));
      o[2 * i + 1] = pack_bf16x2(__fmul_rn(f[2], s), __fmul_rn(f[3], s));
    }
    store8_bf16(y + row * K, k0, K, yv, o);
    store8_bf16(y + row * K, k0 + 8, K, yv, o + 4);
  }
}

// The gate's forward value h = RNb(RNb(max(g, 0)^2) u) of a training step,
// with everything the backward pass and the down projection need kept in 8
// bits: the codes of g, u and h, each with its row's absmax.
struct GluSaveArgs {
  const uint16_t* g;
  int64_t ldg;
  const uint16_t* u;
  int64_t ldu;
  int M, N;
  int8_t *qg, *qu, *qh;                // [M, N]
  float *gg, *gu, *gh;                 // [M]
  int32_t* rowsum;                     // [M] sums of h's codes, or null
  int wpr;
};

// Warps and groups as in layernorm_kernel.
template <int G>
__global__ void __launch_bounds__(32 * kQuantWarps, G <= 2 ? 3 : 2) relu2_glu_quant_kernel(const GluSaveArgs a) {
  __shared__ uint32_t s_mx[3][kQuantWarps];
  __shared__ int32_t s_sum[kQuantWarps];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = a.wpr, N = a.N;
  const int rloc = warp / wpr, sub = warp - rloc * wpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kQuantWarps / wpr) + rloc;
  const bool active = row < a.M;
  const uint16_t* gr = a.g + (active ? row : 0) * a.ldg;
  const uint16_t* ur = a.u + (active ? row : 0) * a.ldu;
  const bool vg = (a.ldg % 8) == 0 && (reinterpret_cast<uintptr_t>(a.g) & 15u) == 0;
  const bool vu = (a.ldu % 8) == 0 && (reinterpret_cast<uintptr_t>(a.u) & 15u) == 0;
  const int groups = (N + 15) / 16, gstride = 32 * wpr, g0 = sub * 32 + lane;
  const bool in_regs = groups <= G * gstride;

  uint32_t v[G][16];  // g then u
  auto load = [&](int g, uint32_t (&r)[16]) {
    uint32_t t[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      load8_raw(h < 2 ? gr : ur, 16 * g + 8 * (h & 1), N, h < 2 ? vg : vu, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[4 * h + i] = t[i];
    }
  };
  if (active && in_regs) {
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (g0 + j * gstride < groups) load(g0 + j * gstride, v[j]);
  }
  auto for_groups = [&](auto&& f) {
    if (!active) return;
    if (in_regs) {
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (g0 + j * gstride < groups) f(g0 + j * gstride, v[j]);
    } else {
      for (int g = g0; g < groups; g += gstride) {
        uint32_t r[16];
        load(g, r);
        f(g, r);
      }
    }
  };
  auto hword = [](uint32_t g, uint32_t u) {  // two elements
    return relu2_glu_bf16(static_cast<uint16_t>(g), static_cast<uint16_t>(u)) |
           (static_cast<uint32_t>(relu2_glu_bf16(static_cast<uint16_t>(g >> 16), static_cast<uint16_t>(u >> 16))) << 16);
  };
  // |x| as bit patterns order like the values
  uint32_t mx[3] = {0u, 0u, 0u};
  for_groups([&](int, const uint32_t (&r)[16]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w[3] = {r[i], r[8 + i], hword(r[i], r[8 + i])};
#pragma unroll
      for (int p = 0; p < 3; ++p) mx[p] = max(mx[p], max((w[p] << 16) & 0x7FFF0000u, w[p] & 0x7FFF0000u));
    }
  });
#pragma unroll
  for (int p = 0; p < 3; ++p) mx[p] = __reduce_max_sync(0xffffffffu, mx[p]);
  if (wpr > 1) {
    if (lane == 0)
      for (int p = 0; p < 3; ++p) s_mx[p][warp] = mx[p];
    __syncthreads();
    for (int i = 0; i < wpr; ++i)
#pragma unroll
      for (int p = 0; p < 3; ++p) mx[p] = max(mx[p], s_mx[p][rloc * wpr + i]);
  }
  float c[3], d[3];
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    d[p] = __fadd_rn(__uint_as_float(mx[p]), kEps);
    c[p] = __fmul_rn(kQb, __frcp_rn(d[p]));
  }
  int32_t sum = 0;
  const size_t at = static_cast<size_t>(active ? row : 0) * N;
  const bool vq = (N % 16) == 0 && ((reinterpret_cast<uintptr_t>(a.qg) | reinterpret_cast<uintptr_t>(a.qu) |
                                     reinterpret_cast<uintptr_t>(a.qh)) & 15u) == 0;
  for_groups([&](int g, const uint32_t (&r)[16]) {
    int8_t* const out[3] = {a.qg + at, a.qu + at, a.qh + at};
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      uint32_t r0[4], r1[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r0[i] = p < 2 ? r[8 * p + i] : hword(r[i], r[8 + i]);
        r1[i] = p < 2 ? r[8 * p + 4 + i] : hword(r[4 + i], r[12 + i]);
      }
      int32_t sm = 0;
      const uint4 w = group_codes<false>(r0, r1, c[p], d[p], sm);
      if (p == 2) sum += sm;
      store16_codes(out[p], 16 * g, N, vq, w);
    }
  });
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (wpr > 1) {
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    sum = 0;
    for (int i = 0; i < wpr; ++i) sum += s_sum[rloc * wpr + i];
  }
  if (active && sub == 0 && lane == 0) {
    a.gg[row] = __uint_as_float(mx[0]);
    a.gu[row] = __uint_as_float(mx[1]);
    a.gh[row] = __uint_as_float(mx[2]);
    if (a.rowsum) a.rowsum[row] = sum;
  }
}

// dg = RNb(2 dh r u~), du = RNb(dh r^2) with g~, u~ the values the codes stand
// for and r = max(g~, 0); rows and lanes as in dequant_act_kernel.
__global__ void __launch_bounds__(256) relu2_glu_backward_kernel(
    const uint16_t* __restrict__ dh, int64_t lddh, const int8_t* __restrict__ qg, const float* __restrict__ gg,
    const int8_t* __restrict__ qu, const float* __restrict__ gu, int M, int N, uint16_t* __restrict__ dg,
    uint16_t* __restrict__ du, int lanes) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int r = threadIdx.x / lanes, t = threadIdx.x - r * lanes;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / lanes) + r;
  if (row >= M) return;
  const float sg = __fdiv_rn(gg[row], kQb), su = __fdiv_rn(gu[row], kQb);
  const bool vq = (N % 16) == 0 && ((reinterpret_cast<uintptr_t>(qg) | reinterpret_cast<uintptr_t>(qu)) & 15u) == 0;
  const bool vh = (lddh % 8) == 0 && (reinterpret_cast<uintptr_t>(dh) & 15u) == 0;
  const bool vo = (N % 8) == 0 && ((reinterpret_cast<uintptr_t>(dg) | reinterpret_cast<uintptr_t>(du)) & 15u) == 0;
  const uint16_t* dhr = dh + row * lddh;
  const size_t at = static_cast<size_t>(row) * N;
  for (int k0 = 16 * t; k0 < N; k0 += 16 * lanes) {
    uint32_t wg[4], wu[4], h0[4], h1[4];
    load16_codes(qg + at, k0, N, vq, wg);
    load16_codes(qu + at, k0, N, vq, wu);
    load8_raw(dhr, k0, N, vh, h0);
    load8_raw(dhr, k0 + 8, N, vh, h1);
    uint32_t og[8], ou[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float fg[4], fu[4], a[4], b[4];
      codes4_f32(wg[i], fg);
      codes4_f32(wu[i], fu);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t hw = i < 2 ? h0[2 * i + (e >> 1)] : h1[2 * (i - 2) + (e >> 1)];
        const float d = (e & 1) ? bf16_hi(hw) : bf16_lo(hw);
        const float rp = fmaxf(__fmul_rn(fg[e], sg), 0.0f);
        const float dr = d * rp;
        a[e] = 2.0f * dr * __fmul_rn(fu[e], su);
        b[e] = dr * rp;
      }
      og[2 * i] = pack_bf16x2(a[0], a[1]);
      og[2 * i + 1] = pack_bf16x2(a[2], a[3]);
      ou[2 * i] = pack_bf16x2(b[0], b[1]);
      ou[2 * i + 1] = pack_bf16x2(b[2], b[3]);
    }
    store8_bf16(dg + at, k0, N, vo, og);
    store8_bf16(dg + at, k0 + 8, N, vo, og + 4);
    store8_bf16(du + at, k0, N, vo, ou);
    store8_bf16(du + at, k0 + 8, N, vo, ou + 4);
  }
}

}  // namespace bl
