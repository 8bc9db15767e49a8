// train_rows.cuh -- row-wise kernels of BitLinear's training side: layer norm
// forward (to bf16 or to the 8-bit codes a BitLinear reads), the backward
// passes of layer norm and RMSNorm, the 8-bit checkpoint of the squared-ReLU
// gated FFN with the backward pass that reads it, and the restored activation.
//
// Every input is read once and every output written once, with a few operations
// per element.  What bounds them: memory for the restored activation and the
// gate's gradients (the copy rate at 4096 x 11008), latency between a row's
// passes for the layer norm, instructions for the codes of three matrices and
// for the norm gradients, both near half of the issue slots.
#pragma once
#include "gemv.cuh"

namespace bl {

// ----------------------------------------------------------------- helpers
// Everything here walks rows in chunks of 8 columns, 16 bytes of bf16 a lane,
// and computes two columns an instruction (float2).

__device__ __forceinline__ float2 splat2(float v) { return make_float2(v, v); }

// The larger of two, NaN if either is: a row's maximum must not hide one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 8 fp32 parameters from k0 (zero past K); one 32-byte load where p is 32-byte aligned.
__device__ __forceinline__ void load8_f32(const float* p, int k0, int K, bool vec, float2 (&v)[4]) {
  if (vec && k0 + 8 <= K) {
    uint32_t r[8];
    ld_global_nc_v8(p + k0, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i].x = k0 + 2 * i < K ? p[k0 + 2 * i] : 0.0f;
      v[i].y = k0 + 2 * i + 1 < K ? p[k0 + 2 * i + 1] : 0.0f;
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float2 bf16_2(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

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

// The same for rows of any alignment, whole words where the address allows.
__device__ __forceinline__ void store8_bf16_any(uint16_t* row, int k0, int K, const uint32_t* o) {
  uint16_t* p = row + k0;
  if (k0 + 8 > K) {
    store8_bf16(row, k0, K, false, o);
  } else if ((reinterpret_cast<uintptr_t>(p) & 2u) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(p)[i] = o[i];
  } else {
    p[0] = static_cast<uint16_t>(o[0]);
#pragma unroll
    for (int i = 0; i < 3; ++i) reinterpret_cast<uint32_t*>(p + 1)[i] = __funnelshift_r(o[i], o[i + 1], 16);
    p[7] = static_cast<uint16_t>(o[3] >> 16);
  }
}

// 8 bf16 values of a row from k0 as 4 words (zero past K), rows of any
// alignment: the two 16-byte blocks that hold them, shifted into place, unless
// a block reaches out of the matrix [lo, hi) (its first and last ones).  A row
// element by element took three to eleven times the aligned one's time.
__device__ __forceinline__ void load8_any(const uint16_t* row, int k0, int K, const uint16_t* lo, const uint16_t* hi,
                                          uint32_t (&r)[4]) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(row + k0), a = p & ~static_cast<uintptr_t>(15);
  const uint32_t s = static_cast<uint32_t>(p & 15u);
  const uintptr_t b = s ? a + 16 : a;
  if (a < reinterpret_cast<uintptr_t>(lo) || b + 16 > reinterpret_cast<uintptr_t>(hi)) {
    load8_raw(row, k0, K, false, r);
    return;
  }
  const uint4 x = *reinterpret_cast<const uint4*>(a), y = *reinterpret_cast<const uint4*>(b);
  uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  if (s & 8u)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (s & 4u)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (s & 2u) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
  if (k0 + 8 > K) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = k0 + 2 * i >= K ? 0u : k0 + 2 * i + 1 >= K ? r[i] & 0xFFFFu : r[i];
  }
}

// 8 codes at row[k0 ..], those past K left out; vec: the row's chunks are 8-byte aligned, else the widest stores that
// the address allows (bytes alone: 72 us for the three codes of 4096 x 2561).
__device__ __forceinline__ void store8_codes(int8_t* row, int k0, int K, bool vec, const uint2 w) {
  int8_t* p = row + k0;
  if (k0 + 8 > K) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k0 + i < K) p[i] = static_cast<int8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  } else if (vec) {
    *reinterpret_cast<uint2*>(p) = w;
  } else {
    const uint32_t m = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 3u;
    if (m == 0) {
      reinterpret_cast<uint32_t*>(p)[0] = w.x;
      reinterpret_cast<uint32_t*>(p)[1] = w.y;
    } else if (m == 2) {
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w.x);
      *reinterpret_cast<uint32_t*>(p + 2) = __funnelshift_r(w.x, w.y, 16);
      *reinterpret_cast<uint16_t*>(p + 6) = static_cast<uint16_t>(w.y >> 16);
    } else if (m == 1) {
      p[0] = static_cast<int8_t>(w.x);
      *reinterpret_cast<uint16_t*>(p + 1) = static_cast<uint16_t>(w.x >> 8);
      *reinterpret_cast<uint32_t*>(p + 3) = __funnelshift_r(w.x, w.y, 24);
      p[7] = static_cast<int8_t>(w.y >> 24);
    } else {
      p[0] = static_cast<int8_t>(w.x);
      *reinterpret_cast<uint32_t*>(p + 1) = __funnelshift_r(w.x, w.y, 8);
      *reinterpret_cast<uint16_t*>(p + 5) = static_cast<uint16_t>(w.y >> 8);
      p[7] = static_cast<int8_t>(w.y >> 24);
    }
  }
}

// 16 codes from row[k0 ..] (zero past K), one by one.
__device__ __forceinline__ void load16_codes(const int8_t* row, int k0, int K, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k0 + 4 * i + j < K) w[i] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k0 + 4 * i + j])) << (8 * j);
  }
}

// The same for rows of any alignment inside [lo, hi), as load8_any.
__device__ __forceinline__ void load16_codes_any(const int8_t* row, int k0, int K, const int8_t* lo, const int8_t* hi,
                                                 uint32_t (&r)[4]) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(row + k0), a = p & ~static_cast<uintptr_t>(15);
  const uint32_t s = static_cast<uint32_t>(p & 15u);
  const uintptr_t b = s ? a + 16 : a;
  if (k0 + 16 > K || a < reinterpret_cast<uintptr_t>(lo) || b + 16 > reinterpret_cast<uintptr_t>(hi)) {
    load16_codes(row, k0, K, r);
    return;
  }
  const uint4 x = *reinterpret_cast<const uint4*>(a), y = *reinterpret_cast<const uint4*>(b);
  uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  if (s & 8u)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (s & 4u)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __funnelshift_r(w[i], w[i + 1], 8 * (s & 3u));
}

// Four int8 codes as fp32, exactly: the code plus 128 goes into the low byte
// of 2^23, whose last place is 1.
__device__ __forceinline__ void codes4_f32(uint32_t w, float2 (&f)[2]) {
  const uint32_t u = w ^ 0x80808080u;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    f[j] = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + 2 * j)),
                                  __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441 + 2 * j))),
                      splat2(-8388736.0f));
}

// Four codes from the low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
  return __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410);
}
__device__ __forceinline__ int32_t code_sum(const uint2 w) {
  return __dp4a(static_cast<int>(w.y), 0x01010101, __dp4a(static_cast<int>(w.x), 0x01010101, 0));
}

// The codes of 8 values by codes8f's division-free rounding, two values an
// instruction.  emax grows to the largest distance to a code; past kCodesNear
// some value lies so near the middle of two codes that codes8_exact has to
// decide.  The two are apart because the exact one is long and rare (one chunk
// in a thousand): inlined into every chunk's step it filled the instruction
// cache (a fifth of the stalls of a 4096 x 2560 layer norm).
constexpr float kCodesNear = 0.5f - 6.103515625e-05f;
__device__ __forceinline__ uint2 codes8_near(const float2 (&v)[4], float c, float& emax) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 sm = __ffma2_rn(v[i], splat2(c), splat2(kMagic));
    const float2 e = __ffma2_rn(v[i], splat2(-c), __fadd2_rn(sm, splat2(-kMagic)));
    emax = fmaxf(emax, fmaxf(fabsf(e.x), fabsf(e.y)));
    b[2 * i] = __float_as_uint(sm.x);
    b[2 * i + 1] = __float_as_uint(sm.y);
  }
  return make_uint2(low_bytes(b[0], b[1], b[2], b[3]), low_bytes(b[4], b[5], b[6], b[7]));
}
__device__ __forceinline__ uint2 codes8_exact(const float2 (&v)[4], float d) {
  uint32_t b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    b[e] = static_cast<uint32_t>(__float2int_rn(__fdiv_rn(__fmul_rn((e & 1) ? v[e >> 1].y : v[e >> 1].x, kQb), d)));
  return make_uint2(low_bytes(b[0], b[1], b[2], b[3]), low_bytes(b[4], b[5], b[6], b[7]));
}

// ----------------------------------------------------------------- layer norm
// Per row: s1 = sum x, s2 = sum x^2 in fp64; mean = RN32(s1 / K), var = RN32(max(0, (K s2 - s1^2) / K^2)), rstd = RN32(1 /
// sqrt(var + eps)), each computed in fp64 (1 / K rounded there once, so that no quotient stands in a row's way).  The
// one-pass variance loses nothing that a two-pass one would keep: if all entries lie within a factor of two of each
// other, they are multiples of one 2^e below 2^9 of it, and with K <= 2^16 both K s2 and s1^2 are whole numbers below
// 2^53 of 4^e, their difference exact (0 for a constant row; s2 - s1^2 / K, with its rounded quotient, gave rows of 1e6
// a variance of up to 5e-5 and rows of 1e30 an infinite one); otherwise the two are 2^-19 apart or more, which leaves
// 34 of 53 bits.  Then
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
  int lw;          // log2 of the warps per row
  double dk;       // K
  double inv_k;    // 1 / K
};

// A row belongs to wpr warps of a 256-thread CTA; a lane owns the 8-wide
// chunks c = sub * 32 + lane + j * 32 * wpr, at most G of them, in registers:
// the row is read once, all its loads in flight together, and with codes its
// normalised values stay in registers between the maximum and the rounding, so
// the parameters are read once a row as well (read twice, 16 columns a lane,
// they filled the L1 pipe for 42 us at 4096 x 2560).  Without kAny (rows and
// parameters that 16- and 32-byte loads can take, K % 8 == 0) no load is
// conditional, so that those of several chunks go out together: chunks past K
// read the last one and are left out of sums, maximum and output.
// G = 0: rows longer than any G holds are read again for each pass, from L2.
template <bool kCodes, bool kAny, int G>
__global__ void __launch_bounds__(32 * kQuantWarps, G >= 1 && G <= 4 ? 3 : 2) layernorm_kernel(const LnArgs a) {
  constexpr bool kRegs = G > 0;
  constexpr int GR = kRegs ? G : 1;
  __shared__ double s_s1[kQuantWarps], s_s2[kQuantWarps];
  __shared__ float s_mx[kQuantWarps];
  __shared__ int32_t s_sum[kQuantWarps];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = 1 << a.lw, K = a.K;
  const int rloc = warp >> a.lw, sub = warp & (wpr - 1);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kQuantWarps >> a.lw) + rloc;
  const bool active = row < a.M;  // inactive warps still reach the CTA barriers
  const uint16_t* xr = a.x + (active ? row : 0) * a.ldx;
  const uint16_t* const end = a.x + static_cast<int64_t>(a.M - 1) * a.ldx + K;
  const bool wvec = !kAny || (reinterpret_cast<uintptr_t>(a.w) & 31u) == 0;
  const bool bvec = !kAny || (reinterpret_cast<uintptr_t>(a.b) & 31u) == 0;
  auto load = [&](int c, uint32_t (&r)[4]) {
    if (kAny) {
      load8_any(xr, 8 * c, K, a.x, end, r);
    } else {
      const uint4 t = *reinterpret_cast<const uint4*>(xr + 8 * c);
      r[0] = t.x; r[1] = t.y; r[2] = t.z; r[3] = t.w;
    }
  };
  const int chunks = (K + 7) / 8;
  const int cstride = 32 * wpr;
  const int c0 = sub * 32 + lane;

  uint32_t v[GR][4];
  if (kRegs) {
#pragma unroll
    for (int j = 0; j < GR; ++j) load(min(c0 + j * cstride, chunks - 1), v[j]);
  }
  // f(j, chunk, its words) for each of the lane's chunks, and with G > 0 for those past K too
  auto for_chunks = [&](auto&& f) {
    if constexpr (kRegs) {
#pragma unroll
      for (int j = 0; j < GR; ++j) f(j, c0 + j * cstride, v[j]);
    } else if (active) {
      for (int c = c0; c < chunks; c += cstride) {
        uint32_t r[4];
        load(c, r);
        f(0, c, r);
      }
    }
  };

  double t1[2] = {0.0, 0.0}, t2[2] = {0.0, 0.0};  // two chains of additions each
  for_chunks([&](int, int c, const uint32_t (&r)[4]) {  // zero past K
    if (c >= chunks) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double x[2] = {static_cast<double>(bf16_lo(r[i])), static_cast<double>(bf16_hi(r[i]))};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        t1[h] += x[h];
        t2[h] = __fma_rn(x[h], x[h], t2[h]);
      }
    }
  });
  double s1 = t1[0] + t1[1], s2 = t2[0] + t2[1];
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
  const float mean = __double2float_rn(s1 * a.inv_k);
  const double vard = (a.dk * s2 - s1 * s1) * a.inv_k * a.inv_k;
  const float var = __double2float_rn(vard < 0.0 ? 0.0 : vard);  // NaN stays NaN
  const float rstd = __double2float_rn(rsqrt(static_cast<double>(var) + static_cast<double>(a.eps)));
  if (active && sub == 0 && lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }

  // a chunk's normalised values
  auto normed = [&](int c, const uint32_t (&r)[4], float2 (&xn)[4]) {
    float2 w[4], b[4];
    load8_f32(a.w, 8 * c, K, wvec, w);
    if (a.b) load8_f32(a.b, 8 * c, K, bvec, b);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      xn[i] = __fmul2_rn(__fmul2_rn(__fadd2_rn(bf16_2(r[i]), splat2(-mean)), splat2(rstd)), w[i]);
    if (a.b)
#pragma unroll
      for (int i = 0; i < 4; ++i) xn[i] = __fadd2_rn(xn[i], b[i]);
  };
  const bool qvec = !kAny || ((K % 8) == 0 && (reinterpret_cast<uintptr_t>(a.q) & 7u) == 0);

  if (!kCodes) {
    uint16_t* yr = a.y + (active ? row : 0) * K;
    for_chunks([&](int, int c, const uint32_t (&r)[4]) {
      float2 xn[4];
      normed(kRegs ? min(c, chunks - 1) : c, r, xn);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(xn[i].x, xn[i].y);
      if (!active || c >= chunks) return;
      if (kAny)
        store8_bf16_any(yr, 8 * c, K, o);
      else
        *reinterpret_cast<uint4*>(yr + 8 * c) = make_uint4(o[0], o[1], o[2], o[3]);
    });
    return;
  }

  float2 xs[kCodes ? GR : 1][4];  // kept between the passes (G > 0)
  float mx = 0.0f;
  for_chunks([&](int j, int c, const uint32_t (&r)[4]) {
    float2(&xn)[4] = xs[kCodes ? j : 0];
    normed(kRegs ? min(c, chunks - 1) : c, r, xn);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_nan(m, max_nan(fabsf(xn[i].x), fabsf(xn[i].y)));
    mx = c < chunks ? max_nan(mx, m) : mx;
  });
  mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
  if (wpr > 1) {
    if (lane == 0) s_mx[warp] = mx;
    __syncthreads();
    for (int i = 0; i < wpr; ++i) mx = max_nan(mx, s_mx[rloc * wpr + i]);
  }
  const float d = __fadd_rn(mx, kEps);
  const float c127 = __fmul_rn(kQb, __frcp_rn(d));
  int32_t sum = 0;
  uint32_t redo = 0u;  // chunks whose codes take the exact quotient
  int8_t* qr = a.q + (active ? row : 0) * K;
  auto exact = [&](int c) {  // replaces the chunk's codes
    uint32_t r[4];
    float2 xn[4];
    load(c, r);
    normed(c, r, xn);
    float emax = 0.0f;
    const uint2 w = codes8_exact(xn, d);
    sum += code_sum(w) - code_sum(codes8_near(xn, c127, emax));
    store8_codes(qr, 8 * c, K, qvec, w);
  };
  for_chunks([&](int j, int c, const uint32_t (&r)[4]) {
    float2(&xn)[4] = xs[kCodes ? j : 0];
    if (!kRegs) normed(c, r, xn);
    float emax = 0.0f;
    const uint2 w = codes8_near(xn, c127, emax);
    if (!active || c >= chunks) return;
    sum += code_sum(w);
    store8_codes(qr, 8 * c, K, qvec, w);
    if (emax > kCodesNear) {
      if (kRegs)
        redo |= 1u << j;
      else
        exact(c);
    }
  });
  while (kRegs && redo) {
    const int c = c0 + (__ffs(redo) - 1) * cstride;
    redo &= redo - 1;
    exact(c);
  }
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
// What a row costs beside its columns (two sums across the group, a barrier,
// the quotients) is paid per warp, so few threads with several chunks each and
// more groups beside each other beat one wide group.
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

// Chunks a thread (G) and the most threads of a CTA, by what fits the registers:
// 16 G of column sums (layer norm), 16 G of the row's values, 8 G of the next
// row's words.  Measured (us, layer norm / RMSNorm, both launches, before the
// running row pointers, with which G = 2 takes 17.2 / 15.8 at 4096 x 2560):
//   M x K          G = 1 (768)   G = 2 (512)   G = 4 (384)
//   4096 x 2560    19.7 / 19.0   18.8 / 17.0   28.1 / 20.9
//   256 x 2560      6.8 / 6.1     7.6 / 6.6    11.3 / 8.6
//   8192 x 640     14.1 / 12.5   15.6 / 13.5   25.0 / 17.8
//   999 x 11008        --        39.9 / 29.7 (768 threads)   39.3 / 24.6
__host__ __device__ constexpr int nb_max_threads(int G) { return G == 1 ? 768 : G == 2 ? 512 : 384; }
constexpr int kNbMaxGroups = 8;                                // one named barrier each
constexpr int kNbMaxWarps = 24;                                // of a group
constexpr int kNbMaxK = 8 * 4 * nb_max_threads(4);             // longer rows take the split kernels

// RMSNorm of a row whose squares fp32 cannot add up (mean square beyond 2^100 or, with next to no eps, below 2^-100): r
// and mean_k(a xh) with sums in fp64, which hold the square of every bf16 value.  Called by whole warps, each of which
// reads the row again by itself.
constexpr uint32_t kRmsLow = 0x0D800000u, kRmsHigh = 0x71800000u;  // bits of 2^-100 and 2^100
constexpr uint32_t kRmsMark = 0xFFFFFFFFu;  // two bf16 that no conversion gives: its NaN is 0x7FFF
__device__ __forceinline__ bool rms_far(float m) { return __float_as_uint(m) - kRmsLow > kRmsHigh - kRmsLow; }
__device__ __forceinline__ float rsqrt_normal(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __noinline__ float2 rms_far_row(const uint16_t* x, const uint16_t* dy, const float* w, int K, float eps) {
  const int lane = threadIdx.x & 31;
  auto sum = [](double v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  double ss = 0.0, c = 0.0;
  for (int k = lane; k < K; k += 32) {
    const double v = bf16_bits_to_f32(x[k]);
    ss = __fma_rn(v, v, ss);
  }
  const double r = 1.0 / sqrt(sum(ss) / K + static_cast<double>(eps));
  for (int k = lane; k < K; k += 32)
    c = __fma_rn(static_cast<double>(bf16_bits_to_f32(dy[k])) * w[k], bf16_bits_to_f32(x[k]) * r, c);
  return make_float2(__double2float_rn(r), __double2float_rn(sum(c) / K));
}

// kFast: 16-byte accesses everywhere (columns past K, a whole chunk then, are read from the last chunk and zeroed).
template <bool kLayer, bool kFast, int G>
__global__ void __launch_bounds__(nb_max_threads(G), 1) norm_backward_kernel(const NbArgs a) {
  // [2][P] float4: the weight's columns 8 c .. 8 c + 3 and 8 c + 4 .. 8 c + 7 of each chunk, zero past K; then the
  // same shape of column sums, handed from group to group (rg > 1)
  extern __shared__ float4 s_nb[];
  __shared__ __align__(16) float2 s_red[2][kNbMaxGroups][kNbMaxWarps];  // sums of a group's warps, then one zero
  constexpr int P = G * nb_max_threads(G);  // float4 of a plane
  constexpr bool kAhead = !(kLayer && G == 4);  // the next row's words fit the registers
  const int T = a.T, K = a.K;
  float4* s_acc = s_nb + 2 * P;
  for (int k = threadIdx.x; k < 8 * G * T; k += blockDim.x)
    reinterpret_cast<float*>(s_nb)[4 * ((k & 4 ? P : 0) + (k >> 3)) + (k & 3)] = k < K ? a.w[k] : 0.0f;
  const int grp = threadIdx.x / T, t = threadIdx.x - grp * T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gw = warp - grp * (T / 32), nw = T / 32;
  for (int i = threadIdx.x; i < 2 * kNbMaxGroups * kNbMaxWarps; i += blockDim.x) (&s_red[0][0][0])[i] = splat2(0.0f);
  const int chunks = (K + 7) / 8;
  const uint16_t* const xend = a.x + static_cast<int64_t>(a.M - 1) * a.ldx + K;
  const uint16_t* const yend = a.dy + static_cast<int64_t>(a.M - 1) * a.lddy + K;
  const float inv_k = __fdiv_rn(1.0f, static_cast<float>(K));
  const int64_t stride = static_cast<int64_t>(gridDim.x) * a.rg;

  float2 dwv[G][4], dbv[G][4];
#pragma unroll
  for (int j = 0; j < G; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) dwv[j][i] = dbv[j][i] = splat2(0.0f);
  uint32_t nx[G][4], ny[G][4];  // the next row's words
  float nmean = 0.0f, nrstd = 1.0f;
  bool far = false;  // RMSNorm: some row was put off (rms_far); it adds nothing here and is marked in dx
  int64_t row = static_cast<int64_t>(blockIdx.x) * a.rg + grp;
  // the thread's first chunk of the row to load next and of the row to write, and the steps between a group's rows
  const uint16_t* px = a.x + row * a.ldx + 8 * t;
  const uint16_t* py = a.dy + row * a.lddy + 8 * t;
  uint16_t* pd = a.dx + row * K + 8 * t;
  const int64_t sx = stride * a.ldx, sy = stride * a.lddy, sd = stride * K;
  auto load = [&](int64_t row) {  // advances px and py
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int c = t + j * T;
      if (kFast) {
        const int at = 8 * j * T - (j == G - 1 && c >= chunks ? 8 * (c - chunks + 1) : 0);
        const uint4 p = *reinterpret_cast<const uint4*>(px + at);
        const uint4 q = *reinterpret_cast<const uint4*>(py + at);
        nx[j][0] = p.x; nx[j][1] = p.y; nx[j][2] = p.z; nx[j][3] = p.w;
        ny[j][0] = q.x; ny[j][1] = q.y; ny[j][2] = q.z; ny[j][3] = q.w;
      } else if (c < chunks) {
        load8_any(px - 8 * t, 8 * c, K, a.x, xend, nx[j]);
        load8_any(py - 8 * t, 8 * c, K, a.dy, yend, ny[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) nx[j][i] = ny[j][i] = 0u;
      }
    }
    px += sx;
    py += sy;
    if (kLayer) {
      nmean = a.mean[row];
      nrstd = a.rstd[row];
    }
  };
  auto weight = [&](int j, float2 (&w)[4]) {
    const float4 p = s_nb[t + j * T], q = s_nb[P + t + j * T];
    w[0] = make_float2(p.x, p.y);
    w[1] = make_float2(p.z, p.w);
    w[2] = make_float2(q.x, q.y);
    w[3] = make_float2(q.z, q.w);
  };
  __syncthreads();
  if (kAhead && row < a.M) load(row);
  for (int it = 0; row < a.M; row += stride, it ^= 1) {
    if (!kAhead) load(row);
    const float mean = nmean;
    float rstd = nrstd;
    float2 xf[G][4], yf[G][4];  // layer: xh; RMS: x.  And dy
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const bool past = kFast && j == G - 1 && t + j * T >= chunks;  // only the last chunk can be: (G - 1) T < chunks
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xf[j][i] = bf16_2(past ? 0u : nx[j][i]);
        yf[j][i] = bf16_2(past ? 0u : ny[j][i]);
        if (kLayer) xf[j][i] = __fmul2_rn(__fadd2_rn(xf[j][i], splat2(-mean)), splat2(rstd));
      }
    }
    if (kAhead && row + stride < a.M) load(row + stride);  // in flight while this row's sums go round
    float2 p1 = splat2(0.0f), p2 = splat2(0.0f);  // layer: sum a, sum a xh; RMS: sum x^2, sum a x
#pragma unroll
    for (int j = 0; j < G; ++j) {
      float2 w[4];
      weight(j, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // past K the weight and dy are zero: nothing of such a column reaches a sum or is stored
        const float2 av = __fmul2_rn(yf[j][i], w[i]);
        p1 = kLayer ? __fadd2_rn(p1, av) : __ffma2_rn(xf[j][i], xf[j][i], p1);
        p2 = __ffma2_rn(av, xf[j][i], p2);
      }
    }
    float c1 = p1.x + p1.y, c2 = p2.x + p2.y;
    {  // both sums in one butterfly: the lower half-warp's lanes take the first, the upper's the second
      float v = lane < 16 ? c1 : c2;
      v += __shfl_xor_sync(0xffffffffu, lane < 16 ? c2 : c1, 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      c1 = v;
    }
    if (nw > 1) {
      if ((lane & 15) == 0) reinterpret_cast<float*>(&s_red[it][grp][gw])[lane >> 4] = c1;
      bar_sync_n(1 + grp, T);  // one barrier a row: s_red[it] is written again only after the next row's barrier
      c1 = c2 = 0.0f;
      for (int i = 0; i < nw; i += 2) {
        const float4 v = *reinterpret_cast<const float4*>(&s_red[it][grp][i]);
        c1 += v.x + v.z;
        c2 += v.y + v.w;
      }
    } else {
      c2 = __shfl_sync(0xffffffffu, c1, 16);
      c1 = __shfl_sync(0xffffffffu, c1, 0);
    }
    c1 *= inv_k;
    c2 *= inv_k;
    bool out = false;
    if (!kLayer) {
      const float m = c1 + a.eps;
      out = rms_far(m);
      rstd = out ? 0.0f : rsqrt_normal(m);  // within 2 ulp, as good as the sums
      c2 *= rstd * rstd;                    // against x instead of xh
      far |= out;
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int c = t + j * T;
      float2 w[4];
      weight(j, w);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 s = __ffma2_rn(xf[j][i], splat2(-c2), __fmul2_rn(yf[j][i], w[i]));
        if (kLayer) s = __fadd2_rn(s, splat2(-c1));
        s = __fmul2_rn(s, splat2(rstd));
        const float2 xh = kLayer ? xf[j][i] : __fmul2_rn(xf[j][i], splat2(rstd));
        dwv[j][i] = __ffma2_rn(yf[j][i], xh, dwv[j][i]);
        if (kLayer) dbv[j][i] = __fadd2_rn(dbv[j][i], yf[j][i]);
        o[i] = pack_bf16x2(s.x, s.y);
      }
      if (j == 0 && out) o[0] = kRmsMark;
      if (kFast) {
        if (j < G - 1 || c < chunks) *reinterpret_cast<uint4*>(pd + 8 * j * T) = make_uint4(o[0], o[1], o[2], o[3]);
      } else if (c < chunks) {
        store8_bf16_any(pd - 8 * t, 8 * c, K, o);
      }
    }
    pd += sd;
  }
  if (!kLayer && far) {  // the same for the whole group
    // the rows put off, known by their first entry; here, since the same branch inside the rows above costs them time
    // even where none takes it (4096 x 2560: 15.4 us, so 14.7, without any such rows 14.3; 8192 x 640: 13.1, 11.5, 11.5)
    bar_sync_n(1 + grp, T);
#pragma unroll 1
    for (row = static_cast<int64_t>(blockIdx.x) * a.rg + grp; row < a.M; row += stride) {
      const uint16_t *xr = a.x + row * a.ldx, *yr = a.dy + row * a.lddy;
      uint16_t* const dr = a.dx + row * K;
      if (*dr != static_cast<uint16_t>(kRmsMark)) continue;
      bar_sync_n(1 + grp, T);  // every warp has read the mark
      const float2 v = rms_far_row(xr, yr, a.w, K, a.eps);
#pragma unroll
      for (int j = 0; j < G; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int k = 8 * (t + j * T) + e;
          if (k < K) {
            const float xh = bf16_bits_to_f32(xr[k]) * v.x, dy = bf16_bits_to_f32(yr[k]);
            dr[k] = static_cast<uint16_t>(pack_bf16x2(fmaf(xh, -v.y, dy * a.w[k]) * v.x, 0.0f));
            float& sum = (e & 1) ? dwv[j][e >> 1].y : dwv[j][e >> 1].x;
            sum = fmaf(dy, xh, sum);
          }
        }
    }
  }
  pdl_launch_dependents();
  // the groups' column sums, added in order of the groups; the last writes the CTA's partial row
#pragma unroll
  for (int p = 0; p < (kLayer ? 2 : 1); ++p) {
    float* out = a.part + (static_cast<size_t>(blockIdx.x) * (kLayer ? 2 : 1) + p) * K;
    for (int g = 0; g < a.rg; ++g) {
      if (a.rg > 1) __syncthreads();
      if (g != grp) continue;
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const int c = t + j * T;
        const float2(&s)[4] = p ? dbv[j] : dwv[j];
        float4 lo = make_float4(s[0].x, s[0].y, s[1].x, s[1].y), hi = make_float4(s[2].x, s[2].y, s[3].x, s[3].y);
        if (g > 0) {
          const float4 u = s_acc[c], v = s_acc[P + c];
          lo = make_float4(lo.x + u.x, lo.y + u.y, lo.z + u.z, lo.w + u.w);
          hi = make_float4(hi.x + v.x, hi.y + v.y, hi.z + v.z, hi.w + v.w);
        }
        if (g + 1 < a.rg) {
          s_acc[c] = lo;
          s_acc[P + c] = hi;
        } else if (K % 4 == 0 && 8 * c + 8 <= K) {
          *reinterpret_cast<float4*>(out + 8 * c) = lo;
          *reinterpret_cast<float4*>(out + 8 * c + 4) = hi;
        } else {
          const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (8 * c + e < K) out[8 * c + e] = v[e];
        }
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
    if (rms_far(c1 + a.eps)) {
      const float2 far = rms_far_row(xr, dyr, a.w, K, a.eps);
      rstd = far.x;
      c2 = far.y;
    } else {
      rstd = __fdiv_rn(1.0f, __fsqrt_rn(c1 + a.eps));
      c2 *= rstd;
    }
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

// 16 values of a chunk: RN(code s) as bf16 pairs.
__device__ __forceinline__ void dequant16(const uint4 q, float s, uint32_t (&o)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f[2];
    codes4_f32(w[i], f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f[h] = __fmul2_rn(f[h], splat2(s));
      o[2 * i + h] = pack_bf16x2(f[h].x, f[h].y);
    }
  }
}

// y = RNbf16 of it: the activation, restored in its own type.  A CTA of 256
// threads takes 256 / lanes rows, `lanes` threads a row, 16 codes each a step.
__global__ void __launch_bounds__(256) dequant_act_kernel(const int8_t* __restrict__ q, int64_t ldq,
                                                          const float* __restrict__ gamma, int M, int K,
                                                          uint16_t* __restrict__ y, int64_t ldy, int lanes) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int r = threadIdx.x / lanes, t = threadIdx.x - r * lanes;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / lanes) + r;
  if (row >= M) return;
  const float s = __fdiv_rn(gamma[row], kQb);
  const int8_t* const end = q + static_cast<int64_t>(M - 1) * ldq + K;
  const bool yv = (ldy % 8) == 0 && (reinterpret_cast<uintptr_t>(y) & 15u) == 0;
  for (int k0 = 16 * t; k0 < K; k0 += 16 * lanes) {
    uint32_t w[4], o[8];
    load16_codes_any(q + row * ldq, k0, K, q, end, w);
    dequant16(make_uint4(w[0], w[1], w[2], w[3]), s, o);
    store8_bf16(y + row * ldy, k0, K, yv, o);
    store8_bf16(y + row * ldy, k0 + 8, K, yv, o + 4);
  }
}

// The element-wise kernels for contiguous matrices of at least 16 columns (the
// matrix as one row of `count` elements): chunks of 16 are dealt to threads
// regardless of the rows, of which a chunk meets at most two, and each thread's
// loads go out together: 5.5 us for 4096 x 2560 restored values, 9.6 for the
// gate's gradients there.  The two kernels for rows that are apart wait for one
// chunk before they ask for the next (8.8 and 16.8; latency takes three quarters
// of their time).  What is left of the last chunk goes element by element.
struct FlatChunk {
  uint32_t row;   // of its first element
  uint32_t left;  // elements of the chunk in that row
};
__device__ __forceinline__ FlatChunk flat_chunk(uint32_t i, uint32_t K) {
  const uint32_t row = 16u * i / K;
  return {row, K - (16u * i - row * K)};
}
constexpr int kFlatChunks = 4;
__global__ void __launch_bounds__(256) dequant_flat_kernel(const int8_t* __restrict__ q, const float* __restrict__ gamma,
                                                           uint32_t K, uint32_t count, uint16_t* __restrict__ y) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const uint32_t total = count / 16;
  const uint32_t i0 = blockIdx.x * (256 * kFlatChunks) + threadIdx.x;
  uint4 w[kFlatChunks];
  float s[kFlatChunks], s1[kFlatChunks];
  uint32_t left[kFlatChunks];
#pragma unroll
  for (int j = 0; j < kFlatChunks; ++j) {
    const uint32_t i = min(i0 + 256 * j, total - 1);
    w[j] = reinterpret_cast<const uint4*>(q)[i];
    const FlatChunk f = flat_chunk(i, K);
    left[j] = f.left;
    s[j] = gamma[f.row];
    s1[j] = f.left < 16 ? gamma[f.row + 1] : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < kFlatChunks; ++j) {
    if (i0 + 256 * j >= total) continue;
    uint32_t o[8];
    dequant16(w[j], __fdiv_rn(s[j], kQb), o);
    if (left[j] < 16) {  // the next row's part
      uint32_t n[8];
      dequant16(w[j], __fdiv_rn(s1[j], kQb), n);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e] = 2 * e >= left[j] ? n[e] : 2 * e + 1 >= left[j] ? (o[e] & 0xFFFFu) | (n[e] & 0xFFFF0000u) : o[e];
    }
    st_global_v8(y + 16 * static_cast<size_t>(i0 + 256 * j), o);
  }
  if (blockIdx.x == 0 && threadIdx.x < count % 16) {
    const uint32_t e = 16 * total + threadIdx.x;
    y[e] = static_cast<uint16_t>(
        pack_bf16x2(__fmul_rn(static_cast<float>(q[e]), __fdiv_rn(gamma[e / K], kQb)), 0.0f));
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
  int lw;                              // log2 of the warps per row
};

// Warps and chunks as in layernorm_kernel; h is cheaper computed again (three
// bf16x2 operations a pair) than kept.
template <bool kAny, int G>
__global__ void __launch_bounds__(32 * kQuantWarps, G >= 1 && G <= 6 ? 3 : 2)
    relu2_glu_quant_kernel(const GluSaveArgs a) {
  constexpr bool kRegs = G > 0;
  constexpr int GR = kRegs ? G : 1;
  __shared__ uint32_t s_mx[3][kQuantWarps];
  __shared__ int32_t s_sum[kQuantWarps];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpr = 1 << a.lw, N = a.N;
  const int rloc = warp >> a.lw, sub = warp & (wpr - 1);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kQuantWarps >> a.lw) + rloc;
  const bool active = row < a.M;
  const uint16_t* gr = a.g + (active ? row : 0) * a.ldg;
  const uint16_t* ur = a.u + (active ? row : 0) * a.ldu;
  const uint16_t* const gend = a.g + static_cast<int64_t>(a.M - 1) * a.ldg + N;
  const uint16_t* const uend = a.u + static_cast<int64_t>(a.M - 1) * a.ldu + N;
  const int chunks = (N + 7) / 8, cstride = 32 * wpr, c0 = sub * 32 + lane;

  auto load = [&](int c, uint32_t (&r)[2][4]) {
    if (!kAny) {
      const uint4 t = *reinterpret_cast<const uint4*>(gr + 8 * c), y = *reinterpret_cast<const uint4*>(ur + 8 * c);
      r[0][0] = t.x; r[0][1] = t.y; r[0][2] = t.z; r[0][3] = t.w;
      r[1][0] = y.x; r[1][1] = y.y; r[1][2] = y.z; r[1][3] = y.w;
    } else {
      load8_any(gr, 8 * c, N, a.g, gend, r[0]);
      load8_any(ur, 8 * c, N, a.u, uend, r[1]);
    }
  };
  uint32_t v[GR][2][4];  // g, u
  if (kRegs) {
#pragma unroll
    for (int j = 0; j < GR; ++j) load(min(c0 + j * cstride, chunks - 1), v[j]);
  }
  // f(j, chunk, its words) for each of the lane's chunks
  auto for_chunks = [&](auto&& f) {
    if (!active) return;
    if constexpr (kRegs) {
#pragma unroll
      for (int j = 0; j < GR; ++j)
        if (c0 + j * cstride < chunks) f(j, c0 + j * cstride, v[j]);
    } else {
      for (int c = c0; c < chunks; c += cstride) {
        uint32_t r[2][4];
        load(c, r);
        f(0, c, r);
      }
    }
  };
  auto as2 = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
  auto bits = [](__nv_bfloat162 h) { return *reinterpret_cast<const uint32_t*>(&h); };
  // two of h: each product is exact in more bits than bf16 keeps and is rounded once
  auto hword = [&](uint32_t g, uint32_t u) {
    const __nv_bfloat162 r = __hmax2_nan(as2(g), as2(0u));  // a NaN must reach h and its row's maximum
    return bits(__hmul2_rn(__hmul2_rn(r, r), as2(u)));
  };
  uint32_t mx[3] = {0u, 0u, 0u};  // two maxima of |.| each; NaN is kept
  for_chunks([&](int, int, const uint32_t (&r)[2][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[3] = {r[0][i], r[1][i], hword(r[0][i], r[1][i])};
#pragma unroll
      for (int p = 0; p < 3; ++p) mx[p] = bits(__hmax2_nan(as2(mx[p]), __habs2(as2(w[p]))));
    }
  });
#pragma unroll
  for (int p = 0; p < 3; ++p)  // |x| as bit patterns order like the values
    mx[p] = __reduce_max_sync(0xffffffffu, max(mx[p] << 16, mx[p] & 0xFFFF0000u));
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
  uint32_t redo = 0u;  // chunks with codes that take the exact quotient
  const size_t at = static_cast<size_t>(active ? row : 0) * N;
  const bool vq = !kAny || ((N % 8) == 0 && ((reinterpret_cast<uintptr_t>(a.qg) | reinterpret_cast<uintptr_t>(a.qu) |
                                              reinterpret_cast<uintptr_t>(a.qh)) & 7u) == 0);
  int8_t* const out[3] = {a.qg + at, a.qu + at, a.qh + at};
  auto values = [&](int p, const uint32_t (&r)[2][4], float2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = bf16_2(p < 2 ? r[p][i] : hword(r[0][i], r[1][i]));
  };
  auto exact = [&](int ch) {
    uint32_t r[2][4];
    load(ch, r);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      float2 f[4];
      values(p, r, f);
      float emax = 0.0f;
      const uint2 w0 = codes8_near(f, c[p], emax);
      if (emax > kCodesNear) {
        const uint2 w = codes8_exact(f, d[p]);
        store8_codes(out[p], 8 * ch, N, vq, w);
        if (p == 2) sum += code_sum(w) - code_sum(w0);
      }
    }
  };
  for_chunks([&](int j, int ch, const uint32_t (&r)[2][4]) {
    float emax = 0.0f;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      float2 f[4];
      values(p, r, f);
      const uint2 w = codes8_near(f, c[p], emax);
      if (p == 2) sum += code_sum(w);
      store8_codes(out[p], 8 * ch, N, vq, w);
    }
    if (emax > kCodesNear) {
      if (kRegs)
        redo |= 1u << j;
      else
        exact(ch);
    }
  });
  while (kRegs && redo) {
    const int j = __ffs(redo) - 1;
    redo &= redo - 1;
    exact(c0 + j * cstride);
  }
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

// The step of a row's codes, NaN where the row's maximum is infinite too: such a row's codes are without meaning (most
// are 0), and max(., 0) would turn some of their products into zero gradients.
__device__ __forceinline__ float grad_step(float gamma) {
  const float s = __fdiv_rn(gamma, kQb);
  return __fadd_rn(s, __fsub_rn(s, s));
}

// Two of dg = RNb(2 dh r u~) and du = RNb(dh r^2), r = max(g~, 0), of two codes' values g, u each.
__device__ __forceinline__ void glu_grads2(float2 g, float2 u, uint32_t dh, float2 sg, float2 su, uint32_t& dg,
                                           uint32_t& du) {
  const float2 d = bf16_2(dh);
  float2 rp = __fmul2_rn(g, sg);
  rp = make_float2(max_nan(rp.x, 0.0f), max_nan(rp.y, 0.0f));
  const float2 dr = __fmul2_rn(d, rp);
  const float2 p = __fmul2_rn(__fadd2_rn(dr, dr), __fmul2_rn(u, su)), q = __fmul2_rn(dr, rp);
  dg = pack_bf16x2(p.x, p.y);
  du = pack_bf16x2(q.x, q.y);
}

// As dequant_flat_kernel, two chunks a thread (64 bytes each).  kSplit: chunks may meet two rows (rows of a multiple of
// 16 columns: 11.7 us at 4096 x 2560, with the selects 15.2).
template <bool kSplit>
__global__ void __launch_bounds__(256, 4)
    relu2_glu_backward_flat_kernel(const uint16_t* __restrict__ dh, const int8_t* __restrict__ qg,
                                   const float* __restrict__ gg, const int8_t* __restrict__ qu,
                                   const float* __restrict__ gu, uint32_t N, uint32_t count,
                                   uint16_t* __restrict__ dg, uint16_t* __restrict__ du) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const uint32_t total = count / 16;
  const uint32_t i0 = blockIdx.x * 512 + threadIdx.x;
  uint4 wg[2], wu[2];
  uint32_t h[2][8], left[2];
  float sg[2][2], su[2][2];  // of the chunk's row and the next
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t i = min(i0 + 256 * j, total - 1);
    wg[j] = reinterpret_cast<const uint4*>(qg)[i];
    wu[j] = reinterpret_cast<const uint4*>(qu)[i];
    ld_global_nc_v8(dh + 16 * static_cast<size_t>(i), h[j]);
    const FlatChunk f = flat_chunk(i, N);
    left[j] = f.left;
    sg[j][0] = gg[f.row];
    su[j][0] = gu[f.row];
    if (kSplit) {
      const uint32_t next = f.row + (f.left < 16 ? 1u : 0u);
      sg[j][1] = gg[next];
      su[j][1] = gu[next];
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float a[2], b[2];
#pragma unroll
    for (int r = 0; r < (kSplit ? 2 : 1); ++r) {
      a[r] = grad_step(sg[j][r]);
      b[r] = grad_step(su[j][r]);
    }
    const uint32_t g4[4] = {wg[j].x, wg[j].y, wg[j].z, wg[j].w}, u4[4] = {wu[j].x, wu[j].y, wu[j].z, wu[j].w};
    uint32_t og[8], ou[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 fg[2], fu[2];
      codes4_f32(g4[i], fg);
      codes4_f32(u4[i], fu);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t k = 4 * i + 2 * e;
        const float2 sa = make_float2(kSplit && k >= left[j] ? a[1] : a[0], kSplit && k + 1 >= left[j] ? a[1] : a[0]);
        const float2 sb = make_float2(kSplit && k >= left[j] ? b[1] : b[0], kSplit && k + 1 >= left[j] ? b[1] : b[0]);
        glu_grads2(fg[e], fu[e], h[j][2 * i + e], sa, sb, og[2 * i + e], ou[2 * i + e]);
      }
    }
    if (i0 + 256 * j < total) {
      const size_t at = 16 * static_cast<size_t>(i0 + 256 * j);
      st_global_v8(dg + at, og);
      st_global_v8(du + at, ou);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x < count % 16) {
    const uint32_t e = 16 * total + threadIdx.x, row = e / N;
    uint32_t p, q;
    glu_grads2(splat2(static_cast<float>(qg[e])), splat2(static_cast<float>(qu[e])), dh[e],
               splat2(grad_step(gg[row])), splat2(grad_step(gu[row])), p, q);
    dg[e] = static_cast<uint16_t>(p);
    du[e] = static_cast<uint16_t>(q);
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
  const float sg = grad_step(gg[row]), su = grad_step(gu[row]);
  const uint16_t* const end = dh + static_cast<int64_t>(M - 1) * lddh + N;
  const size_t codes = static_cast<size_t>(M) * N;
  const bool vo = (N % 8) == 0 && ((reinterpret_cast<uintptr_t>(dg) | reinterpret_cast<uintptr_t>(du)) & 15u) == 0;
  const uint16_t* dhr = dh + row * lddh;
  const size_t at = static_cast<size_t>(row) * N;
  for (int k0 = 16 * t; k0 < N; k0 += 16 * lanes) {
    uint32_t wg[4], wu[4], h0[4], h1[4];
    load16_codes_any(qg + at, k0, N, qg, qg + codes, wg);
    load16_codes_any(qu + at, k0, N, qu, qu + codes, wu);
    load8_any(dhr, k0, N, dh, end, h0);
    load8_any(dhr, k0 + 8, N, dh, end, h1);
    uint32_t og[8], ou[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 fg[2], fu[2];
      codes4_f32(wg[i], fg);
      codes4_f32(wu[i], fu);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        glu_grads2(fg[h], fu[h], i < 2 ? h0[2 * i + h] : h1[2 * (i - 2) + h], splat2(sg), splat2(su), og[2 * i + h], ou[2 * i + h]);
    }
    store8_bf16(dg + at, k0, N, vo, og);
    store8_bf16(dg + at, k0 + 8, N, vo, og + 4);
    store8_bf16(du + at, k0, N, vo, ou);
    store8_bf16(du + at, k0 + 8, N, vo, ou + 4);
  }
}

}  // namespace bl
