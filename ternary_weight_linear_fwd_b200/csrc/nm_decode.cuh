// nm_decode.cuh -- packed N:M rows as dense 2-bit codes.  Plain C++ on host and
// device, so that what it reads can be checked on the CPU.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define BL_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define BL_HOST_DEVICE inline
#endif

namespace bl {

struct ExpandArgs {
  const uint8_t* codes;
  const uint8_t* meta;
  int64_t ldc, ldm, ldd;  // ldd: row stride of the dense codes, bytes (bf16: of the values, elements)
  int N, K, nm_n, nm_m;
  uint32_t* out;
};

// The 16 dense codes from k0 (a multiple of 16) of row n of an N:M matrix; positions past K get code 1.  K is a multiple
// of m, so those before K lie in whole blocks, and only what belongs to these is read: a row of n:8 codes is as long as
// its kept codes, rounded up to 16 bytes, and may end before the word of a position past K would (7:8, K = 72: 16 bytes,
// the last words' codes at bytes 14 to 27).  Kept positions are read by half-words (2:4's codes too), whose last one is
// inside the row: 2 ceil(K / 16) <= 16 ceil(K / 128).
BL_HOST_DEVICE uint32_t nm_codes16(const ExpandArgs& a, int64_t n, int k0) {
  uint32_t o = 0x55555555u;
  if (k0 >= a.K) return o;
  const int w = k0 >> 4;
  const uint32_t mt = *reinterpret_cast<const uint16_t*>(a.meta + n * a.ldm + 2 * w);  // 4 nibbles, or 2 masks
  if (a.nm_m == 4) {
    const uint32_t c = *reinterpret_cast<const uint16_t*>(a.codes + n * a.ldc + 2 * w);  // 8 kept codes
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t s0 = 8 * b + 2 * ((mt >> (4 * b)) & 3u), s1 = 8 * b + 2 * ((mt >> (4 * b + 2)) & 3u);
      // code 1 (01) is there: its place becomes c by flipping c ^ 1
      if (k0 + 4 * b < a.K) o ^= ((((c >> (4 * b)) & 3u) ^ 1u) << s0) ^ ((((c >> (4 * b + 2)) & 3u) ^ 1u) << s1);
    }
  } else {
    const int first = 4 * a.nm_n * w;                          // bit of the first kept code
    const int bits = 2 * a.nm_n * (k0 + 8 < a.K ? 2 : 1);      // of the one or two blocks before K
    const uint8_t* p = a.codes + n * a.ldc + (first >> 3);
    const int shift = first & 7;
    uint64_t v = 0;
    for (int i = 0; 8 * i < bits + shift; ++i) v |= static_cast<uint64_t>(p[i]) << (8 * i);
    uint32_t c = static_cast<uint32_t>(v >> shift);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t kept = c >> (2 * a.nm_n * b);
      if (k0 + 8 * b < a.K)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((mt >> (8 * b + j)) & 1u) {
            o ^= ((kept & 3u) ^ 1u) << (16 * b + 2 * j);
            kept >>= 2;
          }
    }
  }
  return o;
}

}  // namespace bl
