// Logits as ordered whole numbers, and ranges of them split into bins: the arithmetic of the
// searches in sample.cu. Plain C++ for the host too.
#pragma once

#include <stdint.h>
#include <string.h>

#ifdef __CUDACC__
#define DMTP_KEYS __host__ __device__ __forceinline__
#else
#define DMTP_KEYS inline
#endif

DMTP_KEYS uint32_t key_bits(float l) {
#ifdef __CUDA_ARCH__
  return __float_as_uint(l);
#else
  uint32_t u;
  memcpy(&u, &l, 4);
  return u;
#endif
}

// Unsigned keys in the order of the logits. -0 and +0 share one key and every other number has one
// of its own with none left out between them, so "lo <= key_of(x) <= hi" and
// "logit_of(lo) <= x <= logit_of(hi)" are the same: what a float comparison lets into a range has
// its place in the range's bins.
DMTP_KEYS uint32_t key_of(float l) {
  const uint32_t u = key_bits(l);
  return u & 0x80000000u ? 0u - u : u | 0x80000000u;
}
DMTP_KEYS float logit_of(uint32_t key) {
  const uint32_t u = key & 0x80000000u ? key & 0x7fffffffu : 0u - key;
#ifdef __CUDA_ARCH__
  return __uint_as_float(u);
#else
  float l;
  memcpy(&l, &u, 4);
  return l;
#endif
}
constexpr uint32_t kMaskedKey = 0x00800000u;      // minus infinity
constexpr uint32_t kLowestKey = kMaskedKey + 1u;  // the lowest finite number

// Bits to drop of hi - key so that the range lo..hi falls into 2^bits bins, the largest keys first.
DMTP_KEYS int range_shift(uint32_t lo, uint32_t hi, int bits) {
  int n = 0;
#ifdef __CUDA_ARCH__
  n = 32 - __clz((int)(hi - lo)) - bits;
#else
  while (n < 32 && (hi - lo) >> n) ++n;
  n -= bits;
#endif
  return n > 0 ? n : 0;
}
// The range of bin f of lo..hi.
DMTP_KEYS void take_bin(uint32_t& lo, uint32_t& hi, int shift, uint32_t f) {
  hi -= f << shift;
  lo = hi - lo < (1u << shift) ? lo : hi - ((1u << shift) - 1);
}
