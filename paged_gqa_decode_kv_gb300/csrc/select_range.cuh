// select_range.cuh -- the block selection's keys and its search for the least
// selected one: a range of unsigned keys narrowed to the one of 256 equal bins
// that holds a wanted rank, until it is one key or wholly wanted.  On the host
// too, where its arithmetic is tested over the whole range of keys.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PGD_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PGD_HOST_DEVICE inline
#endif

namespace pgd {

constexpr int kRangeBins = 256;
// 32 bits of keys, 8 taken a pass.
constexpr int kRangePasses = 4;

// A score's bits as an unsigned integer of the same order, above 0.
PGD_HOST_DEVICE uint32_t score_key(uint32_t bits) {
  return (bits & 0x80000000u) ? ~bits : (bits | 0x80000000u);
}

// Key k in [lo, hi] falls into bin (k - lo) >> range_shift(lo, hi) < 256; lo < hi.
PGD_HOST_DEVICE int range_shift(uint32_t lo, uint32_t hi) {
#ifdef __CUDA_ARCH__
  const int top = __clz(hi - lo);
#else
  const int top = __builtin_clz(hi - lo);
#endif
  return top < 24 ? 24 - top : 0;
}

// The range becomes its bin `bin`, one that begins in it.  (By the distance
// from its start: the end of the last bin can lie past 2^32.)
PGD_HOST_DEVICE void narrow_range(uint32_t &lo, uint32_t &hi, uint32_t bin, int shift) {
  lo += bin << shift;
  const uint32_t rest = hi - lo, size = (1u << shift) - 1u;
  hi = lo + (rest < size ? rest : size);
}

}  // namespace pgd
