// Candidates of beam search (gfx950): a logit and its place in the row as one
// key, totals in 64 bits, and what selecting the best of many needs.
#pragma once

#include "common.hpp"

namespace mss {

// Bits of a float or double made monotonic (-0 as +0, which are equal): larger
// values have larger bits.
__device__ __forceinline__ uint32_t ordered_bits(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o ^ ((uint32_t)((int32_t)~o >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t ordered_bits(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  return u ^ ((uint64_t)((int64_t)u >> 63) | (1ull << 63));
}
__device__ __forceinline__ double value_of(uint64_t o) {
  return __builtin_bit_cast(double, o ^ ((uint64_t)((int64_t)~o >> 63) | (1ull << 63)));
}
constexpr uint32_t kOrderedNegInf = 0x007fffffu;  // ordered_bits(-infinity): what is above it is a candidate
constexpr uint64_t kOrderedNegInf64 = 0x000fffffffffffffull;

// Order of a row's candidates: the larger logit first, then the lower place.
__device__ __forceinline__ uint64_t key_of(uint32_t ordered, uint32_t place) { return (uint64_t)ordered << 32 | ~place; }
__device__ __forceinline__ uint32_t place_of(uint64_t key) { return ~(uint32_t)key; }

// The largest prefix of BITS bits such that at least `want` of the wave's 64 lanes
// hold a value not below it (0 where fewer hold one above 0).
template <int BITS, typename T>
__device__ __forceinline__ T wave_threshold(T mine, int want) {
  T t = 0;
#pragma unroll
  for (int b = 8 * (int)sizeof(T) - 1; b >= 8 * (int)sizeof(T) - BITS; --b) {
    const T with = t | ((T)1 << b);
    if (__popcll(__ballot(mine >= with)) >= want) t = with;
  }
  return t;
}

}  // namespace mss
