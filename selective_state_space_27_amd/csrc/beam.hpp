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

// The largest prefix of BITS bits such that at least `want` of the values that the
// wave's lanes hold, G each, are not below it (0 where fewer are above 0).
template <int BITS, int G>
__device__ __forceinline__ uint32_t wave_threshold(const uint32_t (&mine)[G], int want) {
  uint32_t t = 0;
  for (int b = 31; b >= 32 - BITS; --b) {
    const uint32_t with = t | 1u << b;
    int c = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) c += (int)__popcll(__ballot(mine[g] >= with));
    if (c >= want) t = with;
  }
  return t;
}
// The same of the values v[W][64] in LDS, of which the largest of every lane count
// (`fine`: of every lane and quarter of the rows).  The want-th of 64 is a good bound
// while the best lie in different lanes: not for 64 of them, nor where they lie in one
// beam's few slices.
template <int BITS, int W>
__device__ __forceinline__ uint32_t lds_threshold(const uint32_t (*v)[64], bool fine, int want) {
  uint32_t mine[4], most[1];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    mine[g] = v[g * (W / 4)][threadIdx.x & 63];
#pragma unroll
    for (int w = 1; w < W / 4; ++w) mine[g] = max(mine[g], v[g * (W / 4) + w][threadIdx.x & 63]);
  }
  if (fine) return wave_threshold<BITS, 4>(mine, want);
  most[0] = max(max(mine[0], mine[1]), max(mine[2], mine[3]));
  return wave_threshold<BITS, 1>(most, want);
}
constexpr int kLanesEnough = 32;

}  // namespace mss
