// Candidates of beam search (gfx950): a logit and its place in the row as one
// key, totals in 64 bits, and the order they are taken in.
#pragma once

#include "common.hpp"

namespace mss {

// Order of candidates in a row: the larger logit first, then the lower place.
// As one unsigned key: the float's bits made monotonic (-0 as +0, which are
// equal), then the place's complement.
__device__ __forceinline__ uint32_t ordered_bits(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o ^ ((uint32_t)((int32_t)~o >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t place) {
  return (uint64_t)ordered_bits(v) << 32 | (uint32_t)~place;
}
__device__ __forceinline__ uint32_t place_of(uint64_t key) { return ~(uint32_t)key; }

// A candidate of a sequence: its total (never NaN) and place beam * vocab + token.
struct Candidate {
  double total;
  int64_t place;
};
__device__ __forceinline__ bool before(const Candidate& a, const Candidate& b) {
  return a.total > b.total || (a.total == b.total && a.place < b.place);
}

}  // namespace mss
