// Shape of the norm kernels (add_norm.hip, gated_norm.hip): how rows are laid
// over lanes, and the sums over rows for the weights' gradients.
//
// A "segment" is what one norm runs over: a row, or one group of a row's
// columns.  Segments of up to 512 columns take 32 or 64 lanes of a wave
// (LANES; a workgroup of 256 threads holds 256 / LANES of them, the sums need
// no barrier); longer ones take a workgroup (LANES = 0) of just enough waves
// for eight columns per thread, or for sixteen (K = 2) past kOneVectorMax
// columns.  Workgroups walk over rows with a stride, the next row's loads
// issued before the present one's sums, and keep the weights (and the
// gradients' partial sums over rows) in registers.
#pragma once

#include <type_traits>

#include "launch.hpp"
#include "rows.hpp"

namespace mss {

constexpr int kNormCUs = 256;
constexpr int kOneVectorMax = 8192;  // columns of a segment with one vector per thread

// Segment layout of a launch.
struct NormShape {
  int lanes;    // 32, 64, or 0 (workgroup)
  int k;        // vectors of 8 columns per thread
  int threads;  // of a workgroup
  int segs;     // segments a workgroup holds at a time
};

inline NormShape norm_shape(int64_t cols) {
  if (cols <= 256) return {32, 1, 256, 8};
  if (cols <= 512) return {64, 1, 256, 4};
  const int k = cols <= kOneVectorMax ? 1 : 2;
  const int threads = (int)((cols + 8 * k - 1) / (8 * k) + 63) / 64 * 64;
  return {0, k, threads, 1};
}

// Workgroups per group of columns, no more than there are rows.  One to two rows
// of the model's width in flight on a CU stream best: at 32768 x 5120 (640
// threads) the gated norm takes 231 us with one workgroup per CU and 255 with
// two, its backward 444 and 459 (498 with sixteen, which also writes and reads
// more partial sums); at 32768 x 2560 (320 threads) add_norm takes 181 us with
// one, 178 with two, 202 with eight.  Narrow rows need more: 768 columns (128
// threads) 190, 90, 75 and 77 us with one, three, six and eight.
inline int64_t norm_blocks(const NormShape& s, int64_t rows, int64_t groups, bool backward) {
  const int per_cu = backward ? (s.threads >= 256 ? 1 : 512 / s.threads) : s.threads >= 640 ? 1 : 640 / s.threads;
  const int64_t slots = (int64_t)kNormCUs * per_cu;
  const int64_t want = slots / groups > 0 ? slots / groups : 1;
  const int64_t most = (rows + s.segs - 1) / s.segs;
  return want < most ? want : most;
}

// Calls f with the shape's LANES and K, the most threads of its workgroups and
// whether rows are whole vectors, as constants.  768 threads at most leave 168
// registers for two vectors each (columns up to 12288), 1024 leave 128.
template <typename F>
inline hipError_t with_shape(const NormShape& s, bool whole, F&& f) {
  typedef std::integral_constant<int, 0> group;
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  const std::integral_constant<int, 256> t256;
  const std::integral_constant<int, 768> t768;
  const std::integral_constant<int, 1024> t1024;
  const auto with = [&](auto w) {
    if (s.lanes == 32) return f(std::integral_constant<int, 32>{}, one, t256, w);
    if (s.lanes == 64) return f(std::integral_constant<int, 64>{}, one, t256, w);
    if (s.k == 1) return f(group{}, one, t1024, w);
    return s.threads <= 768 ? f(group{}, two, t768, w) : f(group{}, two, t1024, w);
  };
  return whole ? with(std::true_type{}) : with(std::false_type{});
}

// Where a thread is: which of the workgroup's segments, its first column, and
// the column its k-th vector starts at.
template <int LANES>
struct Place {
  int seg;   // segment of the workgroup
  int nseg;  // segments of the workgroup
  __device__ __forceinline__ Place() {
    if constexpr (LANES == 0) seg = 0, nseg = 1;
    else seg = (int)threadIdx.x / LANES, nseg = 256 / LANES;
  }
  __device__ __forceinline__ int col(int k) const {
    if constexpr (LANES == 0) return (k * (int)blockDim.x + (int)threadIdx.x) * 8;
    else return ((int)threadIdx.x % LANES) * 8;
  }
};

// Eight weights (fp32, any alignment of 4), zeros past the end.
template <bool WHOLE>
__device__ __forceinline__ void load_w(const float* w, int col, int n, float (&v)[8]) {
  widen<kSrcF32>(load_raw<kSrcF32, WHOLE>(w, nullptr, col, n), v);
}

// A workgroup's sums over its rows, `part[col]`: the sums of its segments (the
// same columns, different rows) meet in LDS, in a fixed order.
template <int LANES, bool WHOLE>
__device__ __forceinline__ void store_partial(float* part, int col, int n, const float (&acc)[8], float* lds) {
  if constexpr (LANES == 0) {
    if (n > 0) store8<true, WHOLE>(part, col, n, acc);
  } else {
    __syncthreads();  // before: `lds` may still be read from the last call
#pragma unroll
    for (int j = 0; j < 8; ++j) lds[threadIdx.x * 8 + j] = acc[j];
    __syncthreads();
    constexpr int W = LANES * 8;  // columns a segment's lanes cover
    const int ncols = col + n;    // the segment's columns (the same for every thread)
    for (int c = threadIdx.x; c < W; c += 256) {
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < 256 / LANES; ++g) s += lds[g * W + c];
      if (c < ncols) part[c] = s;
    }
  }
}
constexpr int kPartialLds = 256 * 8;

// Sums of `nparts` partial rows [nparts][nout][cols]: the first is dweight; the
// second, S, gives dgamma = scale post S and dpost = scale gamma S (each where
// its pointer is given; post and gamma null: 1).
struct SumPartialsArgs {
  const float* part;
  float* dweight;
  float* dgamma;
  float* dpost;
  const float* post;
  const float* gamma;
  float scale;
  int64_t nparts;
  int64_t cols;
  int nout;
  int64_t first = 0;  // column of a launch's first workgroup, set by launch_sum_partials
};
hipError_t launch_sum_partials(const SumPartialsArgs& a, hipStream_t stream);

}  // namespace mss
