// One token of the gated linear recurrence (gfx950): h_out = a h + beta i x per
// channel, the state read from the parent beam's row where parents are given.
// Definitions in include/mambascan.h, arithmetic in recurrence.hpp.
//
// Four neighbouring channels a thread, with accesses of 8 and 16 bytes at any
// alignment; everything a thread reads but its parent's state is under way at
// once.  256 x 5120 bf16 from parents' states (21 MB): 6.8 us, 3.1 TB/s, bound by the
// two trips to memory one after the other (one channel a thread: 9.0 us); one row
// of 2560: 3.6 us, the least a launch takes.
#include "launch.hpp"
#include "recurrence.hpp"
#include "rows.hpp"

namespace mss {
namespace {

constexpr int kChannels = 4, kThreadsStep = 256;
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));

// Channels d .. d + 3 of a row; n of them exist (the rest: 0).
template <bool BF16>
__device__ __forceinline__ void load4(const void* row, int64_t d, int n, float (&v)[kChannels]) {
  if constexpr (BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(row) + d;
    if (n >= kChannels) {
      const u32x2 w = *reinterpret_cast<const u32x2_a2*>(p);
      v[0] = bf16_lo(w[0]), v[1] = bf16_hi(w[0]), v[2] = bf16_lo(w[1]), v[3] = bf16_hi(w[1]);
    } else {
#pragma unroll
      for (int j = 0; j < kChannels; ++j) v[j] = j < n ? bf16_to_f32(p[j]) : 0.0f;
    }
  } else {
    const float* p = static_cast<const float*>(row) + d;
    if (n >= kChannels) {
      const u32x4 w = *reinterpret_cast<const u32x4_a4*>(p);
#pragma unroll
      for (int j = 0; j < kChannels; ++j) v[j] = __uint_as_float(w[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kChannels; ++j) v[j] = j < n ? p[j] : 0.0f;
    }
  }
}
template <bool BF16>
__device__ __forceinline__ void store4(void* row, int64_t d, int n, const float (&v)[kChannels]) {
  if constexpr (BF16) {
    uint16_t* p = static_cast<uint16_t*>(row) + d;
    if (n >= kChannels) {
      *reinterpret_cast<u32x2_a2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
#pragma unroll
      for (int j = 0; j < kChannels - 1; ++j)
        if (j < n) p[j] = f32_to_bf16(v[j]);
    }
  } else {
    float* p = static_cast<float*>(row) + d;
    if (n >= kChannels) {
      *reinterpret_cast<u32x4_a4*>(p) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                              __float_as_uint(v[3])};
    } else {
#pragma unroll
      for (int j = 0; j < kChannels - 1; ++j)
        if (j < n) p[j] = v[j];
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreadsStep) recurrence_step_kernel(RecurrenceStepParams p, uint32_t vecs) {
  const uint32_t i = blockIdx.x * kThreadsStep + threadIdx.x, r = i / vecs;
  const int64_t row = r, d = (int64_t)(i - r * vecs) * kChannels;
  if (row >= p.rows) return;
  const int n = (int)(p.dim - d < kChannels ? p.dim - d : kChannels);
  constexpr int64_t es = BF16 ? 2 : 4;
  int64_t from = row;
  if (p.parents != nullptr) {
    const int64_t parent = p.parents[row];
    if (parent >= 0 && parent < p.beams) from = row - row % (uint32_t)p.beams + parent;
  }
  float x[kChannels], ga[kChannels], gx[kChannels], lam[kChannels], h[kChannels];
  load4<BF16>(static_cast<const char*>(p.gate_a) + row * p.gate_a_stride * es, d, n, ga);
  load4<BF16>(static_cast<const char*>(p.gate_x) + row * p.gate_x_stride * es, d, n, gx);
  load4<BF16>(static_cast<const char*>(p.x) + row * p.x_stride * es, d, n, x);
  load4<false>(p.lam, d, n, lam);
  load4<false>(p.h + from * p.dim, d, n, h);
#pragma unroll
  for (int j = 0; j < kChannels; ++j) {
    const float m = decay_of<false, !BF16>(decay_rate(p.c, lam[j]) * sigmoid_of<!BF16>(ga[j]));
    h[j] = decayed<false>(m, h[j]) + beta_of(rest_of<false>(m)) * sigmoid_of<!BF16>(gx[j]) * x[j];
  }
  store4<false>(p.h_out + row * p.dim, d, n, h);
  store4<BF16>(static_cast<char*>(p.y) + row * p.y_stride * es, d, n, h);
}

}  // namespace

hipError_t launch_recurrence_step(const RecurrenceStepParams& p, hipStream_t stream) {
  const int64_t vecs = (p.dim + kChannels - 1) / kChannels;  // rows * vecs below 2^31 + rows
  const dim3 grid((unsigned)((p.rows * vecs + kThreadsStep - 1) / kThreadsStep));
  const auto kernel = p.bf16 ? recurrence_step_kernel<true> : recurrence_step_kernel<false>;
  hipLaunchKernelGGL(kernel, grid, dim3(kThreadsStep), 0, stream, p, (uint32_t)vecs);
  return hipGetLastError();
}

}  // namespace mss
