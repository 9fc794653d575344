// One token of the gated linear recurrence (gfx950): h_out = a h + beta i x per
// channel, the state read from the parent beam's row where parents are given.
// Definitions in include/mambascan.h, arithmetic in recurrence.hpp.
//
// One channel per thread, one workgroup row per state row.
#include "launch.hpp"
#include "recurrence.hpp"

namespace mss {
namespace {

template <bool BF16>
__global__ void __launch_bounds__(256) recurrence_step_kernel(RecurrenceStepParams p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.rows * p.dim) return;
  const int64_t row = i / p.dim, d = i - row * p.dim;
  int64_t from = row;
  if (p.parents != nullptr) {
    const int64_t parent = p.parents[row];
    if (parent >= 0 && parent < p.beams) from = row / p.beams * p.beams + parent;
  }
  float x, ga, gx;
  if constexpr (BF16) {
    x = bf16_to_f32(static_cast<const uint16_t*>(p.x)[row * p.x_stride + d]);
    ga = bf16_to_f32(static_cast<const uint16_t*>(p.gate_a)[row * p.gate_a_stride + d]);
    gx = bf16_to_f32(static_cast<const uint16_t*>(p.gate_x)[row * p.gate_x_stride + d]);
  } else {
    x = static_cast<const float*>(p.x)[row * p.x_stride + d];
    ga = static_cast<const float*>(p.gate_a)[row * p.gate_a_stride + d];
    gx = static_cast<const float*>(p.gate_x)[row * p.gate_x_stride + d];
  }
  const float k = decay_rate(p.c, p.lam[d]), h = p.h[from * p.dim + d];
  const float n = exp_less_one<false>(k * sigmoid_of<!BF16>(ga));
  const float out = __builtin_fmaf(n, h, h) + beta_of(n) * sigmoid_of<!BF16>(gx) * x;
  p.h_out[row * p.dim + d] = out;
  if constexpr (BF16) static_cast<uint16_t*>(p.y)[row * p.y_stride + d] = f32_to_bf16(out);
  else static_cast<float*>(p.y)[row * p.y_stride + d] = out;
}

}  // namespace

hipError_t launch_recurrence_step(const RecurrenceStepParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.rows * p.dim + 255) / 256));
  if (p.bf16) hipLaunchKernelGGL(recurrence_step_kernel<true>, grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(recurrence_step_kernel<false>, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mss
