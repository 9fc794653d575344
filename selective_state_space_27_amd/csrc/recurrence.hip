// Gated linear recurrence: scan over whole sequences and its gradient (gfx950).
// Definitions in include/mambascan.h, arithmetic in recurrence.hpp.
//
// A thread walks one channel of one sequence.
#include "launch.hpp"
#include "norm_common.hpp"
#include "recurrence.hpp"

namespace mss {
namespace {

template <bool BF16>
__device__ __forceinline__ float load_el(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store_el(void* p, int64_t i, float v) {
  if constexpr (BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
  else static_cast<float*>(p)[i] = v;
}

template <bool BF16>
__global__ void __launch_bounds__(64) recurrence_fwd_kernel(RecurrenceFwdParams p) {
  const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (d == 0 && blockIdx.y == 0) *static_cast<int*>(p.workspace) = 0;  // the status word: nothing waits here
  if (d >= p.dim) return;
  const int64_t b = blockIdx.y, nchunks = (p.seqlen + kRecurrenceChunk - 1) / kRecurrenceChunk;
  const float k = p.c * softplus_of(p.lam[d]);
  float h = p.h0 != nullptr ? p.h0[b * p.dim + d] : 0.f;
  for (int64_t t = 0; t < p.seqlen; ++t) {
    const int64_t row = b * p.seqlen + t;
    if (p.states != nullptr && t % kRecurrenceChunk == 0)
      p.states[(b * nchunks + t / kRecurrenceChunk) * p.dim + d] = h;
    const float x = load_el<BF16>(p.x, row * p.x_stride + d);
    const float m = one_minus_exp<false>(k * sigmoid_of<!BF16>(load_el<BF16>(p.gate_a, row * p.gate_a_stride + d)));
    const float in = sqrtf(m * (2.0f - m)) * sigmoid_of<!BF16>(load_el<BF16>(p.gate_x, row * p.gate_x_stride + d)) * x;
    const bool start = p.starts != nullptr && p.starts[row] != 0;
    h = (start ? 0.f : __builtin_fmaf(-m, h, h)) + in;
    store_el<BF16>(p.y, row * p.y_stride + d, h);
  }
  if (p.h_last != nullptr) p.h_last[b * p.dim + d] = h;
}

template <bool BF16>
__global__ void __launch_bounds__(64) recurrence_bwd_kernel(RecurrenceBwdParams p, float* part) {
  __shared__ float before[kRecurrenceChunk][64];
  const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (d == 0 && blockIdx.y == 0) *static_cast<int*>(p.workspace) = 0;  // the status word: nothing waits here
  if (d >= p.dim) return;
  const int64_t b = blockIdx.y, nchunks = (p.seqlen + kRecurrenceChunk - 1) / kRecurrenceChunk;
  const float sp = softplus_of(p.lam[d]), k = p.c * sp;
  float e = p.dh_last != nullptr ? p.dh_last[b * p.dim + d] : 0.f;  // gradient of the state after the step
  float dlam = 0.f;
  for (int64_t ch = nchunks - 1; ch >= 0; --ch) {
    const int64_t t0 = ch * kRecurrenceChunk;
    const int n = (int)(p.seqlen - t0 < kRecurrenceChunk ? p.seqlen - t0 : kRecurrenceChunk);
    float h = p.states[(b * nchunks + ch) * p.dim + d];
    for (int j = 0; j < n; ++j) {
      const int64_t row = b * p.seqlen + t0 + j;
      before[j][threadIdx.x] = h;
      const float m = one_minus_exp<false>(k * sigmoid_of<!BF16>(load_el<BF16>(p.gate_a, row * p.gate_a_stride + d)));
      const float in = sqrtf(m * (2.0f - m)) *
                       sigmoid_of<!BF16>(load_el<BF16>(p.gate_x, row * p.gate_x_stride + d)) *
                       load_el<BF16>(p.x, row * p.x_stride + d);
      const bool start = p.starts != nullptr && p.starts[row] != 0;
      h = (start ? 0.f : __builtin_fmaf(-m, h, h)) + in;
    }
    for (int j = n - 1; j >= 0; --j) {
      const int64_t row = b * p.seqlen + t0 + j;
      const bool start = p.starts != nullptr && p.starts[row] != 0;
      float rr, ri;
      const float r = sigmoid_of<!BF16>(load_el<BF16>(p.gate_a, row * p.gate_a_stride + d), rr);
      const float i = sigmoid_of<!BF16>(load_el<BF16>(p.gate_x, row * p.gate_x_stride + d), ri);
      const float x = load_el<BF16>(p.x, row * p.x_stride + d);
      const float s = finite_decay(k * r), m = one_minus_exp<false>(s), beta = sqrtf(m * (2.0f - m)), a = 1.0f - m;
      const float g = load_el<BF16>(p.dy, row * p.dy_stride + d) + e;
      const float gi = g * i, gix = gi * x;
      const float from_beta = m > 0.f ? a * a * (s / beta) * gix : (s - s) * gix;
      const float big = from_beta - (start ? 0.f : s * a * (g * before[j][threadIdx.x]));
      store_el<BF16>(p.dx, row * p.dx_stride + d, gi * beta);
      store_el<BF16>(p.dgate_x, row * p.dgate_x_stride + d, gix * beta * ri);
      store_el<BF16>(p.dgate_a, row * p.dgate_a_stride + d, big * rr);
      dlam += big;
      e = start ? 0.f : __builtin_fmaf(-m, g, g);
    }
  }
  if (p.dh0 != nullptr) p.dh0[b * p.dim + d] = e;
  part[b * p.dim + d] = dlam * softplus_rate(p.lam[d], sp);
}

dim3 grid_of(int64_t batch, int64_t dim) { return dim3((unsigned)((dim + 63) / 64), (unsigned)batch); }

}  // namespace

size_t recurrence_fwd_workspace_bytes(int64_t, int64_t, int64_t, bool) { return 256; }

hipError_t launch_recurrence_fwd(const RecurrenceFwdParams& p, hipStream_t stream) {
  if (p.bf16) hipLaunchKernelGGL(recurrence_fwd_kernel<true>, grid_of(p.batch, p.dim), dim3(64), 0, stream, p);
  else hipLaunchKernelGGL(recurrence_fwd_kernel<false>, grid_of(p.batch, p.dim), dim3(64), 0, stream, p);
  return hipGetLastError();
}

size_t recurrence_bwd_workspace_bytes(int64_t batch, int64_t, int64_t dim, bool) {
  return 256 + (size_t)batch * dim * sizeof(float);
}

hipError_t launch_recurrence_bwd(const RecurrenceBwdParams& p, hipStream_t stream) {
  float* part = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + 256);
  if (p.bf16) hipLaunchKernelGGL(recurrence_bwd_kernel<true>, grid_of(p.batch, p.dim), dim3(64), 0, stream, p, part);
  else hipLaunchKernelGGL(recurrence_bwd_kernel<false>, grid_of(p.batch, p.dim), dim3(64), 0, stream, p, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  SumPartialsArgs a{};
  a.part = part;
  a.dweight = p.dlam;
  a.nparts = p.batch;
  a.cols = p.dim;
  a.nout = 1;
  return launch_sum_partials(a, stream);
}

}  // namespace mss
