// 8-bit activation checkpoints (gfx950): a [rows, cols] tensor to and from the
// form of rows.hpp.
//
// A thread takes vectors of eight columns (four neighbouring lanes one block of
// 32), kVecs of them a workgroup's width apart with every load issued before
// the first use, so a wave keeps kVecs * 64 vectors in flight: the kernels move
// 2 + 33/32 bytes an element (bf16) and are bound by HBM: 32768 x 5120 packs in
// 103 us and unpacks in 83 us (5.0 and 6.1 TB/s).  Rows of any length and
// stride: a workgroup takes a span of the padded vectors, finds the row of its
// first one with one scalar division and each thread its own with a 32-bit one.
#include "launch.hpp"
#include "rows.hpp"

namespace mss {
namespace {

constexpr int kThreads = 256, kVecs = 4, kSpan = kThreads * kVecs;

struct Args {
  const void* src;
  void* dst;
  int8_t* q;
  uint8_t* scale;
  int64_t stride;  // of the tensor's rows, elements
  int64_t rows;
  int cols, pitch;
  uint32_t vecs;   // per padded row
};

// The row and first column of the span's vector t (t < vecs + kSpan).
struct Spot {
  int64_t row;
  int col;
};
__device__ __forceinline__ Spot spot(const Args& a, int64_t row0, uint32_t rem0, uint32_t t) {
  const uint32_t v = rem0 + t, r = v / a.vecs;
  return {row0 + r, (int)(v - r * a.vecs) * 8};
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) pack8_kernel(Args a) {
  constexpr int S = F32 ? kSrcF32 : kSrcBf16;
  const int64_t first = (int64_t)blockIdx.x * kSpan, row0 = first / a.vecs;
  const uint32_t rem0 = (uint32_t)(first - row0 * a.vecs);
  Raw<S> raw[kVecs];
  Spot at[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    at[i] = spot(a, row0, rem0, i * kThreads + threadIdx.x);
    const char* p = static_cast<const char*>(a.src) + at[i].row * a.stride * (F32 ? 4 : 2);
    raw[i] = load_raw<S>(p, nullptr, at[i].col, at[i].row < a.rows ? a.cols - at[i].col : 0);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float v[8];
    widen<S>(raw[i], v);
    store_p8(a.q + at[i].row * a.pitch, a.scale + at[i].row * (a.pitch >> 5), at[i].col,
             at[i].row < a.rows ? a.pitch : 0, v);
  }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) unpack8_kernel(Args a) {
  const int64_t first = (int64_t)blockIdx.x * kSpan, row0 = first / a.vecs;
  const uint32_t rem0 = (uint32_t)(first - row0 * a.vecs);
  Raw<kSrcP8> raw[kVecs];
  Spot at[kVecs];
  int n[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    at[i] = spot(a, row0, rem0, i * kThreads + threadIdx.x);
    n[i] = at[i].row < a.rows ? a.cols - at[i].col : 0;
    raw[i] = load_raw<kSrcP8>(a.q + at[i].row * a.pitch, a.scale + at[i].row * (a.pitch >> 5), at[i].col, n[i]);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float v[8];
    widen<kSrcP8>(raw[i], v);
    if (n[i] > 0) store8<F32>(static_cast<char*>(a.dst) + at[i].row * a.stride * (F32 ? 4 : 2), at[i].col, n[i], v);
  }
}

Args args_of(const Ckpt8Params& p) {
  const int64_t pitch = (p.cols + 31) / 32 * 32;
  return Args{p.src, p.dst, p.q, p.scale, p.stride, p.rows, (int)p.cols, (int)pitch, (uint32_t)(pitch / 8)};
}
unsigned grid_of(const Args& a) { return (unsigned)((a.rows * a.vecs + kSpan - 1) / kSpan); }

}  // namespace

hipError_t launch_pack8(const Ckpt8Params& p, hipStream_t stream) {
  const Args a = args_of(p);
  if (p.bf16) hipLaunchKernelGGL(pack8_kernel<false>, dim3(grid_of(a)), dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL(pack8_kernel<true>, dim3(grid_of(a)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_unpack8(const Ckpt8Params& p, hipStream_t stream) {
  const Args a = args_of(p);
  if (p.bf16) hipLaunchKernelGGL(unpack8_kernel<false>, dim3(grid_of(a)), dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL(unpack8_kernel<true>, dim3(grid_of(a)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace mss
