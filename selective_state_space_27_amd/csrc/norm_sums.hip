// Sums of the workgroups' partial rows for the weights' gradients (gfx950).
//
// 16 columns x 64 slices of the partial rows per workgroup of 1024 threads:
// each thread sums its slice's rows in order, the slices' sums meet in LDS in a
// fixed order.  4 to 6 us (256 rows of 2560 to 1024 rows of 2 x 1001), of latency
// and of reading: 16 columns are 64 bytes, so each 128-byte line is read by two
// workgroups, or three where rows are not whole lines (24.2 MB for the 8.2 MB of
// 1024 x 2 x 1001).  A layout with 256 rows in flight took the same.
#include "norm_common.hpp"

namespace mss {
namespace {

constexpr int kCols = 16, kSlices = 64;
// Columns of a launch: it has 64 threads a column and, along one axis of the
// grid, fewer than 2^32 in all.
constexpr int64_t kLaunchCols = 1LL << 25;

__global__ void __launch_bounds__(kCols* kSlices) sum_partials_kernel(SumPartialsArgs a) {
  __shared__ float lds[kSlices][kCols + 1];
  const int c = threadIdx.x % kCols, s = threadIdx.x / kCols;
  const int64_t col = a.first + (int64_t)blockIdx.x * kCols + c;
  const int64_t pitch = (int64_t)a.nout * a.cols;
  float v = 0.f;
  if (col < a.cols) {
    const float* p = a.part + (int64_t)blockIdx.y * a.cols + col;
    int64_t i = s;
    for (; i + 3 * kSlices < a.nparts; i += 4 * kSlices) {
      const float v0 = p[i * pitch], v1 = p[(i + kSlices) * pitch], v2 = p[(i + 2 * kSlices) * pitch],
                  v3 = p[(i + 3 * kSlices) * pitch];
      v += (v0 + v1) + (v2 + v3);
    }
    for (; i < a.nparts; i += kSlices) v += p[i * pitch];
  }
  lds[s][c] = v;
  __syncthreads();
  for (int h = kSlices / 2; h > 0; h >>= 1) {
    if (s < h) lds[s][c] += lds[s + h][c];
    __syncthreads();
  }
  if (s != 0 || col >= a.cols) return;
  v = lds[0][c];
  if (blockIdx.y == 0) {
    a.dweight[col] = v;
    return;
  }
  if (a.dgamma != nullptr) a.dgamma[col] = v * (a.post != nullptr ? a.scale * a.post[col] : a.scale);
  if (a.dpost != nullptr) a.dpost[col] = v * (a.gamma != nullptr ? a.scale * a.gamma[col] : a.scale);
}

}  // namespace

hipError_t launch_sum_partials(const SumPartialsArgs& args, hipStream_t stream) {
  SumPartialsArgs a = args;
  for (a.first = 0; a.first < a.cols; a.first += kLaunchCols) {
    const int64_t cols = a.cols - a.first < kLaunchCols ? a.cols - a.first : kLaunchCols;
    hipLaunchKernelGGL(sum_partials_kernel, dim3((unsigned)((cols + kCols - 1) / kCols), (unsigned)a.nout),
                       dim3(kCols * kSlices), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mss
