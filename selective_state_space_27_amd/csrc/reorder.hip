// Reordering of beams' states in place (gfx950): state[b, k] = state[b, parents[b, k]].
//
// The rows of one sequence's beams lie side by side in `beams` rows of
// row_bytes; a thread owns the same 16 bytes of all of them, so that it has read
// every row before it writes any and no other thread touches them.  What it read
// waits in LDS, in slots of its own: no barrier is needed, and a wave has all of a
// column's reads under way at once.  Rows that stay are neither read nor written.
//
// Bound by memory: 32 x 8 beams, four layers of 380 KB each, half of the rows moving
// (388 MB read and written), 76 us on inputs from memory (5.1 TB/s, what a large copy
// reaches).  The same inputs again and again, partly in the last-level cache: 61 us with
// non-temporal stores, 80 us without (what is written then takes the place of what is read
// next in that cache), 108 us with eight beams in registers instead of LDS.
#include "launch.hpp"
#include "rows.hpp"

namespace mss {
namespace {

constexpr int kMaxStates = 32;  // of a launch
constexpr int kMaxBeams = 64;
constexpr int kThreadsReorder = 64;

struct ReorderArgs {
  uint8_t* state[kMaxStates];
  int64_t row_bytes[kMaxStates];
  uint32_t first[kMaxStates + 1];  // workgroup of each state's first columns
  const int64_t* parents;
  int beams, count;
};

// 16 bytes of a row, or its last n.
__device__ __forceinline__ u32x4 load_bytes(const uint8_t* p, int64_t n) {
  if (n >= 16) return *reinterpret_cast<const u32x4_a1*>(p);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 15; ++j)
    if (j < n) v[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  return v;
}
__device__ __forceinline__ void store_bytes(uint8_t* p, int64_t n, u32x4 v) {
  if (n >= 16) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a1*>(p));
    return;
  }
#pragma unroll
  for (int j = 0; j < 15; ++j)
    if (j < n) p[j] = (uint8_t)(v[j >> 2] >> (8 * (j & 3)));
}

__global__ void __launch_bounds__(kThreadsReorder) reorder_kernel(ReorderArgs a) {
  extern __shared__ u32x4 slots[];  // [beams][threads]
  int s = 0;
  while (s + 1 < a.count && blockIdx.x >= a.first[s + 1]) ++s;
  const int64_t row = a.row_bytes[s], col = ((int64_t)(blockIdx.x - a.first[s]) * kThreadsReorder + threadIdx.x) * 16;
  if (col >= row) return;
  uint8_t* base = a.state[s] + (int64_t)blockIdx.y * a.beams * row + col;
  const int64_t* parents = a.parents + (int64_t)blockIdx.y * a.beams;
  const int64_t n = row - col;
  for (int k = 0; k < a.beams; ++k) {
    const int64_t from = parents[k];
    if (from != k && from >= 0 && from < a.beams)
      slots[k * kThreadsReorder + threadIdx.x] = load_bytes(base + from * row, n);
  }
  for (int k = 0; k < a.beams; ++k) {
    const int64_t from = parents[k];
    if (from != k && from >= 0 && from < a.beams) store_bytes(base + k * row, n, slots[k * kThreadsReorder + threadIdx.x]);
  }
}

}  // namespace

hipError_t launch_reorder_states(const ReorderParams& p, hipStream_t stream) {
  for (int64_t at = 0; at < p.count; at += kMaxStates) {
    ReorderArgs a{};
    a.parents = p.parents;
    a.beams = (int)p.beams;
    a.count = (int)(p.count - at < kMaxStates ? p.count - at : kMaxStates);
    for (int s = 0; s < a.count; ++s) {
      a.state[s] = static_cast<uint8_t*>(p.states[at + s]);
      a.row_bytes[s] = p.row_bytes[at + s];
      a.first[s + 1] = a.first[s] + (uint32_t)((a.row_bytes[s] + 16 * kThreadsReorder - 1) / (16 * kThreadsReorder));
    }
    hipLaunchKernelGGL(reorder_kernel, dim3(a.first[a.count], (unsigned)p.batch), dim3(kThreadsReorder),
                       (size_t)a.beams * kThreadsReorder * 16, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mss
