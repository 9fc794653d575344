// Norm after a mixer, fused with its gate (gfx950): forward and backward.
//
// Per row and group of columns, with RMS(v) = v rstd(v), rstd(v) = 1 /
// sqrt(mean(v^2) + eps) over the group, s(z) = z sigma(z), s'(z) = sigma(z)
// (1 + z (1 - sigma(z))):
//   gate first:  v = y s(z);  out = RMS(v) w      (no z: v = y)
//   norm first:  out = RMS(y) w s(z)
// Backward, g the gradient of the normed values times w:
//   gate first:  g = dout w;  dv = rstd g - v rstd^3 mean(g v);
//                dy = dv s(z);  dz = dv y s'(z);  dw = sum_rows dout v rstd
//   norm first:  g = dout w s(z);  dy = rstd g - y rstd^3 mean(g y);
//                dz = dout w y rstd s'(z);  dw = sum_rows dout s(z) y rstd
// rstd is formed again in the backward, in the same reduction as mean(g v).
//
// Every element is read once and written once: both directions are bound by
// HBM.  Rows are laid over lanes as norm_common.hpp describes; a group of
// columns has its own workgroups (grid y).  32768 x 5120, y fp32, z bf16: forward
// 231 us (5.8 TB/s), with the 8-bit forms of y and z 303 us (5.6), backward 444
// us (5.3), from the 8-bit forms 325 us (5.2).
#include <type_traits>

#include "norm_common.hpp"

namespace mss {
namespace {

enum : int { kNoGate = 0, kGateFirst = 1, kNormFirst = 2 };

// sigma(z) = 1 / (1 + 2^t), t = -z log2(e); the limits come out right (exp2
// overflows to inf, 1 / inf = 0).  t rounded to fp32 puts sigma of a nearly closed
// gate off by up to 64 units of 2^-24 (z near -60).  For fp32 gates what t leaves
// out, lo, is put back: 2^(t + lo) = 2^t (1 + lo ln 2), lo below 2^-16.  A gate from
// bf16 or the 8-bit form is itself known to |z| 2^-9 of sigma, 2^15 times as much,
// and spares the instructions (they cost 768 columns from bf16 7% and more).
// Past +-192 sigma is 0 or 1 in fp32 already; the limit keeps infinities out of lo.
// It also drops a NaN, which comes back where z is multiplied in.
template <int SRC>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (SRC == kSrcF32) {
    constexpr float kLog2eRest = (float)(1.4426950408889634 - (double)kLog2e), kLn2 = 0.69314718f;
    const float c = __builtin_amdgcn_fmed3f(z, -192.f, 192.f), t = -c * kLog2e;
    const float lo = __builtin_fmaf(-c, kLog2eRest, __builtin_fmaf(-c, kLog2e, -t));
    return rcp_fast(1.0f + exp2_fast(t) * __builtin_fmaf(lo, kLn2, 1.0f));
  } else {
    return rcp_fast(1.0f + exp2_fast(-z * kLog2e));
  }
}

struct FwdArgs {
  GatedNormFwdParams p;
  int pitch;  // of the 8-bit forms
  int gcols;  // columns of a group
};

template <bool Y32, bool IO32, int MODE, int LANES, int K, int T, bool WHOLE>
__global__ void __launch_bounds__(T)
    __attribute__((amdgpu_waves_per_eu(T == 768 ? 3 : K == 2 ? 4 : 6))) gated_norm_fwd_kernel(FwdArgs a) {
  constexpr int SY = Y32 ? kSrcF32 : kSrcBf16, SZ = IO32 ? kSrcF32 : kSrcBf16;
  __shared__ float lds[LANES ? 1 : kRowSumFloats];
  int half = 0;
  const Place<LANES> at;
  const int c0 = (int)blockIdx.y * a.gcols;
  const float inv = 1.0f / (float)a.gcols;
  int col[K], n[K];
  float w[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    col[k] = c0 + at.col(k);
    n[k] = a.gcols - at.col(k);
    load_w<WHOLE>(a.p.weight, col[k], n[k], w[k]);
  }
  const int64_t step = (int64_t)gridDim.x * at.nseg;
  int64_t row = (int64_t)blockIdx.x * at.nseg + at.seg;
  Raw<SY> ny[K];
  Raw<SZ> nz[MODE != kNoGate ? K : 1];
  auto fetch = [&](int64_t i) {
    const char* yr = static_cast<const char*>(a.p.y) + i * a.p.y_stride * (Y32 ? 4 : 2);
    const char* zr = static_cast<const char*>(a.p.z) + i * a.p.z_stride * (IO32 ? 4 : 2);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      ny[k] = load_raw<SY, WHOLE>(yr, nullptr, col[k], n[k]);
      if constexpr (MODE != kNoGate) nz[k] = load_raw<SZ, WHOLE>(zr, nullptr, col[k], n[k]);
    }
  };
  if (row < a.p.rows) fetch(row);
  for (; row < a.p.rows; row += step) {
    float y[K][8], z[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      widen<SY>(ny[k], y[k]);
      if constexpr (MODE != kNoGate) widen<SZ>(nz[k], z[k]);
    }
    if (row + step < a.p.rows) fetch(row + step);
    const int64_t prow = row * a.pitch, srow = row * (a.pitch >> 5);
    if (a.p.y_q != nullptr) {
      const int pend = a.p.ngroups == 1 ? a.pitch : c0 + a.gcols;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        store_p8(a.p.y_q + prow, a.p.y_scale + srow, col[k], pend, y[k]);
        if constexpr (MODE != kNoGate) store_p8(a.p.z_q + prow, a.p.z_scale + srow, col[k], pend, z[k]);
      }
    }
    float sum[1] = {};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (MODE == kGateFirst) y[k][j] *= z[k][j] * sigmoid<SZ>(z[k][j]);
        sum[0] = __builtin_fmaf(y[k][j], y[k][j], sum[0]);
      }
    row_sums<LANES>(sum, lds, half);
    const float rstd = rsqrtf(__builtin_fmaf(sum[0], inv, a.p.eps));
    char* out = static_cast<char*>(a.p.out) + row * a.p.out_stride * (IO32 ? 4 : 2);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] = y[k][j] * rstd * w[k][j];
        if constexpr (MODE == kNormFirst) o[j] *= z[k][j] * sigmoid<SZ>(z[k][j]);
      }
      if (n[k] > 0) store8<IO32, WHOLE>(out, col[k], n[k], o);
      if (a.p.out_q != nullptr) {
        as_stored<IO32>(o);  // the form of the output as it is stored
        store_p8(a.p.out_q + prow, a.p.out_scale + srow, col[k], a.p.ngroups == 1 ? a.pitch : c0 + a.gcols, o);
      }
    }
  }
}

struct BwdArgs {
  GatedNormBwdParams p;
  float* part;  // [blocks][cols]
  int pitch;
  int gcols;
  int* status;
};

template <bool Y32, bool IO32, bool PACKED, int MODE, int LANES, int K, int T, bool WHOLE>
__global__ void __launch_bounds__(T)
    __attribute__((amdgpu_waves_per_eu(T == 768 ? 3 : 4))) gated_norm_bwd_kernel(BwdArgs a) {
  constexpr int SO = IO32 ? kSrcF32 : kSrcBf16;
  constexpr int SY = PACKED ? kSrcP8 : Y32 ? kSrcF32 : kSrcBf16, SZ = PACKED ? kSrcP8 : SO;
  // The next row is fetched ahead where the registers hold it: not with two
  // vectors per thread in workgroups of up to 1024, nor in fp32 with a gate where
  // rows are not whole vectors (4096 x 10001: 165 us, ahead 177 to 188).  With two,
  // the row is kept as loaded and widened a second time after the sums (8192 x 10240
  // from the 8-bit forms: 167 us; in workgroups of up to 1024 333 without and 479
  // with the next row ahead, for registers that spill).
  constexpr bool kHeld = T == 768 && (WHOLE || PACKED || !IO32 || MODE == kNoGate);
  constexpr bool kAhead = K == 1 || kHeld, kRenew = K == 2;
  __shared__ float lds[LANES ? kPartialLds : kRowSumFloats];
  int half = 0;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = 0;
  const Place<LANES> at;
  const int c0 = (int)blockIdx.y * a.gcols;
  const float inv = 1.0f / (float)a.gcols;
  int col[K], n[K];
  float w[K][8], dw[K][8] = {};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    col[k] = c0 + at.col(k);
    n[k] = a.gcols - at.col(k);
    load_w<WHOLE>(a.p.weight, col[k], n[k], w[k]);
  }
  const int64_t step = (int64_t)gridDim.x * at.nseg;
  int64_t row = (int64_t)blockIdx.x * at.nseg + at.seg;
  Raw<SO> nd[K];
  Raw<SY> ny[K];
  Raw<SZ> nz[MODE != kNoGate ? K : 1];
  auto fetch = [&](int64_t i) {
    const char* dr = static_cast<const char*>(a.p.dout) + i * a.p.dout_stride * (IO32 ? 4 : 2);
    const char* yr = static_cast<const char*>(a.p.y) + i * (PACKED ? a.pitch : a.p.y_stride * (Y32 ? 4 : 2));
    const char* zr = static_cast<const char*>(a.p.z) + i * (PACKED ? a.pitch : a.p.z_stride * (IO32 ? 4 : 2));
    const uint8_t* ys = PACKED ? a.p.y_scale + i * (a.pitch >> 5) : nullptr;
    const uint8_t* zs = PACKED ? a.p.z_scale + i * (a.pitch >> 5) : nullptr;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      nd[k] = load_raw<SO, WHOLE>(dr, nullptr, col[k], n[k]);
      ny[k] = load_raw<SY, WHOLE>(yr, ys, col[k], n[k]);
      if constexpr (MODE != kNoGate) nz[k] = load_raw<SZ, WHOLE>(zr, zs, col[k], n[k]);
    }
  };
  if (kAhead && row < a.p.rows) fetch(row);
  for (; row < a.p.rows; row += step) {
    if constexpr (!kAhead) fetch(row);
    Raw<SO> rd[K];
    Raw<SY> ry[K];
    Raw<SZ> rz[MODE != kNoGate ? K : 1];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      rd[k] = nd[k], ry[k] = ny[k];
      if constexpr (MODE != kNoGate) rz[k] = nz[k];
    }
    if (kAhead && row + step < a.p.rows) fetch(row + step);
    float d[K][8], y[K][8], z[K][8];
    auto widen_row = [&](int k) {
      widen<SO>(rd[k], d[k]), widen<SY>(ry[k], y[k]);
      if constexpr (MODE != kNoGate) widen<SZ>(rz[k], z[k]);
    };
    float sum[2] = {};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      widen_row(k);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float g = d[k][j] * w[k][j], v = y[k][j];
        if constexpr (MODE != kNoGate) {
          const float s = z[k][j] * sigmoid<SZ>(z[k][j]);
          if constexpr (MODE == kGateFirst) v *= s;
          else g *= s;
        }
        sum[0] = __builtin_fmaf(v, v, sum[0]);
        sum[1] = __builtin_fmaf(g, v, sum[1]);
      }
      if constexpr (kRenew) {
        renew(rd[k]), renew(ry[k]);
        if constexpr (MODE != kNoGate) renew(rz[k]);
        __builtin_amdgcn_sched_barrier(0);  // one vector at a time
      }
    }
    row_sums<LANES>(sum, lds, half);
    const float rstd = rsqrtf(__builtin_fmaf(sum[0], inv, a.p.eps));
    const float c1 = sum[1] * inv * rstd * rstd * rstd;
    char* dyr = static_cast<char*>(a.p.dy) + row * a.p.dy_stride * (Y32 ? 4 : 2);
    char* dzr = static_cast<char*>(a.p.dz) + row * a.p.dz_stride * (IO32 ? 4 : 2);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float dy[8], dz[8];
      if constexpr (kRenew) widen_row(k);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float g = d[k][j] * w[k][j];
        if constexpr (MODE == kNoGate) {
          dy[j] = rstd * g - y[k][j] * c1;
          dw[k][j] = __builtin_fmaf(d[k][j], y[k][j] * rstd, dw[k][j]);
        } else {
          const float sg = sigmoid<SZ>(z[k][j]), s = z[k][j] * sg;
          const float ds = __builtin_fmaf(s, 1.0f - sg, sg);  // sigma (1 + z (1 - sigma))
          if constexpr (MODE == kGateFirst) {
            const float v = y[k][j] * s, dv = rstd * g - v * c1;
            dw[k][j] = __builtin_fmaf(d[k][j], v * rstd, dw[k][j]);
            dy[j] = dv * s;
            dz[j] = dv * y[k][j] * ds;
          } else {
            const float nh = y[k][j] * rstd;
            dw[k][j] = __builtin_fmaf(d[k][j], nh * s, dw[k][j]);
            dy[j] = rstd * (g * s) - y[k][j] * c1;
            dz[j] = g * nh * ds;
          }
        }
      }
      if (n[k] > 0) {
        store8<Y32, WHOLE>(dyr, col[k], n[k], dy);
        if constexpr (MODE != kNoGate) store8<IO32, WHOLE>(dzr, col[k], n[k], dz);
      }
      if constexpr (kRenew) __builtin_amdgcn_sched_barrier(0);
    }
  }
  float* part = a.part + (int64_t)blockIdx.x * a.p.cols + c0;
#pragma unroll
  for (int k = 0; k < K; ++k) store_partial<LANES, WHOLE>(part, at.col(k), n[k], dw[k], lds);
}

template <bool Y32, bool IO32, int MODE>
hipError_t fwd_mode(const GatedNormFwdParams& p, hipStream_t stream) {
  const int64_t gcols = p.cols / p.ngroups;
  const NormShape s = norm_shape(gcols);
  const dim3 grid((unsigned)norm_blocks(s, p.rows, p.ngroups, false), (unsigned)p.ngroups), block((unsigned)s.threads);
  const FwdArgs a{p, (int)((p.cols + 31) / 32 * 32), (int)gcols};
  return with_shape(s, gcols % 8 == 0, [&](auto lanes, auto k, auto t, auto whole) {
    hipLaunchKernelGGL((gated_norm_fwd_kernel<Y32, IO32, MODE, lanes.value, k.value, t.value, whole.value>), grid, block, 0, stream, a);
    return hipGetLastError();
  });
}

template <bool Y32, bool IO32>
hipError_t fwd_typed(const GatedNormFwdParams& p, hipStream_t stream) {
  if (p.z == nullptr) return fwd_mode<Y32, IO32, kNoGate>(p, stream);
  return p.norm_first ? fwd_mode<Y32, IO32, kNormFirst>(p, stream) : fwd_mode<Y32, IO32, kGateFirst>(p, stream);
}

template <bool Y32, bool IO32, bool PACKED, int MODE>
hipError_t bwd_mode(const GatedNormBwdParams& p, hipStream_t stream) {
  const int64_t gcols = p.cols / p.ngroups;
  const NormShape s = norm_shape(gcols);
  const int64_t blocks = norm_blocks(s, p.rows, p.ngroups, true);
  const BwdArgs a{p, reinterpret_cast<float*>(static_cast<char*>(p.workspace) + 256), (int)((p.cols + 31) / 32 * 32),
                  (int)gcols, static_cast<int*>(p.workspace)};
  const hipError_t e = with_shape(s, gcols % 8 == 0, [&](auto lanes, auto k, auto t, auto whole) {
    hipLaunchKernelGGL((gated_norm_bwd_kernel<Y32, IO32, PACKED, MODE, lanes.value, k.value, t.value, whole.value>),
                       dim3((unsigned)blocks, (unsigned)p.ngroups), dim3((unsigned)s.threads), 0, stream, a);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  return launch_sum_partials(
      SumPartialsArgs{a.part, p.dweight, nullptr, nullptr, nullptr, nullptr, 1.f, blocks, p.cols, 1}, stream);
}

template <bool Y32, bool IO32, bool PACKED>
hipError_t bwd_gate(const GatedNormBwdParams& p, hipStream_t stream) {
  if (p.z == nullptr) return bwd_mode<Y32, IO32, PACKED, kNoGate>(p, stream);
  return p.norm_first ? bwd_mode<Y32, IO32, PACKED, kNormFirst>(p, stream)
                      : bwd_mode<Y32, IO32, PACKED, kGateFirst>(p, stream);
}

template <bool Y32, bool IO32>
hipError_t bwd_typed(const GatedNormBwdParams& p, hipStream_t stream) {
  return p.y_scale != nullptr ? bwd_gate<Y32, IO32, true>(p, stream) : bwd_gate<Y32, IO32, false>(p, stream);
}

}  // namespace

hipError_t launch_gated_norm_fwd(const GatedNormFwdParams& p, hipStream_t stream) {
  if (!p.io_bf16) return fwd_typed<true, true>(p, stream);
  return p.y_bf16 ? fwd_typed<false, false>(p, stream) : fwd_typed<true, false>(p, stream);
}

size_t gated_norm_bwd_workspace_bytes(int64_t rows, int64_t cols, int64_t ngroups) {
  return 256 + (size_t)norm_blocks(norm_shape(cols / ngroups), rows, ngroups, true) * (size_t)cols * sizeof(float);
}

hipError_t launch_gated_norm_bwd(const GatedNormBwdParams& p, hipStream_t stream) {
  if (!p.io_bf16) return bwd_typed<true, true>(p, stream);
  return p.y_bf16 ? bwd_typed<false, false>(p, stream) : bwd_typed<true, false>(p, stream);
}

}  // namespace mss
