// Norm before a block, fused with the residual (gfx950): forward and backward.
//
// Per row, with RMS(v) = v rstd(v), rstd(v) = 1 / sqrt(mean(v^2) + eps) and
// m_c = scale * gamma_c:
//   x' = post ? RMS(x) post : x;  r = residual + m x';  out = RMS(r) w.
// Backward at the stored r, with g = dout w:
//   dr = rstd g - r rstd^3 mean(g r) + dresidual_out      (dresidual)
//   dw = sum_rows dout r rstd
//   dx = m dr, or with post, n = RMS(x), g2 = m post dr:
//   dx = rstd_x g2 - x rstd_x^3 mean(g2 x);  with S = sum_rows dr n (n = x
//   without post):  dgamma = scale post S,  dpost = m S.  One sum serves both.
// rstd is formed again from r in the backward: sum(r^2) and sum(g r) are one
// reduction, so it costs nothing and needs no tensor of its own.
//
// Every element is read once and written once, nothing else: both directions
// are bound by HBM.  Rows are laid over lanes as norm_common.hpp describes.
// 32768 x 2560, bf16 with an fp32 residual: forward 180 us (5.6 TB/s), with the
// 8-bit form of out 205 us (5.2), backward 239 us (5.6; a device copy moves
// 5.1).  One row: 2.4 us, all latency.
#include <type_traits>

#include "norm_common.hpp"

namespace mss {
namespace {

struct FwdArgs {
  AddNormFwdParams p;
  int pitch;
};

template <bool RES32, bool IO32, bool POST, int LANES, int K, int T, bool WHOLE>
__global__ void __launch_bounds__(T)
    __attribute__((amdgpu_waves_per_eu(T == 768 ? 3 : K == 2 ? 4 : 6))) add_norm_fwd_kernel(FwdArgs a) {
  constexpr int SR = RES32 ? kSrcF32 : kSrcBf16, SX = IO32 ? kSrcF32 : kSrcBf16;
  __shared__ float lds[LANES ? 1 : kRowSumFloats];
  int half = 0;
  const Place<LANES> at;
  const int cols = (int)a.p.cols;
  const float inv = 1.0f / (float)cols;
  int col[K], n[K];
  float w[K][8], post[K][8], m[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    col[k] = at.col(k);
    n[k] = cols - col[k];
    load_w<WHOLE>(a.p.weight, col[k], n[k], w[k]);
    if constexpr (POST) load_w<WHOLE>(a.p.post_weight, col[k], n[k], post[k]);
    if (a.p.gamma != nullptr) {
      load_w<WHOLE>(a.p.gamma, col[k], n[k], m[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) m[k][j] *= a.p.scale;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) m[k][j] = a.p.scale;
    }
  }
  const int64_t step = (int64_t)gridDim.x * at.nseg;
  int64_t row = (int64_t)blockIdx.x * at.nseg + at.seg;
  Raw<SX> nx[K];
  Raw<SR> nr[K];
  auto fetch = [&](int64_t i) {
    const char* xr = static_cast<const char*>(a.p.x) + i * a.p.x_stride * (IO32 ? 4 : 2);
    const char* rr = static_cast<const char*>(a.p.residual) + i * a.p.residual_stride * (RES32 ? 4 : 2);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      nx[k] = load_raw<SX, WHOLE>(xr, nullptr, col[k], n[k]);
      nr[k] = load_raw<SR, WHOLE>(rr, nullptr, col[k], a.p.residual != nullptr ? n[k] : 0);
    }
  };
  if (row < a.p.rows) fetch(row);
  for (; row < a.p.rows; row += step) {
    float x[K][8], r[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) widen<SX>(nx[k], x[k]), widen<SR>(nr[k], r[k]);
    if (row + step < a.p.rows) fetch(row + step);
    float sum[1];
    if constexpr (POST) {
      sum[0] = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[0] = __builtin_fmaf(x[k][j], x[k][j], sum[0]);
      row_sums<LANES>(sum, lds, half);
      const float rx = rsqrtf(__builtin_fmaf(sum[0], inv, a.p.eps));
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[k][j] = x[k][j] * rx * post[k][j];
    }
    sum[0] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[k][j] = __builtin_fmaf(m[k][j], x[k][j], r[k][j]);
        sum[0] = __builtin_fmaf(r[k][j], r[k][j], sum[0]);
      }
    char* rout = static_cast<char*>(a.p.residual_out) + row * a.p.residual_out_stride * (RES32 ? 4 : 2);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (n[k] > 0) store8<RES32, WHOLE>(rout, col[k], n[k], r[k]);
    row_sums<LANES>(sum, lds, half);
    const float rstd = rsqrtf(__builtin_fmaf(sum[0], inv, a.p.eps));
    char* out = static_cast<char*>(a.p.out) + row * a.p.out_stride * (IO32 ? 4 : 2);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = r[k][j] * rstd * w[k][j];
      if (n[k] > 0) store8<IO32, WHOLE>(out, col[k], n[k], o);
      if (a.p.out_q != nullptr) {
        as_stored<IO32>(o);  // the form of the output as it is stored
        store_p8(a.p.out_q + row * a.pitch, a.p.out_scale + row * (a.pitch >> 5), col[k], a.pitch, o);
      }
    }
  }
}

struct BwdArgs {
  AddNormBwdParams p;
  float* part;  // [blocks][nout][cols]
  int nout;
  int pitch;
  int* status;
};

// EXTRA: 0 = x unused, 1 = gamma, 2 = post (and gamma where given).
template <bool RES32, bool IO32, bool PACKED, int EXTRA, int LANES, int K, int T, bool WHOLE>
__global__ void __launch_bounds__(T)
    __attribute__((amdgpu_waves_per_eu(LANES ? (EXTRA ? 3 : 4) : T == 768 ? 3 : K == 2 || EXTRA ? 4 : 5)))
    add_norm_bwd_kernel(BwdArgs a) {
  constexpr int SD = RES32 ? kSrcF32 : kSrcBf16, SO = IO32 ? kSrcF32 : kSrcBf16;
  constexpr int SR = PACKED ? kSrcP8 : SD, SX = PACKED ? kSrcP8 : SO;
  // One vector per thread: the next row is fetched ahead (16384 x 2560 bf16 with
  // post: 96 us, 128 without).  Two: the registers do not hold that; the row is
  // kept as loaded and widened a second time after the sums, and where they are
  // short of it still the weights are read again for every row (4096 x 10240, bf16
  // with an fp32 residual: 132 us; gamma 155; post 165, 170 with them kept).
  constexpr bool kAhead = K == 1, kRenew = K == 2;
  __shared__ float lds[LANES ? kPartialLds : kRowSumFloats];
  int half = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  const Place<LANES> at;
  const int cols = (int)a.p.cols;
  const float inv = 1.0f / (float)cols;
  int col[K], n[K];
  float w[K][8], m[K][8];  // m: scale gamma post
  float dw[K][8] = {}, s[K][8] = {};
  constexpr bool kReload = K == 2 && (EXTRA == 2 || (EXTRA == 1 && T == 1024));
  auto weights = [&](int k) {
    load_w<WHOLE>(a.p.weight, col[k], n[k], w[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) m[k][j] = a.p.scale;
    if (EXTRA != 0 && a.p.gamma != nullptr) {
      float g[8];
      load_w<WHOLE>(a.p.gamma, col[k], n[k], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) m[k][j] *= g[j];
    }
    if constexpr (EXTRA == 2) {
      float g[8];
      load_w<WHOLE>(a.p.post_weight, col[k], n[k], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) m[k][j] *= g[j];
    }
  };
#pragma unroll
  for (int k = 0; k < K; ++k) {
    col[k] = at.col(k);
    n[k] = cols - col[k];
    if constexpr (!kReload) weights(k);
  }
  const int64_t step = (int64_t)gridDim.x * at.nseg;
  int64_t row = (int64_t)blockIdx.x * at.nseg + at.seg;
  Raw<SO> nd[K];
  Raw<SD> ne[K];
  Raw<SR> nr[K];
  Raw<SX> nx[EXTRA ? K : 1];
  auto fetch = [&](int64_t i) {
    const char* dr = static_cast<const char*>(a.p.dout) + i * a.p.dout_stride * (IO32 ? 4 : 2);
    const char* er = static_cast<const char*>(a.p.dresidual_out) + i * a.p.dresidual_out_stride * (RES32 ? 4 : 2);
    const char* rr = static_cast<const char*>(a.p.r) + i * (PACKED ? a.pitch : a.p.r_stride * (RES32 ? 4 : 2));
    const uint8_t* rs = PACKED ? a.p.r_scale + i * (a.pitch >> 5) : nullptr;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      nd[k] = load_raw<SO, WHOLE>(dr, nullptr, col[k], n[k]);
      nr[k] = load_raw<SR, WHOLE>(rr, rs, col[k], n[k]);
      ne[k] = load_raw<SD, WHOLE>(er, nullptr, col[k], a.p.dresidual_out != nullptr ? n[k] : 0);
    }
    if constexpr (EXTRA != 0) {
      const char* xr = static_cast<const char*>(a.p.x) + i * (PACKED ? a.pitch : a.p.x_stride * (IO32 ? 4 : 2));
      const uint8_t* xs = PACKED ? a.p.x_scale + i * (a.pitch >> 5) : nullptr;
#pragma unroll
      for (int k = 0; k < K; ++k) nx[k] = load_raw<SX, WHOLE>(xr, xs, col[k], n[k]);
    }
  };
  if (kAhead && row < a.p.rows) fetch(row);
  for (; row < a.p.rows; row += step) {
    if constexpr (!kAhead) fetch(row);
    Raw<SO> rd[K];
    Raw<SD> re[K];
    Raw<SR> rr[K];
    Raw<SX> rx_[EXTRA ? K : 1];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      rd[k] = nd[k], re[k] = ne[k], rr[k] = nr[k];
      if constexpr (EXTRA != 0) rx_[k] = nx[k];
    }
    if (kAhead && row + step < a.p.rows) fetch(row + step);
    float d[K][8], e[K][8], r[K][8], x[K][8];
    auto widen_row = [&](int k) {
      widen<SO>(rd[k], d[k]), widen<SR>(rr[k], r[k]);
      if constexpr (EXTRA != 0) widen<SX>(rx_[k], x[k]);
    };
    float sum[EXTRA == 2 ? 3 : 2] = {};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      widen_row(k);
      if constexpr (kReload) load_w<WHOLE>(a.p.weight, col[k], n[k], w[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum[0] = __builtin_fmaf(r[k][j], r[k][j], sum[0]);
        sum[1] = __builtin_fmaf(d[k][j] * w[k][j], r[k][j], sum[1]);
        if constexpr (EXTRA == 2) sum[2] = __builtin_fmaf(x[k][j], x[k][j], sum[2]);
      }
      if constexpr (kRenew) {
        renew(rd[k]), renew(rr[k]);
        if constexpr (EXTRA != 0) renew(rx_[k]);
        __builtin_amdgcn_sched_barrier(0);  // one vector at a time
      }
    }
    row_sums<LANES>(sum, lds, half);
    const float rstd = rsqrtf(__builtin_fmaf(sum[0], inv, a.p.eps));
    const float c1 = sum[1] * inv * rstd * rstd * rstd;
    float rx = 0.f, sum2[1] = {};
    if constexpr (EXTRA == 2) rx = rsqrtf(__builtin_fmaf(sum[2], inv, a.p.eps));
    char* dres = static_cast<char*>(a.p.dresidual) + row * a.p.dresidual_stride * (RES32 ? 4 : 2);
    char* dx = static_cast<char*>(a.p.dx) + row * a.p.dx_stride * (IO32 ? 4 : 2);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if constexpr (kRenew) widen_row(k);
      if constexpr (kReload) {
        asm volatile("" ::: "memory");
        weights(k);
      }
      widen<SD>(re[k], e[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float rh = r[k][j] * rstd;
        dw[k][j] = __builtin_fmaf(d[k][j], rh, dw[k][j]);
        e[k][j] += rstd * (d[k][j] * w[k][j]) - r[k][j] * c1;  // dr
      }
      if (a.p.dresidual != nullptr && n[k] > 0) store8<RES32, WHOLE>(dres, col[k], n[k], e[k]);
      if constexpr (EXTRA == 0) {
        if (a.p.dx != nullptr && n[k] > 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) e[k][j] *= m[k][j];
          store8<IO32, WHOLE>(dx, col[k], n[k], e[k]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[k][j] = __builtin_fmaf(e[k][j], EXTRA == 2 ? x[k][j] * rx : x[k][j], s[k][j]);
          e[k][j] *= m[k][j];  // dx, or g2
          if constexpr (EXTRA == 2) sum2[0] = __builtin_fmaf(e[k][j], x[k][j], sum2[0]);
        }
        if (EXTRA == 1 && a.p.dx != nullptr && n[k] > 0) store8<IO32, WHOLE>(dx, col[k], n[k], e[k]);
      }
      if constexpr (kRenew) __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (EXTRA == 2) {
      if constexpr (kRenew) {
#pragma unroll
        for (int k = 0; k < K; ++k) renew(rx_[k]);
      }
      row_sums<LANES>(sum2, lds, half);
      const float c2 = sum2[0] * inv * rx * rx * rx;
      if (a.p.dx != nullptr) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if constexpr (kRenew) widen<SX>(rx_[k], x[k]);
#pragma unroll
          for (int j = 0; j < 8; ++j) e[k][j] = rx * e[k][j] - x[k][j] * c2;
          if (n[k] > 0) store8<IO32, WHOLE>(dx, col[k], n[k], e[k]);
        }
      }
    }
  }
  float* part = a.part + (int64_t)blockIdx.x * a.nout * cols;  // [dw][S]
#pragma unroll
  for (int k = 0; k < K; ++k) store_partial<LANES, WHOLE>(part, col[k], n[k], dw[k], lds);
  if constexpr (EXTRA != 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) store_partial<LANES, WHOLE>(part + cols, col[k], n[k], s[k], lds);
  }
}

template <bool RES32, bool IO32>
hipError_t fwd_typed(const AddNormFwdParams& p, hipStream_t stream) {
  const NormShape s = norm_shape(p.cols);
  const dim3 grid((unsigned)norm_blocks(s, p.rows, 1, false)), block((unsigned)s.threads);
  const FwdArgs a{p, (int)((p.cols + 31) / 32 * 32)};
  return with_shape(s, p.cols % 8 == 0, [&](auto lanes, auto k, auto t, auto whole) {
    if (p.post_weight != nullptr)
      hipLaunchKernelGGL((add_norm_fwd_kernel<RES32, IO32, true, lanes.value, k.value, t.value, whole.value>), grid, block, 0,
                         stream, a);
    else
      hipLaunchKernelGGL((add_norm_fwd_kernel<RES32, IO32, false, lanes.value, k.value, t.value, whole.value>), grid, block, 0,
                         stream, a);
    return hipGetLastError();
  });
}

template <bool RES32, bool IO32, bool PACKED, int EXTRA>
hipError_t bwd_typed(const AddNormBwdParams& p, hipStream_t stream) {
  const NormShape s = norm_shape(p.cols);
  const int64_t blocks = norm_blocks(s, p.rows, 1, true);
  BwdArgs a{p, reinterpret_cast<float*>(static_cast<char*>(p.workspace) + 256), 1, (int)((p.cols + 31) / 32 * 32),
            static_cast<int*>(p.workspace)};
  a.nout = EXTRA != 0 ? 2 : 1;
  const SumPartialsArgs sum{a.part,  p.dweight, p.dgamma, p.dpost_weight, p.post_weight,
                            p.gamma, p.scale,   blocks,   p.cols,         a.nout};
  const hipError_t e = with_shape(s, p.cols % 8 == 0, [&](auto lanes, auto k, auto t, auto whole) {
    hipLaunchKernelGGL((add_norm_bwd_kernel<RES32, IO32, PACKED, EXTRA, lanes.value, k.value, t.value, whole.value>),
                       dim3((unsigned)blocks), dim3((unsigned)s.threads), 0, stream, a);
    return hipGetLastError();
  });
  return e != hipSuccess ? e : launch_sum_partials(sum, stream);
}

template <bool RES32, bool IO32>
hipError_t bwd_extra(const AddNormBwdParams& p, hipStream_t stream) {
  const bool packed = p.r_scale != nullptr;
  if (p.post_weight != nullptr)
    return packed ? bwd_typed<RES32, IO32, true, 2>(p, stream) : bwd_typed<RES32, IO32, false, 2>(p, stream);
  if (p.gamma != nullptr)
    return packed ? bwd_typed<RES32, IO32, true, 1>(p, stream) : bwd_typed<RES32, IO32, false, 1>(p, stream);
  return packed ? bwd_typed<RES32, IO32, true, 0>(p, stream) : bwd_typed<RES32, IO32, false, 0>(p, stream);
}

}  // namespace

hipError_t launch_add_norm_fwd(const AddNormFwdParams& p, hipStream_t stream) {
  if (!p.io_bf16) return fwd_typed<true, true>(p, stream);
  return p.res_bf16 ? fwd_typed<false, false>(p, stream) : fwd_typed<true, false>(p, stream);
}

size_t add_norm_bwd_workspace_bytes(int64_t rows, int64_t cols, int ngrads) {
  const size_t sums = ngrads > 1 ? 2 : 1;  // dgamma and dpost_weight are one sum
  return 256 + (size_t)norm_blocks(norm_shape(cols), rows, 1, true) * sums * (size_t)cols * sizeof(float);
}

hipError_t launch_add_norm_bwd(const AddNormBwdParams& p, hipStream_t stream) {
  if (!p.io_bf16) return bwd_extra<true, true>(p, stream);
  return p.res_bf16 ? bwd_extra<false, false>(p, stream) : bwd_extra<true, false>(p, stream);
}

}  // namespace mss
