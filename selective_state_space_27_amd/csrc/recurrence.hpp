// Arithmetic of the gated linear recurrence (gfx950), shared by its scan, its
// gradient and its one-token step.  Per channel and step:
//   r = sigmoid(gate_a), i = sigmoid(gate_x), s = k r with k = c softplus(lam),
//   a = exp(-s), beta = sqrt(1 - a^2), h <- a h + beta i x.
// The decay is kept as m = 1 - a = -expm1(-s): decays are near 1 (s is a few
// hundredths), where a itself would hold only the leading digits of m, and m
// gives both h - m h and beta^2 = m (2 - m) without cancellation.
#pragma once

#include "common.hpp"

namespace mss {

// Of s, for the polynomials of one_minus_exp.
constexpr float kPolySmall = 0.25f, kPolyMax = 0.5f;

// E = exp(-v).  EXACT (fp32 tensors): with what the rounding of the argument
// leaves out, which is |v| units otherwise (bf16's own rounding of v is 2^15
// times that).  Infinities and NaN come out as they should: past +-192 the
// limits hold, and a limit keeps infinities out of the rest term.
template <bool EXACT>
__device__ __forceinline__ float exp_neg(float v) {
  const float t = -v * kLog2e;
  const float e = exp2_fast(t);
  if constexpr (EXACT) {
    constexpr float kLog2eRest = (float)(1.4426950408889634 - (double)kLog2e), kLn2 = 0.69314718f;
    const float lo = __builtin_fmaf(-v, kLog2eRest, __builtin_fmaf(-v, kLog2e, -t));
    return __builtin_fabsf(t) < 256.f ? e * __builtin_fmaf(lo, kLn2, 1.0f) : e;
  } else {
    return e;
  }
}

// sigmoid(v), and with E also 1 - sigmoid(v) without cancellation.
template <bool EXACT>
__device__ __forceinline__ float sigmoid_of(float v) {
  return rcp_fast(1.0f + exp_neg<EXACT>(v));
}
template <bool EXACT>
__device__ __forceinline__ float sigmoid_of(float v, float& rest) {
  const float e = exp_neg<EXACT>(v), s = rcp_fast(1.0f + e);
  rest = e < __builtin_inff() ? e * s : 1.0f;
  return s;
}

// 1 - exp(-s) for s >= 0: s times a polynomial fitted to (1 - exp(-s)) / s at
// Chebyshev points (off by 2.4e-9 of 1 up to 1/4, where decays of a trained layer
// lie; by 1.2e-9 up to 1/2), beyond 1/2 the plain difference, which would lose
// digits below.  SMALL: no s is above kPolySmall.
template <bool SMALL>
__device__ __forceinline__ float one_minus_exp(float s) {
  if constexpr (SMALL) {
    float p = __builtin_fmaf(s, 0.007514301221817732f, -0.04149100184440613f);
    p = __builtin_fmaf(s, p, 0.16665112972259521f);
    p = __builtin_fmaf(s, p, -0.4999995231628418f);
    return __builtin_fmaf(s, p, 1.0f) * s;
  } else {
    float p = __builtin_fmaf(s, -0.0011237150756642222f, 0.008190003223717213f);
    p = __builtin_fmaf(s, p, -0.04163024201989174f);
    p = __builtin_fmaf(s, p, 0.16666245460510254f);
    p = __builtin_fmaf(s, p, -0.4999998211860657f);
    p = __builtin_fmaf(s, p, 1.0f) * s;
    return s > kPolyMax ? 1.0f - exp2_fast(-s * kLog2e) : p;
  }
}

// softplus(lam) = max(lam, 0) + log(1 + e), e = exp(-|lam|), to a few units over
// the whole range: log(1 + e) = 2 atanh(z), z = e / (2 + e) <= 1/3, by its series
// (the first term left out is 1.4e-8 of the sum).
__device__ __forceinline__ float softplus_of(float lam) {
  const float e = exp_neg<true>(__builtin_fabsf(lam)), z = e * rcp_fast(2.0f + e), q = z * z;
  float p = __builtin_fmaf(q, 1.0f / 13.0f, 1.0f / 11.0f);
  p = __builtin_fmaf(q, p, 1.0f / 9.0f);
  p = __builtin_fmaf(q, p, 1.0f / 7.0f);
  p = __builtin_fmaf(q, p, 1.0f / 5.0f);
  p = __builtin_fmaf(q, p, 1.0f / 3.0f);
  p = __builtin_fmaf(q, p, 1.0f);
  return __builtin_fmaf(2.0f * z, p, lam > 0.0f ? lam : 0.0f);
}
// d log softplus / d lam = sigmoid(lam) / softplus(lam), whose limit is 1.
__device__ __forceinline__ float softplus_rate(float lam, float sp) {
  return lam < -80.f ? 1.0f : sigmoid_of<true>(lam) / sp;
}

// s where only s a (and s alone nowhere) is wanted: exp(-200) is 0 in fp32, and
// a finite s keeps s a at 0.  (A NaN stays one.)
__device__ __forceinline__ float finite_decay(float s) { return s > 200.f ? 200.f : s; }

}  // namespace mss
