// Arithmetic of the gated linear recurrence (gfx950), shared by its scan, its
// gradient and its one-token step.  Per channel and step:
//   r = sigmoid(gate_a), i = sigmoid(gate_x), s = k r with k = c softplus(lam),
//   a = exp(-s), beta = sqrt(1 - a^2), h <- a h + beta i x.
// The decay is kept as one number m, whose sign tells which:
//   n = a - 1 = expm1(-s), -1/2 < n <= -0, while s <= 1/2: most decays are near 1 (s is a
//     few hundredths), where a itself would hold only the leading digits of n, and n
//     gives both h + n h and beta^2 = -n (2 + n) without cancellation;
//   a itself, 0 <= a < 0.61, beyond: 1 + n would lose the digits of a small a, and with
//     them those of all that is a product with it (dgate_a, dh0, a state's last traces).
#pragma once

#include "common.hpp"

namespace mss {

// Of s, for the polynomials of decay_of.
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

// sigmoid(v).
template <bool EXACT>
__device__ __forceinline__ float sigmoid_of(float v) {
  return rcp_fast(1.0f + exp_neg<EXACT>(v));
}
// From E = exp(-v), also 1 - sigmoid(v) = E sigmoid(v), without cancellation.  Where
// E is infinite the sigmoid is 0, and so is what its rest is multiplied by; the
// limits, an output modifier of the product, make 0 of infinity times 0.
__device__ __forceinline__ float sigmoid_from(float e, float& rest) {
  const float s = rcp_fast(1.0f + e);
  rest = __builtin_amdgcn_fmed3f(e * s, 0.0f, 1.0f);
  return s;
}

// m for s >= 0.  n is s times a polynomial fitted to (exp(-s) - 1) / s at Chebyshev
// points (with its fp32 coefficients off by 4.8e-9 of itself up to 1/4, where decays of
// a trained layer lie; by 4.5e-9 up to 1/2: a twelfth of a unit); a comes with the
// rounding of its argument put back where the gates' are (EXACT).  SMALL: no s is above
// kPolySmall, so m is n.
template <bool SMALL, bool EXACT>
__device__ __forceinline__ float decay_of(float s) {
  if constexpr (SMALL) {
    float p = __builtin_fmaf(s, -0.007514301221817732f, 0.04149100184440613f);
    p = __builtin_fmaf(s, p, -0.16665112972259521f);
    p = __builtin_fmaf(s, p, 0.4999995231628418f);
    return __builtin_fmaf(s, p, -1.0f) * s;
  } else {
    float p = __builtin_fmaf(s, 0.0011237150756642222f, -0.008190003223717213f);
    p = __builtin_fmaf(s, p, 0.04163024201989174f);
    p = __builtin_fmaf(s, p, -0.16666245460510254f);
    p = __builtin_fmaf(s, p, 0.4999998211860657f);
    p = __builtin_fmaf(s, p, -1.0f) * s;
    return s > kPolyMax ? exp_neg<EXACT>(s) : p;
  }
}
// Whether m is n.
template <bool SMALL>
__device__ __forceinline__ bool is_rest(float m) {
  return SMALL || (int32_t)__float_as_uint(m) < 0;
}
// n, to a few units of it either way.
template <bool SMALL>
__device__ __forceinline__ float rest_of(float m) {
  return is_rest<SMALL>(m) ? m : m - 1.0f;
}
// a, of which 1 + n keeps all digits while n > -1/2.
template <bool SMALL>
__device__ __forceinline__ float factor_of(float m) {
  return is_rest<SMALL>(m) ? 1.0f + m : m;
}
// a v, of a state, a gradient or a product of decays.
template <bool SMALL>
__device__ __forceinline__ float decayed(float m, float v) {
  return __builtin_fmaf(m, v, is_rest<SMALL>(m) ? v : 0.0f);
}
// beta = sqrt(1 - a^2).
__device__ __forceinline__ float beta_of(float n) { return __builtin_amdgcn_sqrtf(-n * (2.0f + n)); }

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

// k = c softplus(lam), so that s = k r; finite, for s a has to come out as 0 where a is.
// (A NaN stays one.)
__device__ __forceinline__ float decay_rate(float c, float lam) {
  const float k = c * softplus_of(lam);
  return k > 1e30f ? 1e30f : k;
}

}  // namespace mss
