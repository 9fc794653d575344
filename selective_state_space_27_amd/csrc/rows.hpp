// Rows of activations as the norm and checkpoint kernels read and write them
// (gfx950): eight consecutive columns per thread, widened to fp32, from bf16,
// fp32 or the 8-bit checkpoint form; sums over the lanes of a row; the 8-bit
// form's rounding.
//
// The 8-bit form of a [rows, cols] tensor: per row and block of 32 columns a
// scale s = 2^(e - 127), the smallest power of two with max|x| / s < 127.5 - 2^-17,
// and q = rint(x / s) in int8 (two's complement).  The bound is 127.5's lower
// neighbour in fp32, where max|x| * (1 / 127.5) reaches 1: an fp32 evaluation by the
// reciprocal, as a division by a constant commonly is on a GPU, finds the same
// scales.  (A correctly rounded division takes the smaller one at that one mantissa;
// no bf16 value lies there.)  Rows of q are padded with zeros to a
// multiple of 32 columns (the pitch), scales are the bytes e, one per 32
// columns.  1 <= e <= 248: a block of zeros or of values below 2^-120 has e = 1,
// and the top of the range (where q s would overflow) saturates at 127 * 2^121.
// |x - q s| <= s / 2, but for what saturates: below s.  A block with an infinity or NaN in it has e = 255
// and q = 0: its values read back as 0 * inf = NaN.  A power of two costs at
// most one bit against a free scale, and buys that q s is exact in bf16 (seven
// bits of magnitude), so the form feeds bf16 matrix products without a
// rounding, that x / s and q s are exact in fp32, and that s takes one byte.
#pragma once

#include "common.hpp"

namespace mss {

// Where a row's values come from.
enum : int { kSrcBf16 = 0, kSrcF32 = 1, kSrcP8 = 2 };

// Rows at any element alignment: the hardware takes 16-byte accesses at any
// address, the type only tells the compiler not to assume 16-byte alignment.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight columns of a row as loaded: 16 bytes of bf16, 32 of fp32, or 8 of q
// and the scale's exponent byte.
template <int SRC>
struct Raw {
  u32x4 a;
};
template <>
struct Raw<kSrcF32> {
  u32x4 a, b;
};
template <>
struct Raw<kSrcP8> {
  u32x2 a;
  uint32_t e;
};

// Columns col .. col + 7 of a row; `n` of them exist (n <= 0: none, zeros).
// For the 8-bit form, whose rows are padded, `row` is the row of q and `srow`
// its scales.  WHOLE: the rows are whole vectors (n >= 8 or n <= 0), which
// leaves the column by column path out of the code.
template <int SRC, bool WHOLE = false>
__device__ __forceinline__ Raw<SRC> load_raw(const void* row, const uint8_t* srow, int col, int n) {
  Raw<SRC> r{};
  if constexpr (SRC == kSrcP8) {
    if (n > 0) {
      r.a = *reinterpret_cast<const u32x2*>(static_cast<const int8_t*>(row) + col);
      r.e = srow[col >> 5];  // shifted into place when used: nothing here waits for it
    }
  } else if constexpr (SRC == kSrcF32) {
    const float* p = static_cast<const float*>(row) + col;
    if (WHOLE ? n > 0 : n >= 8) {
      r.a = *reinterpret_cast<const u32x4_a4*>(p);
      r.b = *reinterpret_cast<const u32x4_a4*>(p + 4);
    } else if (!WHOLE && n > 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r.a[j] = j < n ? __float_as_uint(p[j]) : 0u;
        r.b[j] = j + 4 < n ? __float_as_uint(p[j + 4]) : 0u;
      }
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(row) + col;
    if (WHOLE ? n > 0 : n >= 8) {
      r.a = *reinterpret_cast<const u32x4_a2*>(p);
    } else if (!WHOLE && n > 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = 2 * j < n ? p[2 * j] : 0u, hi = 2 * j + 1 < n ? p[2 * j + 1] : 0u;
        r.a[j] = lo | hi << 16;
      }
    }
  }
  return r;
}

// Makes the compiler take the values as new: what was widened from them before
// is not kept, but widened again.
template <int SRC>
__device__ __forceinline__ void renew(Raw<SRC>& r) {
#pragma unroll
  for (int j = 0; j < (SRC == kSrcP8 ? 2 : 4); ++j) {
    uint32_t w = r.a[j];
    asm volatile("" : "+v"(w));
    r.a[j] = w;
  }
  if constexpr (SRC == kSrcF32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w = r.b[j];
      asm volatile("" : "+v"(w));
      r.b[j] = w;
    }
  }
}

template <int SRC>
__device__ __forceinline__ void widen(const Raw<SRC>& r, float (&v)[8]) {
  if constexpr (SRC == kSrcP8) {
    const float s = __uint_as_float(r.e << 23);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)((int32_t)(r.a[j >> 2] << (24 - 8 * (j & 3))) >> 24) * s;
  } else if constexpr (SRC == kSrcF32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(r.a[j]), v[j + 4] = __uint_as_float(r.b[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(r.a[j]), v[2 * j + 1] = bf16_hi(r.a[j]);
  }
}

// The first n (> 0) of eight values at column col of a row.
template <bool F32, bool WHOLE = false>
__device__ __forceinline__ void store8(void* row, int col, int n, const float (&v)[8]) {
  if constexpr (F32) {
    float* p = static_cast<float*>(row) + col;
    if (WHOLE || n >= 8) {
      *reinterpret_cast<u32x4_a4*>(p) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                              __float_as_uint(v[3])};
      *reinterpret_cast<u32x4_a4*>(p + 4) = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                                                  __float_as_uint(v[7])};
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < n) p[j] = v[j];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(row) + col;
    if (WHOLE || n >= 8) {
      *reinterpret_cast<u32x4_a2*>(p) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < n) p[j] = f32_to_bf16(v[j]);
    }
  }
}

// Values as they are after a store in the given type.
template <bool F32>
__device__ __forceinline__ void as_stored(float (&v)[8]) {
  if constexpr (!F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = bf16_to_f32(f32_to_bf16(v[j]));
  }
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v)));
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

// Eight values (fp32) of four neighbouring lanes are one block of 32: their
// common exponent byte, and this lane's eight q.  The columns past a row's end
// hold zeros.  The maximum is taken on the bits without sign, where infinities
// and NaN are above every finite value and so are not lost.
__device__ __forceinline__ u32x2 quantise8(const float (&v)[8], uint32_t& e) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
  m = max(m, dpp_u32<kDppXor1>(m));
  m = max(m, dpp_u32<kDppXor2>(m));
  // max / 2^(exponent) is in [1, 2): from 127.5/64 less one unit the next power is taken.
  const int up = (m & 0x7fffffu) >= 0x7effffu ? 1 : 0;
  const int b = min(max((int)(m >> 23) - 6 + up, 1), 248);
  const bool finite = m < 0x7f800000u;
  e = finite ? (uint32_t)b : 255u;
  const float s = __uint_as_float((uint32_t)b << 23), inv = __uint_as_float((uint32_t)(254 - b) << 23);
  const float lim = 127.f * s;
  uint32_t w[8];
  // v / s + 1.5 * 2^23 in one rounding to an integer (nearest, ties to even):
  // its low byte is q.  The clamp only acts at the top of the range.
#pragma unroll
  for (int j = 0; j < 8; ++j)
    w[j] = __float_as_uint(__builtin_fmaf(__builtin_amdgcn_fmed3f(v[j], -lim, lim), inv, 12582912.f));
  u32x2 q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // Low bytes of four words.  v_perm: selectors 0-3 take the second operand's bytes, 4-7 the first's.
    const uint32_t lo = __builtin_amdgcn_perm(w[4 * h + 1], w[4 * h], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(w[4 * h + 3], w[4 * h + 2], 0x0c0c0400u);
    q[h] = finite ? lo | hi << 16 : 0u;
  }
  return q;
}

// Writes the 8-bit form of eight values at column col of a row (col below the
// pitch); the four lanes of a block call it together.
__device__ __forceinline__ void store_p8(int8_t* qrow, uint8_t* srow, int col, int pitch, const float (&v)[8]) {
  uint32_t e;
  const u32x2 q = quantise8(v, e);
  if (col < pitch) {
    *reinterpret_cast<u32x2*>(qrow + col) = q;
    if ((threadIdx.x & 3) == 0) srow[col >> 5] = (uint8_t)e;
  }
}

// Sum over the LANES (16, 32 or 64) neighbouring lanes that hold a row, in a
// fixed order; every one of them gets it.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  v += dpp_f32<kDppXor1>(v);
  v += dpp_f32<kDppXor2>(v);
  v += dpp_f32<kDppHalfMirror>(v);
  v += dpp_f32<kDppMirror>(v);
  // The swaps put each pair's values side by side: of 16 lanes, of 32.
  if constexpr (LANES >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (LANES == 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Sums over the lanes of a row, for rows held by LANES lanes of a wave
// (LANES = 16, 32, 64) or by the whole workgroup (LANES = 0, at most 16 waves;
// every thread calls it the same number of times).  For the workgroup, wave
// sums meet in `lds` (kRowSumFloats floats): two halves used in turn, so one
// barrier a call suffices: a half is written again only after the next call's
// barrier, which every thread reaches after it has read.
constexpr int kRowSumMax = 3;
constexpr int kRowSumFloats = 2 * kRowSumMax * 16;
template <int LANES, int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float* lds, int& half) {
  static_assert(NV <= kRowSumMax, "");
  if constexpr (LANES != 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = lanes_sum<LANES>(v[i]);
  } else {
    // Lane i writes its wave's sum i; then 16 lanes take one sum's wave values each.
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
    float* p = lds + half * (kRowSumMax * 16);
    half ^= 1;
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = lanes_sum<64>(v[i]);
      mine = lane == i ? v[i] : mine;
    }
    if (lane < NV) p[lane * 16 + wave] = mine;
    __syncthreads();
    const float t = lanes_sum<16>((lane & 15) < nw && lane < NV * 16 ? p[lane] : 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      v[i] = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(t), 16 * i));
  }
}

}  // namespace mss
