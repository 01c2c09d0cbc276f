// Device helpers of the int8 kernels for gfx950.
#pragma once

#include "i8_internal.hpp"
#include "mx_device.hpp"

namespace aqlm {

typedef int int4_vt __attribute__((ext_vector_type(4)));
typedef int int16_vt __attribute__((ext_vector_type(16)));

// Pins a value in a register at this place of the code.
__device__ __forceinline__ int held(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// v_mfma_i32_16x16x64_i8 / 32x32x32_i8: lane (r, q) gives the 16 bytes q of row r
// of each side (q = lane / 16 or lane / 32).
__device__ __forceinline__ int4_vt i8_mfma16(const uint4 &a, const uint4 &b, int4_vt c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(int4_vt, a), __builtin_bit_cast(int4_vt, b), c, 0,
                                               0, 0);
}
__device__ __forceinline__ int16_vt i8_mfma32(const uint4 &a, const uint4 &b, int16_vt c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(int4_vt, a), __builtin_bit_cast(int4_vt, b), c, 0,
                                               0, 0);
}

// Element e of an octet as float32 (exact).
template <MxType T> __device__ __forceinline__ float octet_value(const Octet<T> &o, int e) {
  if constexpr (T == MxType::kF32) return __builtin_bit_cast(float, o.w[e]);
  const uint32_t w = o.w[e >> 1];
  if constexpr (T == MxType::kF16) return h2f(e & 1 ? w >> 16 : w & 0xFFFFu);
  return __builtin_bit_cast(float, e & 1 ? w & 0xFFFF0000u : w << 16);
}

// Largest magnitude of an octet: its float32 bits without the sign, which order
// like the magnitudes, NaN above infinity above the numbers.
template <MxType T> __device__ __forceinline__ uint32_t octet_max(const Octet<T> &o) {
  uint32_t m = 0;
  if constexpr (T == MxType::kF32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, o.w[e] & 0x7FFFFFFFu);
    return m;
  }
  u16x2_t p = {0, 0};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    p = __builtin_elementwise_max(p, __builtin_bit_cast(u16x2_t, o.w[e] & 0x7FFF7FFFu));
  return max((uint32_t)p.x, (uint32_t)p.y);
}
// octet_max's value as float32 bits.
template <MxType T> __device__ __forceinline__ uint32_t max_bits(uint32_t m) {
  if constexpr (T == MxType::kF16) return __builtin_bit_cast(uint32_t, h2f(m));
  if constexpr (T == MxType::kBF16) return m << 16;
  return m;
}

// Maximum over each 16 lanes, in every one of them.
__device__ __forceinline__ uint32_t row16_max(uint32_t m) {
  auto step = [&](auto ctrl) __attribute__((always_inline)) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, decltype(ctrl)::value, 0xF, 0xF, false));
  };
  step(std::integral_constant<int, kDppQuadXor1>{});
  step(std::integral_constant<int, kDppQuadXor2>{});
  step(std::integral_constant<int, kDppRowHalfMirror>{});
  step(std::integral_constant<int, kDppRowMirror>{});
  return m;
}

// Maximum over the 64 lanes of a wavefront, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  const int m = (int)row16_max(v);
  const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane(m, 0), (uint32_t)__builtin_amdgcn_readlane(m, 16));
  const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane(m, 32), (uint32_t)__builtin_amdgcn_readlane(m, 48));
  return max(a, b);
}

// What a row is quantised with. Rows whose largest magnitude A is below 2^-100 or
// from 2^100 on are taken times 2^100 or 2^-100 first (exact for all that does not
// round to 0), since 127 / A or 127 A would overflow.
struct RowScale {
  float scale;  // A / 127: what a code stands for; NaN for a row that has no number for it
  float top;    // A, times `lift`
  float inv;    // 127 / top, 0 for rows whose codes are zeros
  float lift;   // 1, 2^100 or 2^-100
};
__device__ __forceinline__ RowScale row_scale(uint32_t bits) {
  RowScale r = {0.f, 0.f, 0.f, 1.f};
  if (bits >= 0x7F800000u) {
    r.scale = __builtin_bit_cast(float, 0x7FC00000u);
  } else if (bits != 0u) {
    const float a = __builtin_bit_cast(float, bits);
    r.scale = a / 127.f;
    r.lift = a < 0x1p-100f ? 0x1p100f : a >= 0x1p100f ? 0x1p-100f : 1.f;
    r.top = a * r.lift;
    r.inv = 127.f / r.top;
  }
  return r;
}

// The code of v, exactly round-to-even of 127 v / A. t = v inv is within 2^-16 of
// that (two roundings of 2^-24 each, at most 127), so where it lies further
// than 2^-14 from the middle of two whole numbers the nearer one is right. Near the
// middle m + 1/2 the products 127 v and (m + 1/2) A decide, which float32 holds
// exactly for halves (18 and 19 significant bits) and float64 for float32 (31 and 32).
template <MxType T> __device__ __forceinline__ int code_near_tie(float v, const RowScale &r) {
  typedef std::conditional_t<T == MxType::kF32, double, float> Wide;
  const float low = __builtin_rintf((v * r.lift) * r.inv - 0.5f);
  const Wide x = (Wide)127 * (Wide)(v * r.lift), middle = ((Wide)low + (Wide)0.5) * (Wide)r.top;
  const int n = (int)low;
  return x > middle ? n + 1 : x < middle ? n : n + (n & 1);
}

// Eight codes of an octet, a byte each.
template <MxType T> __device__ __forceinline__ uint2 encode_octet(const Octet<T> &o, const RowScale &r) {
  uint32_t b[8];
  float worst = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float v = r.inv == 0.f ? 0.f : octet_value<T>(o, e) * r.lift;
    // in [2^23, 2^24) the whole numbers are the float32 values: the sum is rounded to
    // even there, and its low byte is the code's
    const float m = __builtin_fmaf(v, r.inv, 0x1.8p23f);
    worst = __builtin_fmaxf(worst, __builtin_fabsf(__builtin_fmaf(v, r.inv, -(m - 0x1.8p23f))));
    b[e] = __builtin_bit_cast(uint32_t, m);
  }
  if (worst > 0.5f - 0x1p-14f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = (uint32_t)code_near_tie<T>(octet_value<T>(o, e), r);
  }
  auto four = [&](int k) {
    const uint32_t lo = __builtin_amdgcn_perm(b[k + 1], b[k], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[k + 3], b[k + 2], 0x04000C0Cu);
    return lo | hi;
  };
  return make_uint2(four(0), four(4));
}

// act(g) and its derivative. e^x is v_exp_f32 of x log2 e: the rounding of that
// product makes a relative error of |x| 2^-24, far below a half's step wherever the
// result is not.
__device__ __forceinline__ float i8_sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// e^(t^2) erfc(t) for t of [0, 10.3], beyond which the e^(-t^2) that it is multiplied by
// is 0 in float32 (the fit goes on to be off by 2^-14 at most). y P(y) with y = 1 / (1 + t
// / 2), P of degree 8 fitted to the quotient at 400 Chebyshev points of y by least
// squares, weighted anew until the largest relative errors were alike. With these
// coefficients it is within 1.5 * 2^-24 of itself, with float32's operations and a
// reciprocal that is off by a unit within 9 * 2^-24. Keeps its precision where 1 + erf has
// none, in a fifth of the instructions of erfcf.
__device__ __forceinline__ float scaled_erfc(float t) {
  const float y = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, t, 1.f));
  float p = -0.059386909f;
  p = __builtin_fmaf(p, y, 0.286126167f);
  p = __builtin_fmaf(p, y, -0.490410924f);
  p = __builtin_fmaf(p, y, 0.28173852f);
  p = __builtin_fmaf(p, y, -0.0291521549f);
  p = __builtin_fmaf(p, y, 0.203754067f);
  p = __builtin_fmaf(p, y, 0.242834732f);
  p = __builtin_fmaf(p, y, 0.282412142f);
  return __builtin_fmaf(p, y, 0.282084316f) * y;
}

__device__ __forceinline__ void act_and_slope(I8Act act, float g, float &a, float &slope) {
  if (act == I8Act::kSilu) {
    const float s = i8_sigmoid(g);
    a = g * s;
    slope = s * (1.f + g * (1.f - s));
  } else if (act == I8Act::kGelu) {  // Phi(g) = erfc(-g / sqrt 2) / 2
    const float e = __expf(-0.5f * g * g);
    const float tail = 0.5f * e * scaled_erfc(0.70710678f * __builtin_fabsf(g));
    const float phi = g < 0.f ? tail : 1.f - tail;
    a = g * phi;
    slope = phi + g * (0.39894228f * e);
  } else {
    const float k = 1.59576912f, c = 0.044715f;  // 2 sqrt(2 / pi)
    const float s = i8_sigmoid(k * (g + c * g * g * g));
    a = g * s;
    // (where g^2 passes 2^40, s (1 - s) is 0 and the polynomial may not be infinite)
    slope = s + g * s * (1.f - s) * (k * (1.f + 3.f * c * __builtin_fminf(g * g, 0x1p40f)));
  }
}

__device__ __forceinline__ float act_value(I8Act act, float g) {
  float a, slope;
  act_and_slope(act, g, a, slope);
  return a;
}

// A sum of codes as the product's value: the channel's scale first, so that a
// token's very small or large one meets a number near the result. (Materialised: a
// rounding to float16 that follows is one of its own in every kernel.)
__device__ __forceinline__ float i8_value(int sum, float channel, float token) {
  return materialize(materialize((float)sum * channel) * token);
}

}  // namespace aqlm
