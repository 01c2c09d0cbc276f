// Device helpers of the microscaled (MXFP4) kernels for gfx950.
#pragma once

#include <type_traits>

#include "aqlm_device.hpp"
#include "mx_internal.hpp"

namespace aqlm {

typedef __bf16 bhalf2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bhalf8_t __attribute__((ext_vector_type(8)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef int int8_vt __attribute__((ext_vector_type(8)));

// Offset past every buffer resource made here: the load returns zero.
constexpr uint32_t kMxOOB = 0x80000000u;

// The E8M0 byte s as a float32 operand of the conversion instructions, which
// read its exponent field alone: s = 0 (bits of 0.0f) is taken as 2^-127, s =
// 255 (bits of infinity) as NaN.
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return __builtin_bit_cast(float, s << 23);
}

__device__ __forceinline__ uint32_t buf_load_u8(Rsrc r, uint32_t off) {
  return (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0);
}

// Eight E2M1 codes (one word, lowest nibble first) times a scale, as eight
// halves; one rounding where the type needs one.
template <MxType T> __device__ __forceinline__ uint4 mx_decode8(uint32_t w, float s) {
  uint4 r;
  if constexpr (T == MxType::kF16) {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3));
  } else {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  }
  return r;
}

// Eight consecutive elements, as loaded.
template <MxType T> struct Octet {
  uint32_t w[T == MxType::kF32 ? 8 : 4];
};

// NT: without a place in the caches.
template <MxType T, bool NT> __device__ __forceinline__ Octet<T> load_octet(const void *x, int64_t i) {
  Octet<T> o;
  const u32x4_t *p = static_cast<const u32x4_t *>(x) + i * (T == MxType::kF32 ? 2 : 1);
#pragma unroll
  for (int k = 0; k < (T == MxType::kF32 ? 2 : 1); ++k) {
    const u32x4_t v = NT ? __builtin_nontemporal_load(p + k) : p[k];
#pragma unroll
    for (int e = 0; e < 4; ++e) o.w[4 * k + e] = v[e];
  }
  return o;
}

// Largest magnitude of a block as float32 bits, from the octets of its four
// lanes. Magnitudes order like their bits read as integers, with NaN above
// infinity above the numbers, so the maximum is taken on integers.
template <MxType T> __device__ __forceinline__ uint32_t block_max(const Octet<T> &o) {
  uint32_t m = 0;
  if constexpr (T == MxType::kF32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, o.w[e] & 0x7FFFFFFFu);
  } else {
    u16x2_t p = {0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      p = __builtin_elementwise_max(p, __builtin_bit_cast(u16x2_t, o.w[e] & 0x7FFF7FFFu));
    m = max((uint32_t)p.x, (uint32_t)p.y);
  }
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppQuadXor1, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppQuadXor2, 0xF, 0xF, false));
  if constexpr (T == MxType::kF16) return __builtin_bit_cast(uint32_t, h2f(m));  // exact
  if constexpr (T == MxType::kBF16) return m << 16;
  return m;
}

// E8M0 byte of a block from its largest magnitude m * 2^e (float32 bits). With
// 1 <= m < 2, m * 2^e / 2^(e-2) = 4 m: at most 6 up to m = 1.5 (mantissa bits
// 0x400000), which is where the ceil rule takes the next power. Exponent
// fields below 3 (subnormals among them) give scales under 2^-127, held as
// 2^-127.
template <bool CEIL> __device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
  if (bits >= 0x7F800000u) return 255u;
  if (bits == 0u) return 127u;
  int b = (int)(bits >> 23) - 2;
  if (CEIL) b += (bits & 0x7FFFFFu) > 0x400000u;
  return (uint32_t)max(b, 0);
}

// Eight codes of an octet: v_cvt_scalef32_pk_fp4 divides by the scale, rounds
// to nearest even and saturates at 6.
template <MxType T> __device__ __forceinline__ uint32_t encode8(const Octet<T> &o, float s) {
  uint32_t r = 0;
  if constexpr (T == MxType::kF16) {
#define AQLM_ENC(i) \
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(half2_t, o.w[i]), s, i);
    AQLM_ENC(0) AQLM_ENC(1) AQLM_ENC(2) AQLM_ENC(3)
#undef AQLM_ENC
  } else if constexpr (T == MxType::kBF16) {
#define AQLM_ENC(i) \
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bhalf2_t, o.w[i]), s, i);
    AQLM_ENC(0) AQLM_ENC(1) AQLM_ENC(2) AQLM_ENC(3)
#undef AQLM_ENC
  } else {
#define AQLM_ENC(i)                                                                              \
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __builtin_bit_cast(float, o.w[2 * i]),         \
                                               __builtin_bit_cast(float, o.w[2 * i + 1]), s, i);
    AQLM_ENC(0) AQLM_ENC(1) AQLM_ENC(2) AQLM_ENC(3)
#undef AQLM_ENC
  }
  return r;
}

// Whether float16 holds every weight of a block with scale byte s exactly:
// 0.5 * 2^(s-127) >= 2^-24 and 6 * 2^(s-127) <= 65504 (NaN needs no care).
__device__ __forceinline__ bool mx_fits_f16(uint32_t s) { return (s - 104u <= 36u) | (s == 255u); }

// The same of 16 scale bytes at once: none of them is more than 36 above 104
// (modulo 2^16) if both halves here are 36 or less. (NaN counts as unfit; either
// way gives NaN.)
__device__ __forceinline__ u16x2_t mx_above_f16(const uint4 &s) {
  const uint32_t w[4] = {s.x, s.y, s.z, s.w};
  u16x2_t m = {0, 0};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const u16x2_t low = {104, 104};
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[u] & 0x00FF00FFu) - low);
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, (w[u] >> 8) & 0x00FF00FFu) - low);
  }
  return m;
}

// Eight float16 activations as the exact sum hi + lo of two bfloat16 vectors
// (11 significant bits: hi takes the first 8, what is left has 3 or fewer and a
// magnitude bfloat16 holds). hi is cut off, not rounded, so that lo has its sign and
// a product with hi overflows only where the whole does, to the same infinity.
// Infinities and NaN stay in hi alone.
__device__ __forceinline__ void split_f16(const uint4 &x, uint4 &hi, uint4 &lo) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t hw[2], lw[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float v = h2f(e ? in[i] >> 16 : in[i] & 0xFFFFu);
      hw[e] = __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u;
      const bool finite = __builtin_fabsf(v) < __builtin_inff();
      lw[e] = __builtin_bit_cast(uint32_t, finite ? v - __builtin_bit_cast(float, hw[e]) : 0.0f);
    }
    h[i] = (hw[0] >> 16) | hw[1];
    l[i] = (lw[0] >> 16) | (lw[1] & 0xFFFF0000u);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Eight bfloat16 weights for the product with lo: an infinity (scale bytes 253 and
// 254) becomes the largest number, since lo is zero for most values and infinity
// times zero would be NaN. The product with hi, whose sign lo has, gives the
// infinity, or the NaN where x is zero. (NaN becomes a number too: hi's product has it.)
__device__ __forceinline__ uint4 finite_bf16(const uint4 &w) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u16x2_t top = {0x7F7F, 0x7F7F};
    const u16x2_t m = __builtin_elementwise_min(__builtin_bit_cast(u16x2_t, in[i] & 0x7FFF7FFFu), top);
    r[i] = (in[i] & 0x80008000u) | __builtin_bit_cast(uint32_t, m);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Scale bytes of 16 consecutive blocks of a row, from block `blk` on: `at` is
// the row's first byte in rs, whose base is a whole word and which ends with
// the matrix's (or the tile's) last byte. Past the row's last block the bytes are
// that block's or 127.
__device__ __forceinline__ uint4 mx_scales16(Rsrc rs, uint32_t at, int blk, int nb) {
  const int left = nb - blk;
  const uint32_t from = at + (uint32_t)blk, to = from & ~3u;
  if ((nb & 3) == 0) {  // words lie whole in a row
    uint4 v = buf_load16(rs, from);
    if (left <= 12) v.w = 0x7F7F7F7Fu;
    if (left <= 8) v.z = 0x7F7F7F7Fu;
    if (left <= 4) v.y = 0x7F7F7F7Fu;
    return v;
  }
  if (left >= 19) {  // five words hold them, and end inside the row
    const uint4 v = buf_load16(rs, to);
    const uint32_t e = buf_load4(rs, to + 16), by = from & 3u;
    return make_uint4(__builtin_amdgcn_alignbyte(v.y, v.x, by), __builtin_amdgcn_alignbyte(v.z, v.y, by),
                      __builtin_amdgcn_alignbyte(v.w, v.z, by), __builtin_amdgcn_alignbyte(e, v.w, by));
  }
  uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int u = 0; u < 16; ++u)
    v[u >> 2] |= buf_load_u8(rs, at + (uint32_t)max(0, min(blk + u, nb - 1))) << (8 * (u & 3));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// v_mfma_f32_16x16x32 / 32x32x16 on halves of type T.
template <MxType T>
__device__ __forceinline__ float4_t mx_mfma16(const uint4 &a, const uint4 &b, float4_t c) {
  if constexpr (T == MxType::kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a),
                                                  __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bhalf8_t, a),
                                                   __builtin_bit_cast(bhalf8_t, b), c, 0, 0, 0);
}
template <MxType T>
__device__ __forceinline__ float16_t mx_mfma32(const uint4 &a, const uint4 &b, float16_t c) {
  if constexpr (T == MxType::kF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a),
                                                  __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bhalf8_t, a),
                                                   __builtin_bit_cast(bhalf8_t, b), c, 0, 0, 0);
}

// float32 -> 16 bits of T, round to nearest even.
template <MxType T> __device__ __forceinline__ uint32_t f2t(float f) {
  if constexpr (T == MxType::kF16) return f2h(f);
  else return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

// Four consecutive results of one output row: one 8-byte store where `packed`
// (n a multiple of 4, so that all four are inside or none is).
template <MxType T>
__device__ __forceinline__ void store4(uint16_t *row, int64_t c, int64_t n, const float4_t &v,
                                       bool packed) {
  if (packed) {
    if (c < n)
      *reinterpret_cast<uint2 *>(row + c) = make_uint2(f2t<T>(v[0]) | (f2t<T>(v[1]) << 16),
                                                       f2t<T>(v[2]) | (f2t<T>(v[3]) << 16));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < n) row[c + e] = (uint16_t)f2t<T>(v[e]);
  }
}

}  // namespace aqlm
