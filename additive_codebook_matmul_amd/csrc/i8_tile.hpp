// What the tile kernels of int8 products and gradients share behind their loops: sums
// of 32 x 32 matrix tiles, V the four numbers of a quarter (float or int32). Register 4 q
// + e of such a tile is result 8 q + 4 h + e along its first side and l32 along the
// tokens, (l32, h) = (lane % 32, lane / 32).
#pragma once

#include "i8_device.hpp"

namespace aqlm {

template <class A> struct I8Quarter;
template <> struct I8Quarter<int16_vt> { typedef int4_vt type; };
template <> struct I8Quarter<float16_t> { typedef float4_t type; };

template <class A> __device__ __forceinline__ typename I8Quarter<A>::type i8_quarter(const A &v, int q) {
  return {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
}

// Adds the sums of K's shares, in order, to those of share 0, through S::kSums bytes of LDS.
// True where the wavefront is done (it is not of share 0). Nothing else may be at work on
// that LDS; behind it share 0 may use all other LDS at once.
template <class S, class A>
__device__ __forceinline__ bool i8_join_shares(A (&acc)[S::RT][S::NT], int kw, int wave, int lane, uint8_t *lds) {
  if constexpr (S::KW > 1) {
    typedef typename I8Quarter<A>::type V;
    auto slot = [&](int i, int j, int q) __attribute__((always_inline)) {
      return reinterpret_cast<V *>(lds + ((((i * S::NT + j) * 4 + q) * S::kWaves + wave) * 64 + lane) * 16);
    };
#pragma unroll 1
    for (int k = 1; k < S::KW; ++k) {
      if (k > 1) __syncthreads();
      if (kw == k) {
#pragma unroll
        for (int i = 0; i < S::RT; ++i)
#pragma unroll
          for (int j = 0; j < S::NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) *slot(i, j, q) = i8_quarter(acc[i][j], q);
      }
      __syncthreads();
      if (kw == 0) {
#pragma unroll
        for (int i = 0; i < S::RT; ++i)
#pragma unroll
          for (int j = 0; j < S::NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const V v = *slot(i, j, q);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
            }
      }
    }
    return kw != 0;
  }
  return false;
}

// A part's sums into the workspace, [job][RT * NT * 4][threads], as the registers lie:
// those of tokens from tok0 on that are below batch.
template <class S, class A>
__device__ __forceinline__ void i8_store_part(const A (&acc)[S::RT][S::NT], typename I8Quarter<A>::type *part, int job,
                                              int wave, int lane, int tok0, int batch) {
  part += (int64_t)job * (S::RT * S::NT * 4 * S::kThreads) + wave * 64 + lane;
#pragma unroll
  for (int i = 0; i < S::RT; ++i)
#pragma unroll
    for (int j = 0; j < S::NT; ++j)
      if (tok0 + 32 * j + (lane & 31) < batch) {
#pragma unroll
        for (int q = 0; q < 4; ++q) part[((i * S::NT + j) * 4 + q) * S::kThreads] = i8_quarter(acc[i][j], q);
      }
}

// The sum of a quarter's parts, `stride` apart, in order.
template <class V> __device__ __forceinline__ V i8_sum_parts(const V *p, int64_t stride, int splits) {
  V v = p[0];
  for (int s = 1; s < splits; s += 4) {  // four loads under way
    V u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = p[min(s + k, splits - 1) * stride];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s + k < splits) v += u[k];
  }
  return v;
}

// Results of 32 OT by 32 tokens of a wavefront, rounded, to y [batch][rows] (rows a multiple
// of 8). A lane's values are four rows apart from the next lane's token; they pass through
// LDS (OT * 2048 bytes, the wavefront's own), from where neighbouring lanes store a token's
// rows: 8-byte stores from the registers left 16 of 64 bytes a line and took 12 to 15 us of
// 2048 x 11008 results.
template <MxType T, int OT>
__device__ __forceinline__ void i8_store_lines(const float4_t (&out)[OT][4], uint8_t *mine, int lane, uint16_t *y,
                                               int tok0, int row0, int batch, int rows) {
  constexpr int kChunks = 4 * OT;  // of 16 bytes, eight rows, for a token
  const int l32 = lane & 31, h = lane >> 5;
#pragma unroll
  for (int i = 0; i < OT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = (4 * i + q) ^ (l32 & (kChunks - 1));
      const float4_t &o = out[i][q];
      *reinterpret_cast<uint2 *>(mine + (l32 * kChunks + c) * 16 + 8 * h) =
          make_uint2(f2t<T>(o[0]) | (f2t<T>(o[1]) << 16), f2t<T>(o[2]) | (f2t<T>(o[3]) << 16));
    }
  wave_exchange();
#pragma unroll
  for (int k = 0; k < kChunks / 2; ++k) {
    const int id = 64 * k + lane, t = id / kChunks, c = id % kChunks;
    const uint4 r = *reinterpret_cast<const uint4 *>(mine + (t * kChunks + (c ^ (t & (kChunks - 1)))) * 16);
    const int tok = tok0 + t, row = row0 + 8 * c;
    if (tok < batch && row < rows) *reinterpret_cast<uint4 *>(y + (int64_t)tok * rows + row) = r;
  }
  wave_exchange();
}

}  // namespace aqlm
