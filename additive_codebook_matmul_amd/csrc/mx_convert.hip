// Microscaled quantisation and expansion.
//
// Both move whole matrices once and compute next to nothing, so HBM bounds
// them (28672 x 8192 float16: quantised at 5.9 TB/s, expanded at 6.1). To quantise,
// a thread owns eight consecutive columns (an octet: one 16-byte access of a half
// matrix, one word of codes), so four neighbouring lanes share a block of 32 and
// every access of a wavefront is contiguous.
#include <algorithm>

#include "mx_device.hpp"

namespace aqlm {
namespace {

constexpr int kCThreads = 256;
constexpr int kCUnroll = 4;  // octets per thread, a block's threads apart

template <MxType T, bool CEIL, bool NT>
__global__ __launch_bounds__(kCThreads) void mx_quantize_kernel(const void *__restrict__ x,
                                                                uint32_t *__restrict__ codes,
                                                                uint8_t *__restrict__ scales,
                                                                int64_t octets) {
  // octets is a multiple of 4 and so is every thread group's start: the four
  // lanes of a block are all inside or all outside
  const int64_t step = (int64_t)gridDim.x * (kCThreads * kCUnroll);
  for (int64_t base = (int64_t)blockIdx.x * (kCThreads * kCUnroll) + threadIdx.x; base < octets;
       base += step) {
    Octet<T> o[kCUnroll];
#pragma unroll
    for (int u = 0; u < kCUnroll; ++u) {
      const int64_t i = base + u * kCThreads;
      if (i < octets) o[u] = load_octet<T, NT>(x, i);
      else o[u] = {};
    }
#pragma unroll
    for (int u = 0; u < kCUnroll; ++u) {
      const int64_t i = base + u * kCThreads;
      const uint32_t b = scale_byte<CEIL>(block_max<T>(o[u]));
      const uint32_t c = b == 255u ? 0u : encode8<T>(o[u], mx_scale(b));
      if (i < octets) {
        codes[i] = c;
        if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)b;
      }
    }
  }
}

// In pieces of 16 bytes of W, eight halves or four floats, a thread each: a store
// of a wavefront is 1 KiB in one run. (float32 by eights, two stores 32 bytes apart,
// took 246 us for 940 MB.)
template <MxType T, bool NT>
__global__ __launch_bounds__(kCThreads) void mx_dequant_kernel(const uint8_t *__restrict__ codes,
                                                               const uint8_t *__restrict__ scales,
                                                               u32x4_t *__restrict__ W,
                                                               int64_t pieces) {
  typedef std::conditional_t<T == MxType::kF32, uint16_t, uint32_t> Codes;
  constexpr int kBlockShift = T == MxType::kF32 ? 3 : 2;  // of a block's pieces
  const Codes *const cp = reinterpret_cast<const Codes *>(codes);
  const int64_t step = (int64_t)gridDim.x * (kCThreads * kCUnroll);
  for (int64_t base = (int64_t)blockIdx.x * (kCThreads * kCUnroll) + threadIdx.x; base < pieces;
       base += step) {
    uint32_t c[kCUnroll], b[kCUnroll];
#pragma unroll
    for (int u = 0; u < kCUnroll; ++u) {
      const int64_t i = base + u * kCThreads;
      const bool in = i < pieces;
      c[u] = in ? (uint32_t)cp[i] : 0u;
      b[u] = in ? scales[i >> kBlockShift] : 127u;
    }
#pragma unroll
    for (int u = 0; u < kCUnroll; ++u) {
      const int64_t i = base + u * kCThreads;
      if (i >= pieces) break;
      const float s = mx_scale(b[u]);
      u32x4_t r;
      if constexpr (T == MxType::kF32) {
        typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
        const u32x2_t lo = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], s, 0));
        const u32x2_t hi = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], s, 1));
        r = u32x4_t{lo.x, lo.y, hi.x, hi.y};
      } else {
        const uint4 v = mx_decode8<T>(c[u], s);
        r = u32x4_t{v.x, v.y, v.z, v.w};
      }
      if constexpr (NT) __builtin_nontemporal_store(r, W + i);
      else W[i] = r;
    }
  }
}

// Workgroups of a pass over `octets`: one per kCUnroll * kCThreads octets, up to
// 2^30 threads (each then takes several turns).
unsigned convert_grid(int64_t octets) {
  const int64_t per = kCThreads * kCUnroll;
  return (unsigned)std::min<int64_t>((octets + per - 1) / per, int64_t(1) << 22);
}

// From these sizes on a half matrix is read, or a matrix written, without a place
// in the caches. A matrix to quantise is read once: 90 MB 22.1 us, without caching
// 19.2 (48.4 and 42.8 together with the kernel that writes it), 470 MB 103.4 and
// 99.9, but 45 MB that lie in the cache 9.9 and 10.5. What is expanded may be read
// next, so that only what the last-level cache (256 MB) cannot hold passes it: 470
// MB 101.3 and 97.1, and 254 and 250 together with a kernel that reads it; 90 MB
// 24.2 and 17.5, but 47 and 54. (470 MB quantised and expanded in turn: 223 and
// 174.) float32 is quantised by two accesses a thread, 32 bytes apart, of which the
// second finds its line in the cache: 940 MB 200 and, without caching, 205.
constexpr int64_t kNtLoad = (int64_t)64 << 20, kNtStore = (int64_t)256 << 20;

template <MxType T, bool CEIL>
void quantize_as(const void *x, int64_t octets, uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  const dim3 grid(convert_grid(octets)), block(kCThreads);
  uint32_t *cw = reinterpret_cast<uint32_t *>(codes);
  if constexpr (T != MxType::kF32)
    if (octets * 16 >= kNtLoad) {
      hipLaunchKernelGGL((mx_quantize_kernel<T, CEIL, true>), grid, block, 0, stream, x, cw, scales, octets);
      return;
    }
  hipLaunchKernelGGL((mx_quantize_kernel<T, CEIL, false>), grid, block, 0, stream, x, cw, scales, octets);
}

template <MxType T>
void quantize_by(const void *x, int64_t octets, bool ceil_rule, uint8_t *codes, uint8_t *scales, hipStream_t stream) {
  if (ceil_rule) quantize_as<T, true>(x, octets, codes, scales, stream);
  else quantize_as<T, false>(x, octets, codes, scales, stream);
}

template <MxType T> void dequant_as(const MxDesc &m, void *W, hipStream_t stream) {
  const int64_t pieces = m.rows * m.cols / (T == MxType::kF32 ? 4 : 8);
  const dim3 grid(convert_grid(pieces)), block(kCThreads);
  u32x4_t *out = static_cast<u32x4_t *>(W);
  if (pieces * 16 >= kNtStore)
    hipLaunchKernelGGL((mx_dequant_kernel<T, true>), grid, block, 0, stream, m.codes, m.scales, out, pieces);
  else
    hipLaunchKernelGGL((mx_dequant_kernel<T, false>), grid, block, 0, stream, m.codes, m.scales, out, pieces);
}

}  // namespace

hipError_t launch_mx_quantize(const void *x, MxType type, int64_t rows, int64_t cols,
                              bool ceil_rule, uint8_t *codes, uint8_t *scales,
                              hipStream_t stream) {
  const int64_t octets = rows * cols / 8;
  switch (type) {
    case MxType::kF16: quantize_by<MxType::kF16>(x, octets, ceil_rule, codes, scales, stream); break;
    case MxType::kBF16: quantize_by<MxType::kBF16>(x, octets, ceil_rule, codes, scales, stream); break;
    case MxType::kF32: quantize_by<MxType::kF32>(x, octets, ceil_rule, codes, scales, stream); break;
  }
  return hipGetLastError();
}

hipError_t launch_mx_dequant(const MxDesc &m, MxType type, void *W, hipStream_t stream) {
  switch (type) {
    case MxType::kF16: dequant_as<MxType::kF16>(m, W, stream); break;
    case MxType::kBF16: dequant_as<MxType::kBF16>(m, W, stream); break;
    case MxType::kF32: dequant_as<MxType::kF32>(m, W, stream); break;
  }
  return hipGetLastError();
}

}  // namespace aqlm
