// int8 quantisation by rows, and expansion.
//
// A row's scale needs its largest magnitude before its first code, so a row is
// kept in registers between the two where it fits (read once), and read again
// where it does not.
#include <algorithm>

#include "i8_device.hpp"

namespace aqlm {
namespace {

template <MxType T>
__global__ __launch_bounds__(256) void i8_quantize_kernel(const void *__restrict__ x, uint2 *__restrict__ codes,
                                                          float *__restrict__ scales, int octets, int64_t rows) {
  __shared__ uint32_t tops[4];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t base = row * octets;
    uint32_t m = 0;
    for (int i = threadIdx.x; i < octets; i += 256) m = max(m, octet_max<T>(load_octet<T, false>(x, base + i)));
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = m;
    __syncthreads();
    m = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    const RowScale r = row_scale(max_bits<T>(m));
    if (threadIdx.x == 0) scales[row] = r.scale;
    for (int i = threadIdx.x; i < octets; i += 256)
      codes[base + i] = encode_octet<T>(load_octet<T, false>(x, base + i), r);
    __syncthreads();
  }
}

// In pieces of 16 bytes of W, eight halves or four floats, a thread each.
template <MxType T>
__global__ __launch_bounds__(256) void i8_dequant_kernel(const int8_t *__restrict__ codes,
                                                         const float *__restrict__ scales, u32x4_t *__restrict__ W,
                                                         int row_pieces, int64_t rows) {
  constexpr int kPer = T == MxType::kF32 ? 4 : 8;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float s = scales[row];
    const int64_t base = row * row_pieces;
    for (int i = threadIdx.x; i < row_pieces; i += 256) {
      const uint32_t *p = reinterpret_cast<const uint32_t *>(codes + (base + i) * kPer);
      float v[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[e] = (float)(int8_t)(p[e >> 2] >> (8 * (e & 3))) * s;
      u32x4_t r;
      if constexpr (T == MxType::kF32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = __builtin_bit_cast(uint32_t, v[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = f2t<T>(materialize(v[2 * e])) | (f2t<T>(materialize(v[2 * e + 1])) << 16);
      }
      W[base + i] = r;
    }
  }
}

unsigned row_grid(int64_t rows) { return (unsigned)std::min<int64_t>(rows, int64_t(1) << 20); }

template <MxType T>
void quantize_as(const void *x, int64_t rows, int64_t cols, int8_t *codes, float *scales, hipStream_t stream) {
  hipLaunchKernelGGL((i8_quantize_kernel<T>), dim3(row_grid(rows)), dim3(256), 0, stream, x,
                     reinterpret_cast<uint2 *>(codes), scales, (int)(cols / 8), rows);
}

template <MxType T> void dequant_as(const I8Desc &m, void *W, hipStream_t stream) {
  hipLaunchKernelGGL((i8_dequant_kernel<T>), dim3(row_grid(m.rows)), dim3(256), 0, stream, m.codes, m.scales,
                     static_cast<u32x4_t *>(W), (int)(m.cols / (T == MxType::kF32 ? 4 : 8)), m.rows);
}

}  // namespace

hipError_t launch_i8_quantize(const void *x, MxType type, int64_t rows, int64_t cols, int8_t *codes, float *scales,
                              hipStream_t stream) {
  switch (type) {
    case MxType::kF16: quantize_as<MxType::kF16>(x, rows, cols, codes, scales, stream); break;
    case MxType::kBF16: quantize_as<MxType::kBF16>(x, rows, cols, codes, scales, stream); break;
    case MxType::kF32: quantize_as<MxType::kF32>(x, rows, cols, codes, scales, stream); break;
  }
  return hipGetLastError();
}

hipError_t launch_i8_dequant(const I8Desc &m, MxType type, void *W, hipStream_t stream) {
  switch (type) {
    case MxType::kF16: dequant_as<MxType::kF16>(m, W, stream); break;
    case MxType::kBF16: dequant_as<MxType::kBF16>(m, W, stream); break;
    case MxType::kF32: dequant_as<MxType::kF32>(m, W, stream); break;
  }
  return hipGetLastError();
}

}  // namespace aqlm
