// int8 quantisation by rows, and expansion.
//
// A row's scale needs its largest magnitude before its first code, so a row is
// kept in registers between the two where it fits (read once), and read again
// where it does not. Both directions move a matrix once and compute little, so HBM
// bounds them (28672 x 8192: float16 quantised in 106 us, 6.6 TB/s, expanded in 100, 7.0
// TB/s; float32, a call among others, 210 and 208, 5.6 TB/s).
#include <algorithm>

#include "i8_device.hpp"

namespace aqlm {
namespace {

// A row by WAVES wavefronts, ROUNDS octets a thread in registers; 256 / (64 WAVES)
// rows a workgroup (one from four wavefronts on).
template <MxType T, int WAVES, int ROUNDS, bool NT>
__global__ __launch_bounds__(WAVES < 4 ? 256 : WAVES * 64) void i8_quantize_rows_kernel(
    const void *__restrict__ x, uint2 *__restrict__ codes, float *__restrict__ scales, int octets, int64_t rows) {
  constexpr int kThreads = WAVES * 64, kPer = WAVES < 4 ? 4 / WAVES : 1;
  __shared__ uint32_t tops[WAVES > 1 ? WAVES : 1];
  static_assert(WAVES == 1 || WAVES >= 4, "tops are one row's");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tid = WAVES == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  for (int64_t row = (int64_t)blockIdx.x * kPer + (WAVES == 1 ? wave : 0); row < rows; row += (int64_t)gridDim.x * kPer) {
    const int64_t base = row * octets;
    Octet<T> o[ROUNDS];
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < ROUNDS; ++u) {
      const int i = tid + u * kThreads;
      if (i < octets) o[u] = load_octet<T, NT>(x, base + i);
      else o[u] = {};
    }
#pragma unroll
    for (int u = 0; u < ROUNDS; ++u) m = max(m, octet_max<T>(o[u]));
    m = wave_max(m);
    if constexpr (WAVES > 1) {
      __syncthreads();  // the row before is done with `tops`
      if ((threadIdx.x & 63) == 0) tops[wave] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WAVES; ++w) m = max(m, tops[w]);
    }
    const RowScale r = row_scale(max_bits<T>(m));
    if (tid == 0) scales[row] = r.scale;
#pragma unroll
    for (int u = 0; u < ROUNDS; ++u) {
      const int i = tid + u * kThreads;
      if (i < octets) codes[base + i] = encode_octet<T>(o[u], r);
    }
  }
}

// Rows of up to 128 values: 16 lanes a row, an octet each (28672 x 128 8.7 us by a
// wavefront a row, 4.8 this way).
template <MxType T>
__global__ __launch_bounds__(256) void i8_quantize_short_kernel(const void *__restrict__ x, uint2 *__restrict__ codes,
                                                                float *__restrict__ scales, int octets, int64_t rows) {
  const int i = threadIdx.x & 15;
  const int64_t step = (int64_t)gridDim.x * 16;
  // (lanes past the last row take its place in the maximum, and nothing else)
  for (int64_t first = (int64_t)blockIdx.x * 16; first < rows; first += step) {
    const int64_t row = first + (threadIdx.x >> 4);
    const bool in = row < rows && i < octets;
    Octet<T> o = {};
    if (in) o = load_octet<T, false>(x, row * octets + i);
    const RowScale r = row_scale(max_bits<T>(row16_max(octet_max<T>(o))));
    if (in) codes[row * octets + i] = encode_octet<T>(o, r);
    if (row < rows && i == 0) scales[row] = r.scale;
  }
}

// Rows longer than registers hold: read twice.
template <MxType T>
__global__ __launch_bounds__(1024) void i8_quantize_long_kernel(const void *__restrict__ x, uint2 *__restrict__ codes,
                                                                float *__restrict__ scales, int octets, int64_t rows) {
  __shared__ uint32_t tops[16];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t base = row * octets;
    uint32_t m = 0;
    for (int i = threadIdx.x; i < octets; i += 1024) m = max(m, octet_max<T>(load_octet<T, false>(x, base + i)));
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 16; ++w) m = max(m, tops[w]);
    const RowScale r = row_scale(max_bits<T>(m));
    if (threadIdx.x == 0) scales[row] = r.scale;
    for (int i = threadIdx.x; i < octets; i += 1024)
      codes[base + i] = encode_octet<T>(load_octet<T, false>(x, base + i), r);
    __syncthreads();
  }
}

// In pieces of 16 bytes of W, eight halves or four floats, a thread each: a store of a
// wavefront is 1 KiB in one run. 2^shift threads a row, which have kUnroll pieces under
// way each, so that short rows share a workgroup.
constexpr int kUnroll = 4;

template <MxType T, bool NT>
__global__ __launch_bounds__(256) void i8_dequant_kernel(const int8_t *__restrict__ codes,
                                                         const float *__restrict__ scales, u32x4_t *__restrict__ W,
                                                         int row_pieces, int64_t rows, int shift) {
  constexpr int kPer = T == MxType::kF32 ? 4 : 8;
  const int lanes = 1 << shift, mine = (int)threadIdx.x & (lanes - 1);
  const int64_t together = 256 >> shift;  // rows of a workgroup
  for (int64_t row = blockIdx.y * together + (threadIdx.x >> shift); row < rows; row += gridDim.y * together) {
    const float s = scales[row];
    const int64_t base = row * row_pieces;
    for (int i0 = (int)blockIdx.x * lanes * kUnroll + mine; i0 < row_pieces; i0 += (int)gridDim.x * lanes * kUnroll) {
      uint32_t c[kUnroll][kPer / 4];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int i = i0 + lanes * k;
        const uint32_t *p = reinterpret_cast<const uint32_t *>(codes + (base + i) * kPer);
#pragma unroll
        for (int e = 0; e < kPer / 4; ++e) c[k][e] = i < row_pieces ? p[e] : 0u;
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int i = i0 + lanes * k;
        if (i >= row_pieces) break;
        float v[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[e] = (float)(int8_t)(c[k][e >> 2] >> (8 * (e & 3))) * s;
        u32x4_t r;
        if constexpr (T == MxType::kF32) {
#pragma unroll
          for (int e = 0; e < 4; ++e) r[e] = __builtin_bit_cast(uint32_t, v[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) r[e] = f2t<T>(materialize(v[2 * e])) | (f2t<T>(materialize(v[2 * e + 1])) << 16);
        }
        if constexpr (NT) __builtin_nontemporal_store(r, W + base + i);
        else W[base + i] = r;
      }
    }
  }
}

unsigned row_grid(int64_t rows) { return (unsigned)std::min<int64_t>(rows, int64_t(1) << 20); }

// From these sizes on a dense matrix is read, or written, without a place in the caches,
// which then keep the codes: 28672 x 8192 quantised and expanded in turn takes 217 us in
// float16 and 379 in float32, 242 and 427 with ordinary loads, 241 and 430 with ordinary
// stores; quantised alone 122 and 210, with ordinary loads 128 and 217.
constexpr int64_t kNtLoad = (int64_t)64 << 20, kNtStore = (int64_t)256 << 20;

template <MxType T, int WAVES, int ROUNDS>
void quantize_rows(const void *x, int64_t rows, int64_t cols, int8_t *codes, float *scales, hipStream_t stream) {
  constexpr int kPer = WAVES < 4 ? 4 / WAVES : 1;
  const dim3 grid(row_grid((rows + kPer - 1) / kPer)), block(WAVES < 4 ? 256 : WAVES * 64);
  uint2 *const c = reinterpret_cast<uint2 *>(codes);
  const int octets = (int)(cols / 8);
  if (rows * cols * (T == MxType::kF32 ? 4 : 2) >= kNtLoad)
    hipLaunchKernelGGL((i8_quantize_rows_kernel<T, WAVES, ROUNDS, true>), grid, block, 0, stream, x, c, scales, octets, rows);
  else
    hipLaunchKernelGGL((i8_quantize_rows_kernel<T, WAVES, ROUNDS, false>), grid, block, 0, stream, x, c, scales, octets, rows);
}

// Wavefronts and octets a thread by the row's length: a row's wavefronts meet twice, so
// short rows take one, and a thread holds up to four octets (256 threads a row read
// twice took 10.6 us for 2048 x 4096, 5.1 this way).
template <MxType T>
void quantize_as(const void *x, int64_t rows, int64_t cols, int8_t *codes, float *scales, hipStream_t stream) {
  const int64_t octets = cols / 8;
  if (octets <= 16)
    hipLaunchKernelGGL((i8_quantize_short_kernel<T>), dim3(row_grid((rows + 15) / 16)), dim3(256), 0, stream, x,
                       reinterpret_cast<uint2 *>(codes), scales, (int)octets, rows);
  else if (octets <= 64) quantize_rows<T, 1, 1>(x, rows, cols, codes, scales, stream);
  else if (octets <= 128) quantize_rows<T, 1, 2>(x, rows, cols, codes, scales, stream);
  else if (octets <= 256) quantize_rows<T, 4, 1>(x, rows, cols, codes, scales, stream);
  else if (octets <= 512) quantize_rows<T, 4, 2>(x, rows, cols, codes, scales, stream);
  else if (octets <= 1024) quantize_rows<T, 4, 4>(x, rows, cols, codes, scales, stream);
  else if (octets <= 2048) quantize_rows<T, 8, 4>(x, rows, cols, codes, scales, stream);
  else if (octets <= 4096) quantize_rows<T, 16, 4>(x, rows, cols, codes, scales, stream);
  else
    hipLaunchKernelGGL((i8_quantize_long_kernel<T>), dim3(row_grid(rows)), dim3(1024), 0, stream, x,
                       reinterpret_cast<uint2 *>(codes), scales, (int)octets, rows);
}

template <MxType T> void dequant_as(const I8Desc &m, void *W, hipStream_t stream) {
  const int64_t pieces = m.cols / (T == MxType::kF32 ? 4 : 8);
  int shift = 1;
  while (shift < 8 && kUnroll << shift < pieces) ++shift;
  const int64_t columns = (pieces + (kUnroll << shift) - 1) / (kUnroll << shift);
  const int64_t groups = (m.rows + (256 >> shift) - 1) / (256 >> shift);
  const dim3 grid((unsigned)std::min<int64_t>(columns, 1024), (unsigned)std::min<int64_t>(groups, 65535));
  u32x4_t *const out = static_cast<u32x4_t *>(W);
  if (m.rows * pieces * 16 >= kNtStore)
    hipLaunchKernelGGL((i8_dequant_kernel<T, true>), grid, dim3(256), 0, stream, m.codes, m.scales, out, (int)pieces,
                       m.rows, shift);
  else
    hipLaunchKernelGGL((i8_dequant_kernel<T, false>), grid, dim3(256), 0, stream, m.codes, m.scales, out, (int)pieces,
                       m.rows, shift);
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
