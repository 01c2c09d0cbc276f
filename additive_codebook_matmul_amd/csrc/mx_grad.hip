// Input gradient of a microscaled layer: dx = dy . W.
//
// The sum runs over the rows of W, along which neither codes nor scales are
// contiguous, so a K step expands a [32 rows][64 columns] tile of W once into
// LDS, transposed to [column][row], where the matrix instructions read their
// operands (8 consecutive rows of one column, 16 bytes).
#include <algorithm>

#include "mx_device.hpp"

namespace aqlm {
namespace {

constexpr int kGThreads = 256;
constexpr int kGCols = 64;     // columns of W per workgroup
constexpr int kGToks = 64;     // tokens per workgroup, 16 per wavefront
constexpr int kGK = 32;        // rows of W per step
constexpr int kGStride = 40;   // halves per LDS column: 80 bytes keep 16-byte alignment

template <MxType T>
__global__ __launch_bounds__(kGThreads) void mx_grad_kernel(
    const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
    const uint16_t *__restrict__ dy, uint16_t *__restrict__ dx, const int rows, const int cols,
    const int batch) {
  __shared__ __attribute__((aligned(16))) uint16_t wt[kGCols * kGStride];
  const int col0 = (int)blockIdx.x * kGCols;
  const int tok0 = (int)blockIdx.y * kGToks;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int fo = threadIdx.x >> 3, fi = threadIdx.x & 7;  // filled row of the step, column octet
  const int tok = tok0 + 16 * wave + r16;
  const bool vec = (rows & 7) == 0;
  float4_t acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = float4_t{0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < rows; k0 += kGK) {
    const int o = k0 + fo, c = col0 + 8 * fi;
    uint32_t w = 0, sb = 127u;
    if (o < rows && c < cols) {
      w = *reinterpret_cast<const uint32_t *>(codes + (int64_t)o * (cols >> 1) + (c >> 1));
      sb = scales[(int64_t)o * (cols >> 5) + (c >> 5)];
    }
    // a step with a scale that float16 weights cannot take runs in bfloat16
    // with dy split exactly in two (the barrier also ends the last step)
    bool wide = false;
    if constexpr (T == MxType::kF16) wide = __syncthreads_or(!mx_fits_f16(sb));
    else __syncthreads();
    const uint4 v = wide ? mx_decode8<MxType::kBF16>(w, mx_scale(sb)) : mx_decode8<T>(w, mx_scale(sb));
    const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      wt[(8 * fi + e) * kGStride + fo] = (uint16_t)(vw[e >> 1] >> (16 * (e & 1)));
    __syncthreads();
    // dy of rows k0 + 8 q .. + 7: past the last row zero
    uint4 b = make_uint4(0, 0, 0, 0);
    const int ko = k0 + 8 * q;
    if (tok < batch) {
      const uint16_t *p = dy + (int64_t)tok * rows + ko;
      if (vec) {
        if (ko < rows) b = *reinterpret_cast<const uint4 *>(p);
      } else {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = ko + e < rows ? p[e] : 0u;
        b = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                       h[6] | (h[7] << 16));
      }
    }
    if (!wide) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 a = *reinterpret_cast<const uint4 *>(wt + (16 * i + r16) * kGStride + 8 * q);
        acc[i] = mx_mfma16<T>(a, b, acc[i]);
      }
    } else {
      uint4 hi, lo;
      split_f16(b, hi, lo);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 a = *reinterpret_cast<const uint4 *>(wt + (16 * i + r16) * kGStride + 8 * q);
        acc[i] = mx_mfma16<MxType::kBF16>(a, hi, acc[i]);
        acc[i] = mx_mfma16<MxType::kBF16>(a, lo, acc[i]);
      }
    }
  }
  if (tok < batch)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      store4<T>(dx + (int64_t)tok * cols, col0 + 16 * i + 4 * q, cols, acc[i], true);
}

}  // namespace

int64_t mx_grad_ws_bytes(const MxDesc &, int64_t) { return 0; }

hipError_t launch_mx_grad(const MxDesc &W, const void *dy, int64_t batch, void *dx, MxType type,
                          void *, hipStream_t stream) {
  const dim3 grid((unsigned)((W.cols + kGCols - 1) / kGCols),
                  (unsigned)((batch + kGToks - 1) / kGToks));
  const uint16_t *in = static_cast<const uint16_t *>(dy);
  uint16_t *out = static_cast<uint16_t *>(dx);
  if (type == MxType::kF16)
    hipLaunchKernelGGL(mx_grad_kernel<MxType::kF16>, grid, dim3(kGThreads), 0, stream, W.codes,
                       W.scales, in, out, (int)W.rows, (int)W.cols, (int)batch);
  else
    hipLaunchKernelGGL(mx_grad_kernel<MxType::kBF16>, grid, dim3(kGThreads), 0, stream, W.codes,
                       W.scales, in, out, (int)W.rows, (int)W.cols, (int)batch);
  return hipGetLastError();
}

}  // namespace aqlm
