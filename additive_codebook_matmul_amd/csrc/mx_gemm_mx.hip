// Product of two microscaled matrices: y = x . W^T on the block-scaled matrix
// instructions, which take E2M1 codes and E8M0 scales as they are.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with 4-bit operands: lane (r, q) = (lane %
// 16, lane / 16) gives the 16 bytes of block q (32 codes) of row r of the
// 128-input chunk and that block's scale byte, for A (rows of W) and B (rows
// of x) alike, so both sides are loaded straight from their row-major arrays.
// The wavefronts of a workgroup split the chunks and add their float32 sums
// through LDS in a fixed order.
#include <algorithm>

#include "mx_device.hpp"

namespace aqlm {
namespace {

__device__ __forceinline__ float4_t mfma_mx16(const uint4 &a, uint32_t sa, const uint4 &b,
                                              uint32_t sb, float4_t c) {
  const int8_vt av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const int8_vt bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

template <MxType T, int RT, int NT, int NW>
__global__ __launch_bounds__(NW * 64) void mx_mx_skinny_kernel(
    const uint8_t *__restrict__ wc, const uint8_t *__restrict__ wsc,
    const uint8_t *__restrict__ xc, const uint8_t *__restrict__ xsc, uint16_t *__restrict__ y,
    const int rows, const int cols, const int batch) {
  extern __shared__ __attribute__((aligned(16))) float4_t red[];  // [NW][RT * NT][64]
  const int row0 = (int)blockIdx.x * (16 * RT);
  const int tok0 = (int)blockIdx.y * (16 * NT);
  const int nb = cols >> 5;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int tile_rows = min(16 * RT, rows - row0);
  const int tile_toks = min(16 * NT, batch - tok0);
  const uint32_t half = (uint32_t)cols >> 1;
  const Rsrc crs = make_rsrc(wc + (int64_t)row0 * half, (uint32_t)tile_rows * half);
  const Rsrc srs = make_rsrc(wsc + (int64_t)row0 * nb, (uint32_t)tile_rows * nb);
  const Rsrc xrs = make_rsrc(xc + (int64_t)tok0 * half, (uint32_t)tile_toks * half);
  const Rsrc xss = make_rsrc(xsc + (int64_t)tok0 * nb, (uint32_t)tile_toks * nb);

  float4_t acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};

  const int chunks = (nb + 3) >> 2;
  for (int c = wave; c < chunks; c += NW) {
    const int blk = 4 * c + q;
    const bool in = blk < nb;  // past the row's end: codes 0 and scales 2^-127 on both sides
    uint4 w[RT], xv[NT];
    uint32_t sw[RT], sx[NT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const uint32_t r = 16u * i + r16;
      w[i] = buf_load16(crs, in ? r * half + (uint32_t)blk * 16u : kMxOOB);
      sw[i] = buf_load_u8(srs, in ? r * nb + (uint32_t)blk : kMxOOB);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint32_t t = 16u * j + r16;
      xv[j] = buf_load16(xrs, in ? t * half + (uint32_t)blk * 16u : kMxOOB);
      sx[j] = buf_load_u8(xss, in ? t * nb + (uint32_t)blk : kMxOOB);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mfma_mx16(w[i], sw[i], xv[j], sx[j], acc[i][j]);
  }

#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[(wave * (RT * NT) + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  const bool packed = (rows & 3) == 0;
  for (int e = threadIdx.x; e < RT * NT * 64; e += NW * 64) {
    float4_t v = red[e];
#pragma unroll
    for (int u = 1; u < NW; ++u) v += red[u * (RT * NT * 64) + e];
    const int l = e & 63, i = (e >> 6) / NT, j = (e >> 6) % NT;
    const int tok = tok0 + 16 * j + (l & 15);
    if (tok < batch) store4<T>(y + (int64_t)tok * rows, row0 + 16 * i + 4 * (l >> 4), rows, v, packed);
  }
}

template <MxType T, int RT, int NT, int NW>
hipError_t launch_skinny(const MxDesc &W, const MxDesc &x, void *y, hipStream_t stream) {
  const dim3 grid((unsigned)((W.rows + 16 * RT - 1) / (16 * RT)),
                  (unsigned)((x.rows + 16 * NT - 1) / (16 * NT)));
  hipLaunchKernelGGL((mx_mx_skinny_kernel<T, RT, NT, NW>), grid, dim3(NW * 64),
                     NW * RT * NT * 64 * sizeof(float4_t), stream, W.codes, W.scales, x.codes,
                     x.scales, static_cast<uint16_t *>(y), (int)W.rows, (int)W.cols, (int)x.rows);
  return hipGetLastError();
}

template <MxType T>
hipError_t gemm_mx_as(const MxDesc &W, const MxDesc &x, void *y, hipStream_t stream) {
  return launch_skinny<T, 1, 1, 8>(W, x, y, stream);
}

}  // namespace

int64_t mx_gemm_mx_ws_bytes(const MxDesc &W, int64_t batch) {
  return batch < kMxTileBatch ? 0 : mx_gemm_mx_tile_ws_bytes(W, batch);
}

hipError_t launch_mx_gemm_mx(const MxDesc &W, const MxDesc &x, void *y, MxType type, void *ws,
                             hipStream_t stream) {
  if (x.rows >= kMxTileBatch) return launch_mx_gemm_mx_tile(W, x, y, type, ws, stream);
  return type == MxType::kF16 ? gemm_mx_as<MxType::kF16>(W, x, y, stream)
                              : gemm_mx_as<MxType::kBF16>(W, x, y, stream);
}

}  // namespace aqlm
