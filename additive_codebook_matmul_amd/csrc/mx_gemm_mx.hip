// Product of two microscaled matrices for up to 16 rows of activations: y = x .
// W^T on the block-scaled matrix instructions, which take E2M1 codes and E8M0
// scales as they are. (Larger tiles, and more rows: mx_gemm_mx_tile.hip.)
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with 4-bit operands: lane (r, q) = (lane %
// 16, lane / 16) gives the 16 bytes of block q (32 codes) of row r of the
// 128-input chunk and that block's scale byte, for A (rows of W) and B (rows
// of x) alike, so both sides are loaded straight from their row-major arrays.
// The wavefronts of a workgroup share K in groups of 512 inputs, four chunks
// with 16 scale bytes of a row, and add their float32 sums through LDS in a
// fixed order.
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

template <MxType T, int NW>
__global__ __launch_bounds__(NW * 64) void mx_mx_skinny_kernel(
    const uint8_t *__restrict__ wc, const uint8_t *__restrict__ wsc,
    const uint8_t *__restrict__ xc, const uint8_t *__restrict__ xsc, uint16_t *__restrict__ y,
    const int rows, const int cols, const int batch) {
  __shared__ __attribute__((aligned(16))) float4_t red[NW * 64];
  const int row0 = (int)blockIdx.x * 16;
  const int nb = cols >> 5;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  // resources that end with the tile's last row: rows past it read zero (their
  // scales are those of the last one)
  const int tile_rows = __builtin_amdgcn_readfirstlane(min(16, rows - row0));
  const uint32_t half = (uint32_t)cols >> 1;
  const int base = (int)(((int64_t)row0 * nb) & 3);
  const Rsrc crs = make_rsrc(wc + (int64_t)row0 * half, (uint32_t)tile_rows * half);
  const Rsrc srs = make_rsrc(wsc + (int64_t)row0 * nb - base, (uint32_t)tile_rows * nb + base);
  const Rsrc xrs = make_rsrc(xc, (uint32_t)batch * half);
  const Rsrc xss = make_rsrc(xsc, (uint32_t)batch * nb);
  const uint32_t srow = (uint32_t)min(r16, tile_rows - 1) * nb + base;
  const uint32_t xrow = (uint32_t)min(r16, batch - 1) * nb;

  float4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int gr = wave; 16 * gr < nb; gr += NW) {
    uint4 w[4], x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int blk = 16 * gr + 4 * c + q;
      const uint32_t at = blk < nb ? (uint32_t)r16 * half + (uint32_t)blk * 16u : kMxOOB;
      w[c] = buf_load16_nt(crs, at);
      x[c] = buf_load16(xrs, at);
    }
    const uint4 sw = mx_scales16(srs, srow, 16 * gr, nb), sx = mx_scales16(xss, xrow, 16 * gr, nb);
    const uint32_t swv[4] = {sw.x, sw.y, sw.z, sw.w}, sxv[4] = {sx.x, sx.y, sx.z, sx.w};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      acc = mfma_mx16(w[c], swv[c] >> (8 * q), x[c], sxv[c] >> (8 * q), acc);
  }

  red[threadIdx.x] = acc;
  __syncthreads();
  // lane (t, q) holds rows 4 q .. 4 q + 3 of token t
  if (threadIdx.x < 64) {
    float4_t v = red[lane];
#pragma unroll
    for (int u = 1; u < NW; ++u) v += red[u * 64 + lane];
    if (r16 < batch) store4<T>(y + (int64_t)r16 * rows, row0 + 4 * q, rows, v, (rows & 3) == 0);
  }
}

template <MxType T, int NW>
hipError_t launch_skinny(const MxDesc &W, const MxDesc &x, void *y, hipStream_t stream) {
  hipLaunchKernelGGL((mx_mx_skinny_kernel<T, NW>), dim3((unsigned)((W.rows + 15) / 16)), dim3(NW * 64), 0,
                     stream, W.codes, W.scales, x.codes, x.scales, static_cast<uint16_t *>(y), (int)W.rows,
                     (int)W.cols, (int)x.rows);
  return hipGetLastError();
}

constexpr int kSkinnyWaves = 8;

// Where the tile kernel is the faster: the skinny one takes 0.9 ns and 0.02 ns a
// row of activations for 16 rows of W and a group of K, spread over the chip,
// or, with few rows, 1.1 us and 0.07 us a row for each turn of its wavefronts
// (fitted to 1024 x 8192 .. 28672 x 8192 at 1, 5 and 16 rows: 4096 x 4096 at 5
// 4.3 us against 6.6, 28672 x 8192 32.2 against 27.4).
bool tiles_pay(const MxDesc &W, int64_t batch) {
  if (batch > 16) return true;
  const double groups = (double)((W.cols / 32 + 15) / 16), tiles = (double)((W.rows + 15) / 16);
  const double turns = (double)(int64_t)((groups + kSkinnyWaves - 1) / kSkinnyWaves);
  const double us = std::max(2.5 + tiles * groups * (0.9e-3 + 0.02e-3 * (double)batch),
                             2.5 + turns * (1.1 + 0.07 * (double)batch));
  return mx_gemm_mx_tile_us(W, batch) < us;
}

// Workspace of quantisation and product: codes, scales, the product's own, each
// from a multiple of 256 bytes on. (One kernel that quantises x into LDS, every
// workgroup again, took about as long as the two: one token with 4096 x 4096 4.7
// us against 5.4, with 28672 x 8192 34 against 30, five with 4096 x 11008 12.7
// against 11.2.)
int64_t ws_scales_at(const MxDesc &W, int64_t batch) { return (batch * (W.cols / 2) + 255) / 256 * 256; }
int64_t ws_product_at(const MxDesc &W, int64_t batch) {
  return ws_scales_at(W, batch) + (batch * (W.cols / 32) + 255) / 256 * 256;
}

}  // namespace

int64_t mx_gemm_quant_ws_bytes(const MxDesc &W, int64_t batch) {
  return ws_product_at(W, batch) + mx_gemm_mx_ws_bytes(W, batch);
}

hipError_t launch_mx_gemm_quant(const MxDesc &W, const void *x, int64_t batch, bool ceil_rule, void *y, MxType type,
                                void *ws, hipStream_t stream) {
  uint8_t *const at = static_cast<uint8_t *>(ws);
  uint8_t *const scales = at + ws_scales_at(W, batch);
  const hipError_t e = launch_mx_quantize(x, type, batch, W.cols, ceil_rule, at, scales, stream);
  if (e != hipSuccess) return e;
  return launch_mx_gemm_mx(W, {batch, W.cols, at, scales}, y, type, at + ws_product_at(W, batch), stream);
}

int64_t mx_gemm_mx_ws_bytes(const MxDesc &W, int64_t batch) {
  return tiles_pay(W, batch) ? mx_gemm_mx_tile_ws_bytes(W, batch) : 0;
}

hipError_t launch_mx_gemm_mx(const MxDesc &W, const MxDesc &x, void *y, MxType type, void *ws,
                             hipStream_t stream) {
  if (tiles_pay(W, x.rows)) return launch_mx_gemm_mx_tile(W, x, y, type, ws, stream);
  return type == MxType::kF16 ? launch_skinny<MxType::kF16, kSkinnyWaves>(W, x, y, stream)
                              : launch_skinny<MxType::kBF16, kSkinnyWaves>(W, x, y, stream);
}

}  // namespace aqlm
