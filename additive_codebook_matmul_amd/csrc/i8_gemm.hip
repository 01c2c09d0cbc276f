// Products of int8 layers and gated blocks.
//
// i8_skinny_kernel: a workgroup computes 16 rows of W (GATED: of both matrices)
// for 16 NT tokens. Its wavefronts share K in groups of 256 inputs: lane (r, q)
// loads the 16 bytes at 64 c + 16 q of row r of W and of x for the four chunks c,
// just what v_mfma_i32_16x16x64_i8 takes. The integer sums meet in LDS.
#include <algorithm>

#include "i8_gemm.hpp"

namespace aqlm {
namespace {

template <MxType T, bool GATED, int NW, int NT>
__global__ __launch_bounds__(NW * 64) void i8_skinny_kernel(const I8Args A) {
  constexpr int M = GATED ? 2 : 1;
  __shared__ __attribute__((aligned(16))) int4_vt red[M][NT][NW * 64];
  const int tok0 = 16 * NT * (int)blockIdx.y, batch = min(16 * NT, A.batch - tok0);
  const int row0 = (int)blockIdx.x * 16;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const uint32_t cols = (uint32_t)A.cols;
  // resources that end with the tile's last row: rows past it read zero
  const int tile_rows = __builtin_amdgcn_readfirstlane(min(16, A.rows - row0));
  Rsrc wrs[M];
#pragma unroll
  for (int m = 0; m < M; ++m) wrs[m] = make_rsrc(A.w[m] + (int64_t)row0 * cols, (uint32_t)tile_rows * cols);
  const Rsrc xrs = make_rsrc(A.x + (int64_t)tok0 * cols, (uint32_t)batch * cols);

  int4_vt acc[M][NT];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[m][j] = int4_vt{0, 0, 0, 0};
  for (uint32_t k0 = 256u * wave; k0 < cols; k0 += 256u * NW) {
    uint4 w[M][4], x[NT][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t k = k0 + 64u * c + 16u * q;
      const uint32_t at = k < cols ? (uint32_t)r16 * cols + k : kMxOOB;
#pragma unroll
      for (int m = 0; m < M; ++m) w[m][c] = buf_load16(wrs[m], at);
#pragma unroll
      for (int j = 0; j < NT; ++j) x[j][c] = buf_load16(xrs, k < cols ? at + (uint32_t)(16 * j) * cols : kMxOOB);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[m][j] = i8_mfma16(w[m][c], x[j][c], acc[m][j]);
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[m][j][threadIdx.x] = acc[m][j];
  __syncthreads();
  // lane (t, q) holds rows 4 q .. 4 q + 3 of token t; wavefront j adds up tile j
  if (wave < NT) {
    int4_vt v[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      v[m] = red[m][wave][lane];
#pragma unroll
      for (int k = 1; k < NW; ++k) v[m] += red[m][wave][k * 64 + lane];
    }
    const int tok = 16 * wave + r16;
    if (tok < batch && row0 + 4 * q < A.rows) i8_store4<T, GATED>(A, tok0 + tok, row0 + 4 * q, v);
  }
}

template <MxType T, bool GATED> hipError_t product_as(const I8Args &A, hipStream_t stream) {
  constexpr int NW = 8;
  const unsigned tiles = (unsigned)((A.rows + 15) / 16);
  if (A.batch <= 16)
    hipLaunchKernelGGL((i8_skinny_kernel<T, GATED, NW, 1>), dim3(tiles), dim3(NW * 64), 0, stream, A);
  else
    hipLaunchKernelGGL((i8_skinny_kernel<T, GATED, NW, 4>), dim3(tiles, (unsigned)((A.batch + 63) / 64)),
                       dim3(NW * 64), 0, stream, A);
  return hipGetLastError();
}

// Workspace of quantised activations: scales, then codes, from multiples of 256 bytes on.
int64_t codes_at(int64_t batch) { return (batch * 4 + 255) / 256 * 256; }
int64_t product_at(const I8Desc &W, int64_t batch) { return codes_at(batch) + (batch * W.cols + 255) / 256 * 256; }

bool tiles_pay(const I8Desc &, bool, int64_t batch) { return batch > 32; }

}  // namespace

int64_t i8_product_ws_bytes(const I8Desc &W, bool gated, int64_t batch, bool quant) {
  return (quant ? product_at(W, batch) : 0) +
         (tiles_pay(W, gated, batch) ? i8_tile_ws_bytes(W.rows, W.cols, gated, batch) : 0);
}

hipError_t launch_i8_product(const I8Product &p, void *ws, hipStream_t stream) {
  I8Args A = {{p.W.codes, p.up.codes}, {p.W.scales, p.up.scales}, p.xcodes, p.xscales,
              static_cast<uint16_t *>(p.y), p.g, p.u, (int)p.W.rows, (int)p.W.cols, (int)p.batch, p.act};
  if (p.x) {
    float *scales = static_cast<float *>(ws);
    int8_t *codes = static_cast<int8_t *>(ws) + codes_at(p.batch);
    const hipError_t e = launch_i8_quantize(p.x, p.type, p.batch, p.W.cols, codes, scales, stream);
    if (e != hipSuccess) return e;
    A.x = codes;
    A.xs = scales;
    ws = static_cast<uint8_t *>(ws) + product_at(p.W, p.batch);
  }
  if (tiles_pay(p.W, p.gated(), p.batch)) return launch_i8_tile(A, p.type, p.gated(), ws, stream);
  if (p.type == MxType::kF16)
    return p.gated() ? product_as<MxType::kF16, true>(A, stream) : product_as<MxType::kF16, false>(A, stream);
  return p.gated() ? product_as<MxType::kBF16, true>(A, stream) : product_as<MxType::kBF16, false>(A, stream);
}

}  // namespace aqlm
