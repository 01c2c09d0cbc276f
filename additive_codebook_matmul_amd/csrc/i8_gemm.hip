// Products of int8 layers and gated blocks.
//
// i8_skinny_kernel: a workgroup computes 16 rows of W (GATED: of both matrices)
// for 16 NT tokens. Its wavefronts share K in groups of 256 inputs: lane (r, q)
// loads the 16 bytes at 64 c + 16 q of row r of W and of x for the four chunks c,
// just what v_mfma_i32_16x16x64_i8 takes. The integer sums meet in LDS. It serves short
// layers, where a launch and two or three round trips to memory are all there is (16 x
// 4096 x 4096 7.2 us, 2048 x 1024 3.6).
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
  const Rsrc w0rs = make_rsrc(A.w[0] + (int64_t)row0 * cols, (uint32_t)tile_rows * cols);
  const Rsrc w1rs = make_rsrc((GATED ? A.w[1] : A.w[0]) + (int64_t)row0 * cols, (uint32_t)tile_rows * cols);
  const Rsrc xrs = make_rsrc(A.x + (int64_t)tok0 * cols, (uint32_t)batch * cols);

  int4_vt acc[M][NT];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[m][j] = int4_vt{0, 0, 0, 0};
  // a group of 256 inputs, loaded while the one before is multiplied
  struct Group {
    uint4 w[M][4], x[NT][4];
  };
  auto load = [&](uint32_t k0, Group &g) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t k = k0 + 64u * c + 16u * q;
      const uint32_t at = k < cols ? (uint32_t)r16 * cols + k : kMxOOB;
      g.w[0][c] = buf_load16(w0rs, at);
      if constexpr (GATED) g.w[M - 1][c] = buf_load16(w1rs, at);
#pragma unroll
      for (int j = 0; j < NT; ++j) g.x[j][c] = buf_load16(xrs, k < cols ? at + (uint32_t)(16 * j) * cols : kMxOOB);
    }
  };
  auto products = [&](const Group &g) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[m][j] = i8_mfma16(g.w[m][c], g.x[j][c], acc[m][j]);
  };
  Group g0, g1;
  uint32_t k = 256u * wave;
  load(k, g0);
  for (; k < cols; k += 512u * NW) {
    load(k + 256u * NW, g1);
    products(g0);
    if (k + 256u * NW >= cols) break;
    load(k + 512u * NW, g0);
    products(g1);
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

template <MxType T, bool GATED> hipError_t skinny_as(const I8Args &A, hipStream_t stream) {
  const unsigned tiles = (unsigned)((A.rows + 15) / 16);
  if (A.batch <= 16)
    hipLaunchKernelGGL((i8_skinny_kernel<T, GATED, 8, 1>), dim3(tiles), dim3(512), 0, stream, A);
  else
    hipLaunchKernelGGL((i8_skinny_kernel<T, GATED, 8, 2>), dim3(tiles, (unsigned)((A.batch + 31) / 32)), dim3(512), 0,
                       stream, A);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_product(const I8Product &p, const I8Route &route, void *ws, hipStream_t stream) {
  I8Args A = {{p.W.codes, p.up.codes}, {p.W.scales, p.up.scales}, p.xcodes, p.xscales,
              static_cast<uint16_t *>(p.y), p.g, p.u, (int)p.W.rows, (int)p.W.cols, (int)p.batch, p.act};
  if (route.inside) return launch_i8_rows(A, p.x, p.type, p.gated(), stream);
  if (p.x) {
    float *scales = static_cast<float *>(ws);
    int8_t *codes = static_cast<int8_t *>(ws) + i8_codes_at(p.batch);
    const hipError_t e = launch_i8_quantize(p.x, p.type, p.batch, p.W.cols, codes, scales, stream);
    if (e != hipSuccess) return e;
    A.x = codes;
    A.xs = scales;
    ws = static_cast<uint8_t *>(ws) + i8_product_at(p.W.cols, p.batch);
  }
  if (route.kind == I8Route::kRows) return launch_i8_rows(A, nullptr, p.type, p.gated(), stream);
  if (route.kind == I8Route::kTiles) return launch_i8_tile(A, route.plan, p.type, p.gated(), ws, stream);
  if (p.type == MxType::kF16)
    return p.gated() ? skinny_as<MxType::kF16, true>(A, stream) : skinny_as<MxType::kF16, false>(A, stream);
  return p.gated() ? skinny_as<MxType::kBF16, true>(A, stream) : skinny_as<MxType::kBF16, false>(A, stream);
}

}  // namespace aqlm
