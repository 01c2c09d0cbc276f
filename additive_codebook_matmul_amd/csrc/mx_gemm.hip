// Product of half activations with microscaled weights: y = x . W^T.
//
// A wavefront takes chunks of 128 inputs of 16-row tiles. Lane (r, q) = (lane
// % 16, lane / 16) loads the 16 bytes that hold block q of the chunk of row r
// (32 codes, one scale byte) and expands them with v_cvt_scalef32_pk into four
// operands of v_mfma_f32_16x16x32: step s multiplies codes 8 s .. 8 s + 7 of
// every block, so the activation operand of lane (t, q) is the 16 bytes of
// inputs 32 q + 8 s of token t. The sum over K does not care which inputs meet
// in one instruction, so no code ever changes lanes. The wavefronts of a
// workgroup split the chunks and add their float32 sums through LDS in a fixed
// order.
#include <algorithm>

#include "mx_device.hpp"

namespace aqlm {
namespace {

struct Group {
  struct Item {
    const uint8_t *codes;
    const uint8_t *scales;
    const uint16_t *x;
    uint16_t *y;
    int rows, cols;
  } item[kMxGroup];
  int first[kMxGroup + 1];  // first workgroup of each layer
  int n;
};

template <MxType T, int RT, int NT, int NW>
__global__ __launch_bounds__(NW * 64) void mx_skinny_kernel(const Group g, const int batch) {
  extern __shared__ __attribute__((aligned(16))) float4_t red[];  // [NW][RT * NT][64]
  int li = 0;
  while (li + 1 < g.n && (int)blockIdx.x >= g.first[li + 1]) ++li;
  const Group::Item &L = g.item[li];
  const int row0 = ((int)blockIdx.x - g.first[li]) * (16 * RT);
  const int tok0 = (int)blockIdx.y * (16 * NT);
  const int rows = L.rows, cols = L.cols;
  const int nb = cols >> 5;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;

  // resources that end with the tile's last row: rows past it read zero
  const int tile_rows = min(16 * RT, rows - row0);
  const int tile_toks = min(16 * NT, batch - tok0);
  const Rsrc crs = make_rsrc(L.codes + (int64_t)row0 * (cols >> 1), (uint32_t)tile_rows * (cols >> 1));
  const Rsrc srs = make_rsrc(L.scales + (int64_t)row0 * nb, (uint32_t)tile_rows * nb);
  const Rsrc xrs = make_rsrc(L.x + (int64_t)tok0 * cols, (uint32_t)tile_toks * cols * 2u);

  float4_t acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};

  const int chunks = (nb + 3) >> 2;
  for (int c = wave; c < chunks; c += NW) {
    const int blk = 4 * c + q;
    const bool in = blk < nb;
    uint4 w[RT];
    uint32_t sb[RT];
    uint4 xv[NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = 16 * i + r16;
      w[i] = buf_load16(crs, in ? (uint32_t)r * (cols >> 1) + (uint32_t)blk * 16u : kMxOOB);
      sb[i] = buf_load_u8(srs, in ? (uint32_t)r * nb + (uint32_t)blk : kMxOOB);
      sb[i] = in && r < tile_rows ? sb[i] : 127u;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        xv[j][s] = buf_load16(
            xrs, in ? (uint32_t)(16 * j + r16) * cols * 2u + (uint32_t)blk * 64u + 16u * s : kMxOOB);
    bool fits = true;
    if constexpr (T == MxType::kF16) {
#pragma unroll
      for (int i = 0; i < RT; ++i) fits = fits && mx_fits_f16(sb[i]);
      fits = __all(fits);
    }
    if (fits) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const float sc = mx_scale(sb[i]);
        const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint4 a = mx_decode8<T>(ww[s], sc);
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = mx_mfma16<T>(a, xv[j][s], acc[i][j]);
        }
      }
    } else {
      // scales that float16 weights cannot take: the same product in
      // bfloat16, which holds every weight, with x split exactly in two
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint4 hi, lo;
          split_f16(xv[j][s], hi, lo);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            const uint4 a = mx_decode8<MxType::kBF16>(ww[s], mx_scale(sb[i]));
            acc[i][j] = mx_mfma16<MxType::kBF16>(a, hi, acc[i][j]);
            acc[i][j] = mx_mfma16<MxType::kBF16>(a, lo, acc[i][j]);
          }
        }
    }
  }

#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[(wave * (RT * NT) + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // lane (t, q) of tile (i, j) holds rows 4 q .. 4 q + 3 of token t
  const bool packed = (rows & 3) == 0;
  for (int e = threadIdx.x; e < RT * NT * 64; e += NW * 64) {
    float4_t v = red[e];
#pragma unroll
    for (int u = 1; u < NW; ++u) v += red[u * (RT * NT * 64) + e];
    const int l = e & 63, i = (e >> 6) / NT, j = (e >> 6) % NT;
    const int tok = tok0 + 16 * j + (l & 15);
    if (tok < batch) store4<T>(L.y + (int64_t)tok * rows, row0 + 16 * i + 4 * (l >> 4), rows, v, packed);
  }
}

template <MxType T, int RT, int NT, int NW>
hipError_t launch_skinny(Group &g, int64_t batch, hipStream_t stream) {
  int blocks = 0;
  for (int i = 0; i < g.n; ++i) {
    g.first[i] = blocks;
    blocks += (g.item[i].rows + 16 * RT - 1) / (16 * RT);
  }
  g.first[g.n] = blocks;
  const dim3 grid((unsigned)blocks, (unsigned)((batch + 16 * NT - 1) / (16 * NT)));
  hipLaunchKernelGGL((mx_skinny_kernel<T, RT, NT, NW>), grid, dim3(NW * 64),
                     NW * RT * NT * 64 * sizeof(float4_t), stream, g, (int)batch);
  return hipGetLastError();
}

Group::Item item_of(const MxDesc &W, const void *x, void *y) {
  return {W.codes, W.scales, static_cast<const uint16_t *>(x), static_cast<uint16_t *>(y),
          (int)W.rows, (int)W.cols};
}

template <MxType T>
hipError_t gemm_as(const MxDesc &W, const void *x, int64_t batch, void *y, hipStream_t stream) {
  Group g;
  g.n = 1;
  g.item[0] = item_of(W, x, y);
  return launch_skinny<T, 1, 1, 8>(g, batch, stream);
}

}  // namespace

hipError_t launch_mx_gemv_batched(const MxDesc *W, const void *const *x, void *const *y, int n,
                                  int batch, MxType type, hipStream_t stream) {
  Group g;
  g.n = n;
  for (int i = 0; i < n; ++i) g.item[i] = item_of(W[i], x[i], y[i]);
  return type == MxType::kF16 ? launch_skinny<MxType::kF16, 1, 1, 8>(g, batch, stream)
                              : launch_skinny<MxType::kBF16, 1, 1, 8>(g, batch, stream);
}

int64_t mx_gemm_ws_bytes(const MxDesc &W, int64_t batch) {
  return batch < kMxTileBatch ? 0 : mx_gemm_tile_ws_bytes(W, batch);
}

hipError_t launch_mx_gemm(const MxDesc &W, const void *x, int64_t batch, void *y, MxType type,
                          void *ws, hipStream_t stream) {
  if (batch >= kMxTileBatch) return launch_mx_gemm_tile(W, x, batch, y, type, ws, stream);
  return type == MxType::kF16 ? gemm_as<MxType::kF16>(W, x, batch, y, stream)
                              : gemm_as<MxType::kBF16>(W, x, batch, y, stream);
}

}  // namespace aqlm
