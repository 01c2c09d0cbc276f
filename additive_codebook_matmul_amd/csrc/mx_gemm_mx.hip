// Product of two microscaled matrices for few rows of activations: y = x .
// W^T on the block-scaled matrix instructions, which take E2M1 codes and E8M0
// scales as they are. (Larger tiles, and more rows: mx_gemm_mx_tile.hip.)
//
// mx_mx_skinny_kernel: v_mfma_scale_f32_16x16x128_f8f6f4 with 4-bit operands: lane (r, q) = (lane %
// 16, lane / 16) gives the 16 bytes of block q (32 codes) of row r of the
// 128-input chunk and that block's scale byte, for A (rows of W) and B (rows
// of x) alike, so both sides are loaded straight from their row-major arrays.
// The wavefronts of a workgroup share K in groups of 512 inputs, four chunks
// with 16 scale bytes of a row, for NT tiles of 16 rows of x, and add their
// float32 sums through LDS in a fixed order.
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

template <MxType T, int NW, int NT>
__global__ __launch_bounds__(NW * 64) void mx_mx_skinny_kernel(
    const uint8_t *__restrict__ wc, const uint8_t *__restrict__ wsc,
    const uint8_t *__restrict__ xc, const uint8_t *__restrict__ xsc, uint16_t *__restrict__ y,
    const int rows, const int cols, const int all_tokens) {
  const int tok0 = 16 * NT * (int)blockIdx.y, batch = min(16 * NT, all_tokens - tok0);
  __shared__ __attribute__((aligned(16))) float4_t red[NT][NW * 64];
  const int row0 = (int)blockIdx.x * 16;
  const int nb = cols >> 5;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  // resources that end with the tile's last row: rows past it read zero (their
  // scales are those of the last one)
  const int tile_rows = __builtin_amdgcn_readfirstlane(min(16, rows - row0));
  const uint32_t half = (uint32_t)cols >> 1;
  const Rsrc crs = make_rsrc(wc + (int64_t)row0 * half, (uint32_t)tile_rows * half);
  const Rsrc srs = make_rsrc(wsc + (int64_t)row0 * nb, (uint32_t)tile_rows * nb);
  const Rsrc xrs = make_rsrc(xc + (int64_t)tok0 * half, (uint32_t)batch * half);
  const Rsrc xss = make_rsrc(xsc + (int64_t)tok0 * nb, (uint32_t)batch * nb);
  const uint32_t srow = (uint32_t)min(r16, tile_rows - 1) * nb;

  float4_t acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = float4_t{0.f, 0.f, 0.f, 0.f};
  for (int gr = wave; 16 * gr < nb; gr += NW) {
    uint4 w[4], x[NT][4], sx[NT];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int blk = 16 * gr + 4 * c + q;
      w[c] = buf_load16(crs, blk < nb ? (uint32_t)r16 * half + (uint32_t)blk * 16u : kMxOOB);
    }
    const uint4 sw = mx_scales16(srs, srow, 16 * gr, nb);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int blk = 16 * gr + 4 * c + q;
        x[j][c] = buf_load16(xrs, blk < nb ? (uint32_t)(16 * j + r16) * half + (uint32_t)blk * 16u : kMxOOB);
      }
      sx[j] = mx_scales16(xss, (uint32_t)min(16 * j + r16, batch - 1) * nb, 16 * gr, nb);
    }
    const uint32_t swv[4] = {sw.x, sw.y, sw.z, sw.w};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint32_t sxv[4] = {sx[j].x, sx[j].y, sx[j].z, sx[j].w};
#pragma unroll
      for (int c = 0; c < 4; ++c)
        acc[j] = mfma_mx16(w[c], swv[c] >> (8 * q), x[j][c], sxv[c] >> (8 * q), acc[j]);
    }
  }

#pragma unroll
  for (int j = 0; j < NT; ++j) red[j][threadIdx.x] = acc[j];
  __syncthreads();
  // lane (t, q) holds rows 4 q .. 4 q + 3 of token t; wavefront j adds up tile j
  if (threadIdx.x < 64 * NT) {
    float4_t v = red[wave][lane];
#pragma unroll
    for (int u = 1; u < NW; ++u) v += red[wave][u * 64 + lane];
    const int tok = 16 * wave + r16;
    if (tok < batch) store4<T>(y + (int64_t)(tok0 + tok) * rows, row0 + 4 * q, rows, v, (rows & 3) == 0);
  }
}

template <MxType T, int NW, int NT>
hipError_t launch_skinny(const MxDesc &W, const MxDesc &x, void *y, hipStream_t stream) {
  const dim3 grid((unsigned)((W.rows + 15) / 16), (unsigned)((x.rows + 16 * NT - 1) / (16 * NT)));
  hipLaunchKernelGGL((mx_mx_skinny_kernel<T, NW, NT>), grid, dim3(NW * 64), 0, stream, W.codes, W.scales,
                     x.codes, x.scales, static_cast<uint16_t *>(y), (int)W.rows, (int)W.cols, (int)x.rows);
  return hipGetLastError();
}

// Up to five rows of activations (B): whole rows of W by a wavefront,
// R at a time, as for half activations (mx_rows_kernel; 28672 x 8192 at one row
// 23.2 us, 5.4 TB/s): lane (m, q) = (lane % 16, lane / 16) gives its own block of W's
// row and the same block of x, so that the result's diagonal (m, m) holds the sums
// of the four lanes of m, and one instruction takes 1 KiB of codes. x lies in LDS,
// codes and scale bytes, 2048 / B blocks of each row at a time.
// Q: x is given quantised (kGiven), or is halves that every workgroup quantises on
// their way into LDS, as mx_quantize_kernel does (four lanes a block).
enum MxInput { kGiven, kFloor, kCeil };

constexpr int kRowThreads = 512;
constexpr int kWaveRows = 2;    // R
constexpr int kXBlocks = 2048;  // blocks in LDS

template <MxType T, int B, int Q>
__global__ __launch_bounds__(kRowThreads) void mx_mx_rows_kernel(
    const uint8_t *__restrict__ wc, const uint8_t *__restrict__ wsc, const void *__restrict__ x,
    const uint8_t *__restrict__ xsc, uint16_t *__restrict__ y, const int rows, const int cols, const int batch) {
  constexpr int R = kWaveRows, kBlocks = kXBlocks / B / 64 * 64, kChunks = kBlocks / 64;
  __shared__ __attribute__((aligned(16))) uint8_t xs[kXBlocks * 16];  // [B][kBlocks][16 bytes]
  __shared__ uint8_t ss[kXBlocks];                                    // [B][kBlocks]
  const int nb = cols >> 5;
  const uint32_t half = (uint32_t)cols >> 1;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row0 = ((int)blockIdx.x * (kRowThreads / 64) + wave) * R;
  // resources that end with the wavefront's last row: rows past it read zero
  const int mine = __builtin_amdgcn_readfirstlane(max(0, min(R, rows - row0)));
  const Rsrc crs = make_rsrc(wc + (int64_t)(mine ? row0 : 0) * half, (uint32_t)mine * half);
  const Rsrc srs = make_rsrc(wsc + (int64_t)(mine ? row0 : 0) * nb, (uint32_t)mine * nb);
  const Rsrc xrs = make_rsrc(x, (uint32_t)batch * cols * 2u / (Q == kGiven ? 4u : 1u));
  const Rsrc xss = make_rsrc(Q == kGiven ? xsc : wsc, (uint32_t)batch * nb);

  float4_t acc[R][B];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int b = 0; b < B; ++b) acc[r][b] = float4_t{0.f, 0.f, 0.f, 0.f};
  uint4 w[2][R];
  uint32_t sb[2][R];
  auto load = [&](int c, uint4 (&wv)[R], uint32_t (&sv)[R]) __attribute__((always_inline)) {
    const int blk = 64 * c + lane;
    const bool in = blk < nb;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      wv[r] = buf_load16_nt(crs, in ? (uint32_t)r * half + (uint32_t)blk * 16u : kMxOOB);
      sv[r] = buf_load_u8(srs, in ? (uint32_t)r * nb + (uint32_t)blk : kMxOOB);
    }
  };
  const int chunks = (nb + 63) >> 6;
  load(0, w[0], sb[0]);
  for (int c0 = 0; c0 < chunks; c0 += kChunks) {  // a segment of x
    if (c0 > 0) __syncthreads();
    const int blocks = min(kBlocks, ((nb - 64 * c0 + 63) >> 6) << 6);  // whole chunks of it
    if constexpr (Q == kGiven) {
      for (int k = threadIdx.x; k < blocks; k += kRowThreads) {
        const int blk = 64 * c0 + k;
        uint4 v[B];
        uint32_t s[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const bool in = (blk < nb) & (b < batch);
          v[b] = buf_load16(xrs, in ? (uint32_t)b * half + (uint32_t)blk * 16u : kMxOOB);
          s[b] = buf_load_u8(xss, in ? (uint32_t)b * nb + (uint32_t)blk : kMxOOB);
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          *reinterpret_cast<uint4 *>(xs + (b * kBlocks + k) * 16) = v[b];
          ss[b * kBlocks + k] = (uint8_t)s[b];
        }
      }
    } else {
      for (int k = threadIdx.x; k < 4 * blocks; k += kRowThreads) {  // (whole wavefronts)
        const int oct = 256 * c0 + k;
        Octet<T> o[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const uint4 v = buf_load16(
              xrs, oct < 4 * nb && b < batch ? (uint32_t)b * cols * 2u + 16u * (uint32_t)oct : kMxOOB);
          o[b].w[0] = v.x;
          o[b].w[1] = v.y;
          o[b].w[2] = v.z;
          o[b].w[3] = v.w;
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const uint32_t s = scale_byte<Q == kCeil>(block_max<T>(o[b]));
          *reinterpret_cast<uint32_t *>(xs + b * (kBlocks * 16) + 4 * k) =
              s == 255u ? 0u : encode8<T>(o[b], mx_scale(s));
          if ((k & 3) == 0) ss[b * kBlocks + (k >> 2)] = (uint8_t)s;
        }
      }
    }
    __syncthreads();
    const int c1 = min(chunks, c0 + kChunks);
    for (int c = c0; c < c1; ++c) {
      load(c + 1, w[1], sb[1]);
      const int lb = (c - c0) * 64 + lane;  // block of the segment
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const uint4 xv = *reinterpret_cast<const uint4 *>(xs + (b * kBlocks + lb) * 16);
        const uint32_t sx = ss[b * kBlocks + lb];
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][b] = mfma_mx16(w[0][r], sb[0][r], xv, sx, acc[r][b]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        w[0][r] = w[1][r];
        sb[0][r] = sb[1][r];
      }
    }
  }

  // the diagonal: place (m, m) is register m % 4 of lane 16 (m / 4) + m
  const bool diagonal = ((lane >> 2) & 3) == (lane >> 4);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const float4_t a = acc[r][b];
      const float v = (lane & 2) ? ((lane & 1) ? a[3] : a[2]) : ((lane & 1) ? a[1] : a[0]);
      const float sum = wave_sum_to_lane63(diagonal ? v : 0.0f);
      if (lane == 63 && r < mine && b < batch) y[(int64_t)b * rows + row0 + r] = (uint16_t)f2t<T>(sum);
    }
}

template <MxType T, int B, int Q>
void launch_rows(const MxDesc &W, const void *x, const uint8_t *xsc, int batch, void *y, hipStream_t stream) {
  constexpr int kRows = kWaveRows * (kRowThreads / 64);
  hipLaunchKernelGGL((mx_mx_rows_kernel<T, B, Q>), dim3((unsigned)((W.rows + kRows - 1) / kRows)),
                     dim3(kRowThreads), 0, stream, W.codes, W.scales, x, xsc, static_cast<uint16_t *>(y),
                     (int)W.rows, (int)W.cols, batch);
}

template <MxType T, int Q>
hipError_t rows_as(const MxDesc &W, const void *x, const uint8_t *xsc, int batch, void *y, hipStream_t stream) {
  if (batch == 1) launch_rows<T, 1, Q>(W, x, xsc, batch, y, stream);
  else if (batch == 2) launch_rows<T, 2, Q>(W, x, xsc, batch, y, stream);
  else if (batch == 3) launch_rows<T, 3, Q>(W, x, xsc, batch, y, stream);
  else if (batch == 4) launch_rows<T, 4, Q>(W, x, xsc, batch, y, stream);
  else launch_rows<T, 5, Q>(W, x, xsc, batch, y, stream);
  return hipGetLastError();
}

// Where whole-row wavefronts are the faster: one or two rows of activations
// (against the better of the other two kernels, 4096 x 4096 2.7 us, 3.6, 28672 x
// 8192 23.3, 27.0), up to four where W has many rows, up to five where they are
// long (four rows: 11008 x 4096 6.8, 7.4, 4096 x 4096 4.4, 3.7; five: 8192 x 28672
// 24.5, 29.4, 11008 x 4096 8.2, 7.7).
bool rows_pay(const MxDesc &W, int64_t batch) {
  return batch <= (W.cols > 16384 ? 5 : W.rows > 4096 ? 4 : 2);
}

// Whether they also quantise x, every workgroup again, rather than a launch of its
// own, which takes 2 us: up to five rows and about 480 million steps of K in all
// rows and tokens (one row: 4096 x 4096 2.9, 4.5 us; five rows of 4096 x 4096 5.4,
// 5.8; three of 28672 x 8192 27.3, 26.6, five of them 34.4, 29.8).
bool quant_pays(const MxDesc &W, int64_t batch) {
  return batch <= 5 && W.rows * W.cols * batch <= (int64_t)480 << 20;
}

constexpr int kSkinnyWaves = 8;

// Of the others, where the tile kernel is the faster: the skinny one takes 0.82 ns
// and 0.022 ns a row of activations for 16 rows of W and a group of K, spread over
// the chip, or, with few rows of W, 1 us and 0.05 us a row for each turn of its
// wavefronts (fitted to 1024 x 8192 .. 28672 x 8192 from 2 to 128 rows: 4096 x 4096
// at 5 3.8 us against 6.6, at 32 5.8 against 7.2, 1024 x 4096 at 64 5.5 against 6.7,
// 28672 x 8192 at 16 36.5 against 27.8).
bool tiles_pay(const MxDesc &W, int64_t batch) {
  if (batch > 128) return true;
  const double groups = (double)((W.cols / 32 + 15) / 16), tiles = (double)((W.rows + 15) / 16);
  const double turns = (double)(int64_t)((groups + kSkinnyWaves - 1) / kSkinnyWaves);
  const double more = (double)((batch - 1) / 32);  // times that W is read again, from the caches
  const double us = 2.7 + 0.5 * more +
                    std::max(tiles * groups * (0.82e-3 * (1 + 0.5 * more) + 0.022e-3 * (double)batch),
                             turns * (1.0 + 0.05 * (double)std::min<int64_t>(batch, 32)));
  return mx_gemm_mx_tile_us(W, batch) < us;
}

// Workspace of quantisation and product: codes, scales, the product's own, each
// from a multiple of 256 bytes on.
int64_t ws_scales_at(const MxDesc &W, int64_t batch) { return (batch * (W.cols / 2) + 255) / 256 * 256; }
int64_t ws_product_at(const MxDesc &W, int64_t batch) {
  return ws_scales_at(W, batch) + (batch * (W.cols / 32) + 255) / 256 * 256;
}

}  // namespace

int64_t mx_gemm_quant_ws_bytes(const MxDesc &W, int64_t batch) {
  return quant_pays(W, batch) ? 0 : ws_product_at(W, batch) + mx_gemm_mx_ws_bytes(W, batch);
}

hipError_t launch_mx_gemm_quant(const MxDesc &W, const void *x, int64_t batch, bool ceil_rule, void *y, MxType type,
                                void *ws, hipStream_t stream) {
  if (quant_pays(W, batch)) {
    if (type == MxType::kF16)
      return ceil_rule ? rows_as<MxType::kF16, kCeil>(W, x, nullptr, (int)batch, y, stream)
                       : rows_as<MxType::kF16, kFloor>(W, x, nullptr, (int)batch, y, stream);
    return ceil_rule ? rows_as<MxType::kBF16, kCeil>(W, x, nullptr, (int)batch, y, stream)
                     : rows_as<MxType::kBF16, kFloor>(W, x, nullptr, (int)batch, y, stream);
  }
  uint8_t *const at = static_cast<uint8_t *>(ws);
  uint8_t *const scales = at + ws_scales_at(W, batch);
  const hipError_t e = launch_mx_quantize(x, type, batch, W.cols, ceil_rule, at, scales, stream);
  if (e != hipSuccess) return e;
  return launch_mx_gemm_mx(W, {batch, W.cols, at, scales}, y, type, at + ws_product_at(W, batch), stream);
}

int64_t mx_gemm_mx_ws_bytes(const MxDesc &W, int64_t batch) {
  return !rows_pay(W, batch) && tiles_pay(W, batch) ? mx_gemm_mx_tile_ws_bytes(W, batch) : 0;
}

hipError_t launch_mx_gemm_mx(const MxDesc &W, const MxDesc &x, void *y, MxType type, void *ws,
                             hipStream_t stream) {
  if (rows_pay(W, x.rows))
    return type == MxType::kF16 ? rows_as<MxType::kF16, kGiven>(W, x.codes, x.scales, (int)x.rows, y, stream)
                                : rows_as<MxType::kBF16, kGiven>(W, x.codes, x.scales, (int)x.rows, y, stream);
  if (tiles_pay(W, x.rows)) return launch_mx_gemm_mx_tile(W, x, y, type, ws, stream);
  if (x.rows > 16)
    return type == MxType::kF16 ? launch_skinny<MxType::kF16, kSkinnyWaves, 2>(W, x, y, stream)
                                : launch_skinny<MxType::kBF16, kSkinnyWaves, 2>(W, x, y, stream);
  return type == MxType::kF16 ? launch_skinny<MxType::kF16, kSkinnyWaves, 1>(W, x, y, stream)
                              : launch_skinny<MxType::kBF16, kSkinnyWaves, 1>(W, x, y, stream);
}

}  // namespace aqlm
