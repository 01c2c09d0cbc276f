// Product of half activations with microscaled weights: y = x . W^T, for the
// batches of token generation. One or two rows of activations: mx_rows_kernel; up
// to 64: mx_skinny_kernel; where its tiles are faster, and above: the tile
// kernels of mx_gemm_tile.hip.
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

// Tiles of 16 rows of activations (up to four) and 16 rows of W, K shared by the
// NW wavefronts of a workgroup in groups of 512 inputs (16 blocks, 256 bytes of
// a row): lane (r, q) = (lane % 16, lane / 16) loads the 16 bytes that hold block
// 4 c + q of the group for c = 0 .. 3, and the group's 16 scale bytes of row r,
// and expands the codes into operands of v_mfma_f32_16x16x32: instruction s of
// chunk c multiplies codes 8 s .. 8 s + 7 of every block, so its activation
// operand is the 16 bytes of inputs 8 s of the same block of the lane's token.
// (The sum over K does not care which inputs meet in one instruction, so no
// code changes lanes.) Activations pass through LDS, which belongs to the
// wavefront alone: in whole lines to it, spread over the banks from it, a group
// of 512 inputs where there are up to 8 rows (H = 1), else half of it of 16 (H =
// 2), at a time. The wavefronts' float32 sums meet in LDS in a fixed order.
// What bounds it are requests, a 128-byte line each: scales byte by byte cost as
// many as the codes, activations read by each lane for itself more (4 rows: 4096 x
// 4096 5.7 us, 11008 x 4096 12.0), and codes loaded past the L1, which has the
// line's second half ready, double (5.1 and 8.9; this 4.5 and 7.8).
template <MxType T, int NW, int H>
__global__ __launch_bounds__(NW * 64, H == 1 ? 6 : 5) void mx_skinny_kernel(const Group g, const int all_tokens) {
  constexpr int kLoads = 8;                     // of x into LDS, at most
  constexpr int kChunkBits = H == 1 ? 6 : 5;    // of 64 / H chunks of 16 bytes of a token
  extern __shared__ __attribute__((aligned(16))) uint8_t xs[];  // [NW][loads][1 KiB]
  const int tok0 = 16 * (int)blockIdx.y, batch = min(16, all_tokens - tok0);
  const uint32_t mine = (threadIdx.x >> 6) * (uint32_t)((batch + H - 1) / H) * 1024u;  // the wavefront's
  int li = 0;
  while (li + 1 < g.n && (int)blockIdx.x >= g.first[li + 1]) ++li;
  const Group::Item &L = g.item[li];
  const int row0 = ((int)blockIdx.x - g.first[li]) * 16;
  const int rows = L.rows, cols = L.cols;
  const int nb = cols >> 5;
  const uint32_t half = (uint32_t)cols >> 1;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;

  // resources that end with the tile's last row: rows past it read zero (their
  // scales are those of the last one, and not stored results theirs)
  const int tile_rows = __builtin_amdgcn_readfirstlane(min(16, rows - row0));
  const Rsrc crs = make_rsrc(L.codes + (int64_t)row0 * half, (uint32_t)tile_rows * half);
  const Rsrc srs = make_rsrc(L.scales + (int64_t)row0 * nb, (uint32_t)tile_rows * nb);
  const Rsrc xrs = make_rsrc(L.x + (int64_t)tok0 * cols, (uint32_t)batch * cols * 2u);
  const uint32_t srow = (uint32_t)min(r16, tile_rows - 1) * nb;

  // Activations of blocks from..from + 16 / H - 1 into the wavefront's LDS: a load
  // takes 1 KiB, a token (two with H = 2), in whole lines. Chunk j of token t lies
  // at place j ^ t, which spreads the 16 tokens of a read over the banks: the lane
  // that fills a place reads the chunk that belongs there.
  const int lt = lane >> kChunkBits, lp = lane & ((1 << kChunkBits) - 1);
  auto fill = [&](int from) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i * H >= batch) break;
      const int t = i * H + lt, j = lp ^ (t & 15), blk = from + (j >> 2);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xrs, (__attribute__((address_space(3))) void *)(xs + (__builtin_amdgcn_readfirstlane(mine) + i * 1024)), 16,
          blk < nb && t < batch ? (uint32_t)t * cols * 2u + (uint32_t)from * 64u + 16u * j : kMxOOB, 0, 0, 0);
    }
  };
  // (tokens past the last read another's: their results are not stored)
  const int tok = min(r16, batch - 1);
  auto x_of = [&](int c, int s) __attribute__((always_inline)) {  // c: chunk of 128 inputs in LDS
    const int j = (4 * c + q) * 4 + s;
    return *reinterpret_cast<const uint4 *>(xs + (mine + tok * (1024 / H) + ((j ^ (tok & 15)) << 4)));
  };

  float4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int gr = wave; 16 * gr < nb; gr += NW) {
    uint4 w[4];
    fill(16 * gr);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int blk = 16 * gr + 4 * c + q;
      w[c] = buf_load16(crs, blk < nb ? (uint32_t)r16 * half + (uint32_t)blk * 16u : kMxOOB);
    }
    const uint4 sc = mx_scales16(srs, srow, 16 * gr, nb);
    const uint32_t sb[4] = {(sc.x >> (8 * q)) & 0xFFu, (sc.y >> (8 * q)) & 0xFFu, (sc.z >> (8 * q)) & 0xFFu,
                            (sc.w >> (8 * q)) & 0xFFu};
    bool fits = true;
    if constexpr (T == MxType::kF16)
      fits = __all(mx_fits_f16(sb[0]) && mx_fits_f16(sb[1]) && mx_fits_f16(sb[2]) && mx_fits_f16(sb[3]));
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    auto products = [&](int c) __attribute__((always_inline)) {
      const uint32_t ww[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
      const float sv = mx_scale(sb[c]);
#pragma unroll
      for (int s = 0; s < 4; ++s) acc = mx_mfma16<T>(mx_decode8<T>(ww[s], sv), x_of(c % (4 / H), s), acc);
    };
    // scales that float16 weights cannot take: the same product in bfloat16,
    // which holds every weight, with x split exactly in two
    auto wide_products = [&](int c) __attribute__((always_inline)) {
      const uint32_t ww[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
      const float sv = mx_scale(sb[c]);
#pragma unroll 1
      for (int s = 0; s < 4; ++s) {
        uint4 hi, lo;
        split_f16(x_of(c % (4 / H), s), hi, lo);
        const uint4 a = mx_decode8<MxType::kBF16>(s == 0 ? ww[0] : s == 1 ? ww[1] : s == 2 ? ww[2] : ww[3], sv);
        acc = mx_mfma16<MxType::kBF16>(a, hi, acc);
        acc = mx_mfma16<MxType::kBF16>(finite_bf16(a), lo, acc);
      }
    };
#pragma unroll
    for (int part = 0; part < H; ++part) {
      if (part > 0) {
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        fill(16 * gr + 8);
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
      }
      if (fits) {
#pragma unroll
        for (int c = 0; c < 4 / H; ++c) products(part * (4 / H) + c);
      } else {
#pragma unroll
        for (int c = 0; c < 4 / H; ++c) wide_products(part * (4 / H) + c);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");  // (before x is overwritten)
  }

  __syncthreads();
  float4_t *const red = reinterpret_cast<float4_t *>(xs);  // (1 KiB a wavefront)
  red[threadIdx.x] = acc;
  __syncthreads();
  // lane (t, q) holds rows 4 q .. 4 q + 3 of token t
  if (threadIdx.x < 64) {
    float4_t v = red[lane];
#pragma unroll
    for (int u = 1; u < NW; ++u) v += red[u * 64 + lane];
    if (r16 < batch) store4<T>(L.y + (int64_t)(tok0 + r16) * rows, row0 + 4 * q, rows, v, (rows & 3) == 0);
  }
}

template <MxType T, int NW, int H> hipError_t launch_skinny(Group &g, int batch, hipStream_t stream) {
  int blocks = 0;
  for (int i = 0; i < g.n; ++i) {
    g.first[i] = blocks;
    blocks += (g.item[i].rows + 15) / 16;
  }
  g.first[g.n] = blocks;
  hipLaunchKernelGGL((mx_skinny_kernel<T, NW, H>), dim3((unsigned)blocks, (unsigned)(batch + 15) / 16), dim3(NW * 64),
                     NW * 1024 * ((std::min(batch, 16) + H - 1) / H), stream, g, batch);
  return hipGetLastError();
}

// One or two rows of activations (B): the weights' bytes bound the product, so a wavefront
// reads whole rows, R at a time, 1 KiB of codes (64 blocks of 32, a block a
// lane) and their 64 scale bytes each (28672 x 8192 25.7 us, 4.9 TB/s; with
// workgroups of four wavefronts instead of eight, four rows each, 27; in 16-row
// tiles whose wavefronts read 64-byte pieces of rows 42).
//   * x lies in LDS, up to kSegment inputs of it at a time (of both rows), read by all wavefronts of the
//     workgroup; a lane takes the 64 bytes of its own block for every row.
//   * v_mfma_f32_16x16x32 sums over the lanes as well: lane (m, q) = (lane % 16,
//     lane / 16) gives eight codes of its block and eight inputs of the same
//     block, so that the result's diagonal (m, m) holds the sums of the four
//     lanes m, 16 + m, ..; the rest of the result is of no use, and the
//     instruction still outruns the loads (64 bytes of codes a clock and CU).
//     The 16 diagonal places are added at the end of a row.
// Chunks of x are permuted (x_place), so that the 16 lanes of an LDS pass touch
// 16 distinct groups of banks.
constexpr int kRowThreads = 512;
constexpr int kSegment = 16384;  // inputs in LDS
__device__ __forceinline__ uint32_t x_place(int blk, int s) {
  return (uint32_t)blk * 64u + (uint32_t)((s ^ ((blk >> 2) & 3)) << 4);
}

template <MxType T, int R, int B>
__global__ __launch_bounds__(kRowThreads) void mx_rows_kernel(const Group g, const int batch) {
  constexpr int kBlocks = kSegment / 32 / B, kChunks = kBlocks / 64;
  __shared__ __attribute__((aligned(16))) uint8_t xs[kSegment * 2];  // [B][kBlocks][64 bytes]
  int li = 0;
  while (li + 1 < g.n && (int)blockIdx.x >= g.first[li + 1]) ++li;
  const Group::Item &L = g.item[li];
  const int rows = L.rows, nb = L.cols >> 5;
  const uint32_t half = (uint32_t)L.cols >> 1;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row0 = (((int)blockIdx.x - g.first[li]) * (kRowThreads / 64) + wave) * R;
  // resources that end with the wavefront's last row: rows past it read zero
  const int mine = __builtin_amdgcn_readfirstlane(max(0, min(R, rows - row0)));
  const Rsrc crs = make_rsrc(L.codes + (int64_t)(mine ? row0 : 0) * half, (uint32_t)mine * half);
  const Rsrc srs = make_rsrc(L.scales + (int64_t)(mine ? row0 : 0) * nb, (uint32_t)mine * nb);

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
  auto compute = [&](int c, const uint4 (&wv)[R], const uint32_t (&sv)[R]) __attribute__((always_inline)) {
    const int lb = (c % kChunks) * 64 + lane;  // block of the segment
    // (by row, so that a row's sums do not depend on its neighbours)
    bool fits[R], all = true;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      fits[r] = T != MxType::kF16 || r >= mine || __ballot((sv[r] - 104u > 36u) & (64 * c + lane < nb)) == 0;
      all = all & fits[r];
    }
    if (all) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint4 x[B];
#pragma unroll
        for (int b = 0; b < B; ++b) x[b] = *reinterpret_cast<const uint4 *>(xs + (b * kBlocks * 64 + x_place(lb, s)));
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint32_t ww[4] = {wv[r].x, wv[r].y, wv[r].z, wv[r].w};
          const uint4 a = mx_decode8<T>(ww[s], mx_scale(sv[r]));
#pragma unroll
          for (int b = 0; b < B; ++b) acc[r][b] = mx_mfma16<T>(a, x[b], acc[r][b]);
        }
      }
    } else {
      // scales that float16 weights cannot take: the same product in bfloat16,
      // which holds every weight, with x split exactly in two
#pragma unroll 1
      for (int s = 0; s < 4; ++s) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const uint4 x = *reinterpret_cast<const uint4 *>(xs + (b * kBlocks * 64 + x_place(lb, s)));
          uint4 hi, lo;
          split_f16(x, hi, lo);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint32_t w = s == 0 ? wv[r].x : s == 1 ? wv[r].y : s == 2 ? wv[r].z : wv[r].w;
            if (fits[r]) {
              acc[r][b] = mx_mfma16<T>(mx_decode8<T>(w, mx_scale(sv[r])), x, acc[r][b]);
            } else {
              const uint4 a = mx_decode8<MxType::kBF16>(w, mx_scale(sv[r]));
              acc[r][b] = mx_mfma16<MxType::kBF16>(a, hi, acc[r][b]);
              acc[r][b] = mx_mfma16<MxType::kBF16>(finite_bf16(a), lo, acc[r][b]);
            }
          }
        }
      }
    }
  };

  const int chunks = (nb + 63) >> 6;
  load(0, w[0], sb[0]);
  for (int c0 = 0; c0 < chunks; c0 += kChunks) {  // a segment of x
    if (c0 > 0) __syncthreads();
    const int blocks = min(kBlocks, ((nb - 64 * c0 + 63) >> 6) << 6);  // whole chunks of it
#pragma unroll
    for (int b = 0; b < B; ++b)
      for (int k = threadIdx.x; k < blocks * 4; k += kRowThreads) {
        const int blk = 64 * c0 + (k >> 2);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (blk < nb && b < batch)
          v = *reinterpret_cast<const uint4 *>(L.x + ((int64_t)b * L.cols + blk * 32 + 8 * (k & 3)));
        *reinterpret_cast<uint4 *>(xs + (b * kBlocks * 64 + x_place(k >> 2, k & 3))) = v;
      }
    __syncthreads();
    const int c1 = min(chunks, c0 + kChunks);
    for (int c = c0; c < c1; ++c) {
      load(c + 1, w[1], sb[1]);
      compute(c, w[0], sb[0]);
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
      if (lane == 63 && r < mine && b < batch) L.y[(int64_t)b * rows + row0 + r] = (uint16_t)f2t<T>(sum);
    }
}

template <MxType T, int R, int B> hipError_t launch_rows(Group &g, int batch, hipStream_t stream) {
  constexpr int kRows = R * (kRowThreads / 64);
  int blocks = 0;
  for (int i = 0; i < g.n; ++i) {
    g.first[i] = blocks;
    blocks += (g.item[i].rows + kRows - 1) / kRows;
  }
  g.first[g.n] = blocks;
  hipLaunchKernelGGL((mx_rows_kernel<T, R, B>), dim3((unsigned)blocks), dim3(kRowThreads), 0, stream, g, batch);
  return hipGetLastError();
}

// Rows of W a wavefront reads at a time: one while all its workgroups find room
// at once (four of them a CU) and x one segment, else two, which keep more bytes
// under way (one, two rows: 4096 x 4096 4.0, 4.1 us, 8192 x 8192 8.2, 9.2; 11008 x
// 4096 7.4, 6.5, three of 4096 x 4096 at once 8.3, 7.3, 8192 x 28672 24.6, 23.1).
template <MxType T, int B> hipError_t rows_as(Group &g, int batch, hipStream_t stream) {
  int64_t rows = 0;
  int cols = 0;
  for (int i = 0; i < g.n; ++i) {
    rows += g.item[i].rows;
    cols = std::max(cols, g.item[i].cols);
  }
  return rows <= 1024 * (kRowThreads / 64) && cols <= kSegment ? launch_rows<T, 1, B>(g, batch, stream)
                                                               : launch_rows<T, 2, B>(g, batch, stream);
}

Group::Item item_of(const MxDesc &W, const void *x, void *y) {
  return {W.codes, W.scales, static_cast<const uint16_t *>(x), static_cast<uint16_t *>(y),
          (int)W.rows, (int)W.cols};
}

constexpr int kSkinnyWaves = 8;

// From three rows on, where the tile kernel is the faster: the skinny one takes
// 0.84 ns and 0.046 ns a row of activations for 16 rows of W and a group of K,
// spread over the chip, or, with few rows of W, 1.15 us and 0.07 us a row for each
// turn of its wavefronts (fitted to 1024 x 8192 .. 28672 x 8192 from 3 to 64 rows:
// 4096 x 4096 at 8 rows 4.7 us against 9.6, at 32 8.1 against 9.2, 1024 x 8192 at 64
// 8.1 against 10.2, 28672 x 8192 at 8 38 against 34).
// Whole-row wavefronts serve two rows of activations better than either (4096 x
// 4096 3.9 us against 4.5, 11008 x 4096 7.9 against 10.8, 28672 x 8192 33 against
// 34, 8192 x 28672 30 against 41), three about as well, four and more worse.
// `split`: K may be split over workgroups.
bool tiles_pay(const MxDesc &W, int64_t batch, bool split) {
  if (batch > 64) return true;
  if (batch <= 2) return false;
  const double groups = (double)((W.cols / 32 + 15) / 16), tiles = (double)((W.rows + 15) / 16);
  const double turns = (double)(int64_t)((groups + kSkinnyWaves - 1) / kSkinnyWaves);
  const double more = (double)((batch - 1) / 16);  // times that W is read again, from the caches
  const double us = 2.7 + std::max(tiles * groups * (0.84e-3 * (1 + 0.5 * more) + 0.046e-3 * (double)batch),
                                   turns * (1.15 + 0.07 * (double)std::min<int64_t>(batch, 16)));
  return mx_gemm_tile_us(W, batch, split) < us;
}

// Without the tile kernel.
template <MxType T> hipError_t few_as(Group &g, int batch, hipStream_t stream) {
  if (batch == 1) return rows_as<T, 1>(g, batch, stream);
  if (batch == 2) return rows_as<T, 2>(g, batch, stream);
  if (batch <= 8) return launch_skinny<T, kSkinnyWaves, 1>(g, batch, stream);
  return launch_skinny<T, kSkinnyWaves, 2>(g, batch, stream);
}

hipError_t launch_few(Group &g, int batch, MxType type, hipStream_t stream) {
  if (g.n == 0) return hipSuccess;
  return type == MxType::kF16 ? few_as<MxType::kF16>(g, batch, stream) : few_as<MxType::kBF16>(g, batch, stream);
}

}  // namespace

hipError_t launch_mx_gemv_batched(const MxDesc *W, const void *const *x, void *const *y, int n,
                                  int batch, MxType type, hipStream_t stream) {
  Group g;
  g.n = 0;
  for (int i = 0; i < n; ++i) {
    if (tiles_pay(W[i], batch, false)) {
      const hipError_t e = launch_mx_gemm_tile(W[i], x[i], batch, y[i], type, false, nullptr, stream);
      if (e != hipSuccess) return e;
    } else {
      g.item[g.n++] = item_of(W[i], x[i], y[i]);
    }
  }
  return launch_few(g, batch, type, stream);
}

int64_t mx_gemm_ws_bytes(const MxDesc &W, int64_t batch) {
  return tiles_pay(W, batch, true) ? mx_gemm_tile_ws_bytes(W, batch) : 0;
}

hipError_t launch_mx_gemm(const MxDesc &W, const void *x, int64_t batch, void *y, MxType type,
                          void *ws, hipStream_t stream) {
  if (tiles_pay(W, batch, true)) return launch_mx_gemm_tile(W, x, batch, y, type, true, ws, stream);
  Group g;
  g.n = 1;
  g.item[0] = item_of(W, x, y);
  return launch_few(g, (int)batch, type, stream);
}

}  // namespace aqlm
