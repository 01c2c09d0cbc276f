// Product of two microscaled matrices for many rows of activations, one
// workgroup per [rows of W] x [tokens] tile (mx_tile.hpp).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 with 4-bit operands: lane (r, h) = (lane %
// 32, lane / 32) gives the 16 bytes of block h (32 codes) of row r of the
// 64-input chunk and, in a byte of a register, that block's scale; W and x
// alike, and both as they lie in memory.
//   * A K step is 256 inputs, four such chunks: 128-byte rows, whole lines of
//     L2 (in 64-byte rows, or with scales loaded by each lane for its own row,
//     the requests cost as much again). Both sides go from memory straight to
//     LDS two steps ahead, into one of three stages; 16-byte chunk c of row r
//     lies at chunk c ^ ((r >> 1) & 7), so that the 16 lanes of an LDS pass touch
//     16 distinct groups of banks.
//   * Scales go through LDS kTurns groups, 32 blocks, at a time; a lane's for
//     two steps are four words of its row. Shifted by 8 h, bytes 0 and 2 of a
//     word are those of two chunks, which the instruction selects.
//   * A 32 x 32 x 64 product takes a SIMD as long as 32 x 32 x 16 of halves,
//     with the same two operand reads of 1 KiB, for four times the sum.
// What bounds it is waiting: at 1999 x 4096 x 11008 (52 to 55 us) the matrix
// cores are busy for 36 % of the time, LDS for 22 % and L2 gives 13 of its 30 TB/s.
// A step begins behind its barrier with reads and has no product to issue until
// they return.
#include <algorithm>

#include "mx_tile.hpp"

namespace aqlm {
namespace {

// Byte offset of block c (of 8) of row r in its part of a stage.
__device__ __forceinline__ uint32_t row_off(int r, int c) {
  return (uint32_t)r * 128u + (uint32_t)((c ^ ((r >> 1) & 7)) << 4);
}

constexpr int kTurns = 2;  // groups whose scales LDS holds

template <int S>
__device__ __forceinline__ float16_t mfma_mx32(const uint4 &a, uint32_t sa, const uint4 &b, uint32_t sb,
                                               float16_t c) {
  const int8_vt av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const int8_vt bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, S, (int)sa, S, (int)sb);
}

template <MxType T, int RT, int NT, int TW, int KW>
__global__ __launch_bounds__(64 * kRowWaves * TW * KW) void mx_mx_tile_kernel(const TileArgs A) {
  constexpr int kWaves = kRowWaves * TW;  // of one share of K
  constexpr int kRows = kRowWaves * RT * 32, kToks = TW * NT * 32;
  constexpr int kWBytes = kRows * 128, kXBytes = kToks * 128;
  constexpr int kStage = kWBytes + kXBytes;
  typedef ScaleStage<kRows, 64 * kWaves, kTurns> WScales;
  typedef ScaleStage<kToks, 64 * kWaves, kTurns> XScales;
  constexpr int kScales = WScales::kBytes + XScales::kBytes;
  constexpr int kSums = tile_sums_bytes<RT, NT, TW>();  // two quarters of a share's sums an array
  static_assert(kStage >= kWaves * kStoreBytes<RT>, "room for the results");
  constexpr int kArray = KW == 1 || KW * kStage > 2 * kSums ? KW * kStage : 2 * kSums;
  // one array per stage: the compiler then knows which loads into LDS a read
  // of LDS can depend on
  __shared__ __attribute__((aligned(16))) uint8_t xa0[kArray], xa1[kArray], xa2[kArray];
  __shared__ __attribute__((aligned(16))) uint8_t sa[KW * kScales];
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = KW == 1 ? 0 : wave_all / kWaves, wave = KW == 1 ? wave_all : wave_all % kWaves;
  const int rw = wave / TW, tw = wave % TW;
  const int l32 = lane & 31, h = lane >> 5;
  const int tiles = A.row_tiles * A.tok_tiles;
  const int job = xcd_job((int)blockIdx.x, tiles * A.splits);
  const int split = __builtin_amdgcn_readfirstlane(job / tiles);
  const TilePlace at = tile_place(job - split * tiles, A.row_tiles, A.tok_tiles);
  const int row0 = at.row_tile * (kRowWaves * 32 * RT), tok0 = at.tok_tile * (32 * NT * TW);
  const int nb = A.cols >> 5;

  // K goes in groups of two steps, 16 blocks. The groups of this split, and
  // of those the wavefront's: each of the KW shares takes as many turns as the
  // largest (past its end with zeros), so that all meet at every barrier.
  const int s0 = split * A.groups_per_split, s1 = min((nb + 15) >> 4, s0 + A.groups_per_split);
  const int share = (s1 - s0 + KW - 1) / KW;
  const int g0 = s0 + kw * share, g1 = min(s1, g0 + share), gend = g0 + share;

  // resources that end with the tile's last row: rows past it read zero
  const uint32_t half = (uint32_t)A.cols >> 1;
  const int tile_rows = __builtin_amdgcn_readfirstlane(min(kRowWaves * 32 * RT, A.rows - row0));
  const int tile_toks = __builtin_amdgcn_readfirstlane(min(32 * NT * TW, A.batch - tok0));
  const Rsrc crs = make_rsrc(A.codes + (int64_t)row0 * half, (uint32_t)tile_rows * half);
  const Rsrc xrs = make_rsrc(static_cast<const uint8_t *>(A.x) + (int64_t)tok0 * half,
                             (uint32_t)tile_toks * half);

  float16_t acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // Step t (of group t / 2) into a stage. One load of a wavefront fills 1 KiB,
  // eight rows, in lane order, so a chunk's place in its row is chosen by where
  // the lane reads from. Blocks past the last one are zeros. Wavefront w of the
  // share makes loads w, w + kWaves, .. of each side.
  constexpr int kWLoads = 16 * RT / kWaves, kXLoads = 4 * NT * TW / kWaves;
  static_assert(16 * RT % kWaves == 0 && 4 * NT * TW % kWaves == 0, "as many loads a wavefront");
  static_assert(kWLoads <= 4 && kXLoads <= 4, "places of a lane's loads");
  // (every load's chunk of a lane is block j of its row, its rows being even
  // multiples of eight apart)
  uint32_t woff[4], xoff[4];
  int jb[4];
  const int lr = lane >> 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * (wave + i * kWaves) + lr;
    jb[i] = (lane & 7) ^ ((r >> 1) & 7);
    woff[i] = xoff[i] = (uint32_t)r * half + 16u * jb[i];
  }
  auto fill = [&](int t, uint8_t *a) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          crs, (__attribute__((address_space(3))) void *)(a + (kw * kStage + (wave + i * kWaves) * 1024)),
          16, woff[i] + (((t < 2 * g1) & (8 * t + jb[i] < nb)) ? (uint32_t)t * 128u : kMxOOB), 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xrs, (__attribute__((address_space(3))) void *)(a + (kw * kStage + kWBytes + (wave + i * kWaves) * 1024)),
          16, xoff[i] + (((t < 2 * g1) & (8 * t + jb[i] < nb)) ? (uint32_t)t * 128u : kMxOOB), 0, 0, 0);
  };

  const int tid = wave * 64 + lane;  // of the share
  WScales wscales(A.scales, row0, tile_rows, nb);
  XScales xscales(A.xscales, tok0, tile_toks, nb);
  uint8_t *const ws = sa + kw * kScales, *const xs = ws + WScales::kBytes;

  // (places of the lane's operands in a stage: 32 rows further on the
  // permutation is the same)
  uint32_t wbase[4], xbase[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    wbase[s] = kw * kStage + row_off(rw * 32 * RT + l32, 2 * s + h);
    xbase[s] = kw * kStage + kWBytes + row_off(tw * 32 * NT + l32, 2 * s + h);
  }
  uint4 w[2][RT], b[2][NT];
  auto reads = [&](const uint8_t *a, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RT; ++i) w[s & 1][i] = *reinterpret_cast<const uint4 *>(a + (wbase[s] + 4096u * i));
#pragma unroll
    for (int j = 0; j < NT; ++j) b[s & 1][j] = *reinterpret_cast<const uint4 *>(a + (xbase[s] + 4096u * j));
  };
  // Step t, the U-th of its group, from stage `a`. `far` is the stage that the step
  // before read, filled for step t + 2: every wavefront's reads of it have returned,
  // since its products used them before the barrier. Before the barrier the wavefront
  // waits until at most its loads of this step are under way: loads complete in
  // order, so behind it step t + 1 lies in LDS.
  uint4 sw[RT], sx[NT];
  auto step = [&](int t, auto u_c, const uint8_t *a, uint8_t *far) __attribute__((always_inline)) {
    constexpr int U = decltype(u_c)::value;
    fill(t + 2, far);
    __builtin_amdgcn_sched_barrier(0);
    reads(a, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, RT + NT, 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) reads(a, s + 1);
      uint32_t wsc[RT], xsc[NT];
#pragma unroll
      for (int i = 0; i < RT; ++i)
        wsc[i] = (U == 0 ? s < 2 ? sw[i].x : sw[i].y : s < 2 ? sw[i].z : sw[i].w) >> (8 * h);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        xsc[j] = (U == 0 ? s < 2 ? sx[j].x : sx[j].y : s < 2 ? sx[j].z : sx[j].w) >> (8 * h);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = s & 1 ? mfma_mx32<2>(w[1][i], wsc[i], b[1][j], xsc[j], acc[i][j])
                            : mfma_mx32<0>(w[0][i], wsc[i], b[0][j], xsc[j], acc[i][j]);
      if (s < 3) __builtin_amdgcn_sched_group_barrier(0x100, RT + NT, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, RT * NT, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    // (keeps the products in their step: nothing else ties them to a place)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j][0] = materialize(acc[i][j][0]);
    asm volatile("s_waitcnt vmcnt(%0)" : : "i"(kWLoads + kXLoads) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  wscales.load(16 * g0, tid);
  xscales.load(16 * g0, tid);
  fill(2 * g0, xa0);
  __builtin_amdgcn_sched_barrier(0);
  fill(2 * g0 + 1, xa1);
  wscales.store(ws, tid);
  xscales.store(xs, tid);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "i"(kWLoads + kXLoads) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
  wscales.load(16 * (g0 + kTurns), tid);
  xscales.load(16 * (g0 + kTurns), tid);
  auto group = [&](int g, const uint8_t *a0, uint8_t *a1, uint8_t *a2) __attribute__((always_inline)) {
    const int turn = (g - g0) % kTurns;
    if (g > g0 && turn == 0) {  // new scales in LDS
      wscales.store(ws, tid);
      xscales.store(xs, tid);
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" : : : "memory");
      wscales.load(16 * (g + kTurns), tid);
      xscales.load(16 * (g + kTurns), tid);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) sw[i] = WScales::read(ws, rw * 32 * RT + 32 * i + l32, turn);
#pragma unroll
    for (int j = 0; j < NT; ++j) sx[j] = XScales::read(xs, tw * 32 * NT + 32 * j + l32, turn);
    step(2 * g, std::integral_constant<int, 0>{}, a0, a2);
    step(2 * g + 1, std::integral_constant<int, 1>{}, a1, const_cast<uint8_t *>(a0));
  };
  for (int g = g0;;) {
    group(g, xa0, xa1, xa2);
    if (++g >= gend) break;
    group(g, xa2, xa0, xa1);
    if (++g >= gend) break;
    group(g, xa1, xa2, xa0);
    if (++g >= gend) break;
  }
  // the zeros past the last group are in LDS before it is used again
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  __syncthreads();

  if (add_shares<RT, NT, TW, KW>(acc, kw, wave, lane, xa0, xa0 + kSums, xa1, xa1 + kSums)) return;
  store_tile<T, RT, NT, TW>(A, acc, job, at, wave, lane, xa2);
}

// Fitted, with the constants of plan_tiles, to 4096 x 4096, 4096 x 11008, 11008 x
// 4096 and 28672 x 8192 from 24 to 2048 rows, each shape measured at each: at
// 64 x 11008 x 4096 the three take 16.9, 9.5 and 8.4 us, at 400 x 4096 x 4096
// 17.1, 9.6 and 14.5, at 2048 x 11008 x 4096 62, 93 and 137.
constexpr TileShape kShapes[] = {
    {2, 2, 2, 1, 1.54, 1.09}, {1, 2, 1, 2, 1.34, 0.71}, {1, 1, 1, 2, 0.98, 0.58}};

TilePlan plan_of(const MxDesc &W, int64_t batch) {
  return plan_tiles(kShapes, W.rows, batch, (W.cols / 32 + 15) / 16);
}

template <MxType T, int RT, int NT, int TW, int KW>
hipError_t launch_tile(const TileArgs &A, hipStream_t stream) {
  const unsigned tiles = (unsigned)(A.row_tiles * A.tok_tiles);
  hipLaunchKernelGGL((mx_mx_tile_kernel<T, RT, NT, TW, KW>), dim3(tiles * A.splits),
                     dim3(64 * kRowWaves * TW * KW), 0, stream, A);
  if (A.splits > 1)
    hipLaunchKernelGGL((mx_tile_sum_kernel<T, RT, NT, TW>), dim3(tiles * RT * NT * 4),
                       dim3(64 * kRowWaves * TW), 0, stream, A);
  return hipGetLastError();
}

template <MxType T> hipError_t tile_as(const TileShape &c, const TileArgs &A, hipStream_t stream) {
  if (c.rt == 2) return launch_tile<T, 2, 2, 2, 1>(A, stream);
  if (c.nt == 2) return launch_tile<T, 1, 2, 1, 2>(A, stream);
  return launch_tile<T, 1, 1, 1, 2>(A, stream);
}

}  // namespace

double mx_gemm_mx_tile_us(const MxDesc &W, int64_t batch) {
  return std::max(plan_of(W, batch).us, mx_read_us(W));
}

int64_t mx_gemm_mx_tile_ws_bytes(const MxDesc &W, int64_t batch) { return plan_of(W, batch).ws_bytes(); }

hipError_t launch_mx_gemm_mx_tile(const MxDesc &W, const MxDesc &x, void *y, MxType type, void *ws,
                                  hipStream_t stream) {
  const TilePlan p = plan_of(W, x.rows);
  const TileArgs A = tile_args(p, W, x.codes, x.scales, x.rows, y, ws);
  return type == MxType::kF16 ? tile_as<MxType::kF16>(p.shape, A, stream)
                              : tile_as<MxType::kBF16>(p.shape, A, stream);
}

}  // namespace aqlm
