// Product of two microscaled matrices for many rows of activations, one
// workgroup per [rows of W] x [tokens] tile (mx_tile.hpp).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 with 4-bit operands: lane (r, h) = (lane %
// 32, lane / 32) gives the 16 bytes of block h (32 codes) of row r of the
// 64-input chunk and, in a byte of a register, that block's scale; W and x
// alike, and both as they lie in memory.
//   * A K step is 128 inputs, two such chunks. Both sides go from memory
//     straight to LDS three steps ahead, into one of four stages of 64-byte
//     rows; four neighbouring lanes load a row's 64 bytes. 16-byte chunk c of
//     row r lies at chunk c ^ ((r >> 2) & 3), so that the 16 lanes of an LDS
//     pass touch 16 distinct groups of banks.
//   * A lane's scales of a step are one word of its row. Shifted by 8 h its
//     bytes 0 and 2 are those of the two chunks, which the instruction selects.
//   * A 32 x 32 x 64 product takes a SIMD as long as 32 x 32 x 16 of halves,
//     with the same two operand reads of 1 KiB: with 64 x 64 per wavefront the
//     reads keep LDS as long as the products keep the matrix cores.
#include <algorithm>

#include "mx_tile.hpp"

namespace aqlm {
namespace {

// Byte offset of block c (of 4) of row r in its part of a stage.
__device__ __forceinline__ uint32_t row_off(int r, int c) {
  return (uint32_t)r * 64u + (uint32_t)((c ^ ((r >> 2) & 3)) << 4);
}

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
  constexpr int kWBytes = kRowWaves * RT * 32 * 64, kXBytes = TW * NT * 32 * 64;
  constexpr int kStage = kWBytes + kXBytes;
  constexpr int kSums = tile_sums_bytes<RT, NT, TW>();
  constexpr int kArray = KW == 1 || KW * kStage > kSums ? KW * kStage : kSums;
  // one array per stage: the compiler then knows which loads into LDS a read
  // of LDS can depend on
  __shared__ __attribute__((aligned(16))) uint8_t xa0[kArray], xa1[kArray], xa2[kArray], xa3[kArray];
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

  // K goes in groups of four steps, 16 blocks. The groups of this split, and
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

  // Step t (of group t / 4) into a stage. One load of a wavefront fills 1 KiB,
  // 16 rows, in lane order, so a chunk's place in its row is chosen by where
  // the lane reads from. Blocks past the last one are zeros. Wavefront w of
  // the share makes loads w, w + kWaves, .. of each side.
  constexpr int kWLoads = 8 * RT / kWaves;                      // 8 RT of codes of W, all whole
  constexpr int kXLoads = (2 * NT * TW + kWaves - 1) / kWaves;  // 2 NT TW of codes of x
  constexpr bool kAllX = (2 * NT * TW) % kWaves == 0;
  static_assert(8 * RT % kWaves == 0, "every wavefront loads as many codes of W");
  constexpr int kLoads = kWLoads + (kAllX ? kXLoads : 0);       // of a wavefront and step, at least
  // (every load's chunk of a lane is block j of its row: c is a multiple of
  // four rows apart from the next)
  const int j = (lane & 3) ^ ((lane >> 4) & 3);
  static_assert(kWLoads <= 4 && kXLoads <= 4, "places of a lane's loads");
  uint32_t woff[4], xoff[4];
#pragma unroll
  for (int i = 0; i < kWLoads; ++i)
    woff[i] = (uint32_t)(16 * (wave + i * kWaves) + (lane >> 2)) * half + 16u * j;
#pragma unroll
  for (int i = 0; i < kXLoads; ++i)
    xoff[i] = (uint32_t)(16 * (wave + i * kWaves) + (lane >> 2)) * half + 16u * j;
  auto fill = [&](int t, uint8_t *a) __attribute__((always_inline)) {
    const bool in = (t < 4 * g1) & (4 * t + j < nb);
    const uint32_t step = in ? (uint32_t)t * 64u : kMxOOB;
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          crs, (__attribute__((address_space(3))) void *)(a + (kw * kStage + (wave + i * kWaves) * 1024)),
          16, woff[i] + step, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      if (kAllX || wave + i * kWaves < 2 * NT * TW)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            xrs, (__attribute__((address_space(3))) void *)(a + (kw * kStage + kWBytes + (wave + i * kWaves) * 1024)),
            16, xoff[i] + step, 0, 0, 0);
  };

  ScaleRows<RT> wscales(A.scales, row0, tile_rows, nb, rw * 32 * RT + l32);
  ScaleRows<NT> xscales(A.xscales, tok0, tile_toks, nb, tw * 32 * NT + l32);
  auto group_at = [&](int g) __attribute__((always_inline)) { return max(0, min(g, g1 - 1)); };

  // (places of the lane's operands in a stage: 32 rows further on the
  // permutation is the same)
  uint32_t wbase[2], xbase[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    wbase[s] = kw * kStage + row_off(rw * 32 * RT + l32, 2 * s + h);
    xbase[s] = kw * kStage + kWBytes + row_off(tw * 32 * NT + l32, 2 * s + h);
  }
  uint4 w[2][RT], b[2][NT];
  auto reads = [&](const uint8_t *a, auto s_c) __attribute__((always_inline)) {
    constexpr int S = decltype(s_c)::value;
#pragma unroll
    for (int i = 0; i < RT; ++i) w[S][i] = *reinterpret_cast<const uint4 *>(a + (wbase[S] + 2048u * i));
#pragma unroll
    for (int j = 0; j < NT; ++j) b[S][j] = *reinterpret_cast<const uint4 *>(a + (xbase[S] + 2048u * j));
  };
  typedef std::integral_constant<int, 0> S0;
  typedef std::integral_constant<int, 1> S1;

  // Step t, the U-th of its group, from stage `a`; `next` is the stage of step
  // t + 1 and `far` the one that the step before read, filled for step t + 3.
  // A step begins with its first operands in registers: they are read at the
  // end of the step before, so that products go on right after the barrier.
  // Before the barrier the wavefront waits until at most its loads of step t +
  // 3 are under way: loads complete in order, so behind the barrier all of
  // step t + 2 lies in LDS. The operand reads of this step have returned,
  // since products used them.
  uint4 sw[RT], sx[NT], swn[RT], sxn[NT];
  auto step = [&](int t, auto u_c, const uint8_t *a, const uint8_t *next, uint8_t *far)
                  __attribute__((always_inline)) {
    constexpr int U = decltype(u_c)::value;
    fill(t + 3, far);
    __builtin_amdgcn_sched_barrier(0);
    uint32_t wsc[RT], xsc[NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
      wsc[i] = (U == 0 ? sw[i].x : U == 1 ? sw[i].y : U == 2 ? sw[i].z : sw[i].w) >> (8 * h);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      xsc[j] = (U == 0 ? sx[j].x : U == 1 ? sx[j].y : U == 2 ? sx[j].z : sx[j].w) >> (8 * h);
    reads(a, S1{});
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mfma_mx32<0>(w[0][i], wsc[i], b[0][j], xsc[j], acc[i][j]);
    // the next instruction's operands are read before this one's products
    __builtin_amdgcn_sched_group_barrier(0x100, RT + NT, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, RT * NT, 0);
    reads(next, S0{});
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mfma_mx32<2>(w[1][i], wsc[i], b[1][j], xsc[j], acc[i][j]);
    __builtin_amdgcn_sched_group_barrier(0x100, RT + NT, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, RT * NT, 0);
    __builtin_amdgcn_sched_barrier(0);
    // (keeps the products in their step: nothing else ties them to a place)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j][0] = materialize(acc[i][j][0]);
    asm volatile("s_waitcnt vmcnt(%0)" : : "i"(kLoads) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  wscales.load(group_at(g0), sw);
  xscales.load(group_at(g0), sx);
  wscales.place(group_at(g0), sw);
  xscales.place(group_at(g0), sx);
  fill(4 * g0, xa0);
  __builtin_amdgcn_sched_barrier(0);
  fill(4 * g0 + 1, xa1);
  __builtin_amdgcn_sched_barrier(0);
  fill(4 * g0 + 2, xa2);
  asm volatile("s_waitcnt vmcnt(%0)" : : "i"(kLoads) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
  reads(xa0, S0{});
  for (int g = g0; g < gend; ++g) {
    wscales.load(group_at(g + 1), swn);
    xscales.load(group_at(g + 1), sxn);
    step(4 * g, std::integral_constant<int, 0>{}, xa0, xa1, xa3);
    step(4 * g + 1, std::integral_constant<int, 1>{}, xa1, xa2, xa0);
    step(4 * g + 2, std::integral_constant<int, 2>{}, xa2, xa3, xa1);
    step(4 * g + 3, std::integral_constant<int, 3>{}, xa3, xa0, xa2);
    wscales.place(group_at(g + 1), swn);
    xscales.place(group_at(g + 1), sxn);
#pragma unroll
    for (int i = 0; i < RT; ++i) sw[i] = swn[i];
#pragma unroll
    for (int j = 0; j < NT; ++j) sx[j] = sxn[j];
  }
  // the zeros past the last group are in LDS before the wavefront can end
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");

  if (add_shares<RT, NT, TW, KW>(acc, kw, wave, lane, xa0, xa1, xa2, xa3)) return;
  store_tile<T, RT, NT, TW>(A, acc, job, at, wave, lane);
}

constexpr TileShape kShapes[] = {
    {2, 2, 2, 1, 1.2, 1.2}, {1, 2, 1, 2, 1.0, 0.8}, {1, 1, 1, 2, 0.9, 0.5}};

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

int64_t mx_gemm_mx_tile_ws_bytes(const MxDesc &W, int64_t batch) { return plan_of(W, batch).ws_bytes(); }

hipError_t launch_mx_gemm_mx_tile(const MxDesc &W, const MxDesc &x, void *y, MxType type, void *ws,
                                  hipStream_t stream) {
  const TilePlan p = plan_of(W, x.rows);
  const TileArgs A = tile_args(p, W, x.codes, x.scales, x.rows, y, ws);
  return type == MxType::kF16 ? tile_as<MxType::kF16>(p.shape, A, stream)
                              : tile_as<MxType::kBF16>(p.shape, A, stream);
}

}  // namespace aqlm
