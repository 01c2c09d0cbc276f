// Product of half activations with microscaled weights for many rows of
// activations: y = x . W^T with one workgroup per [rows of W] x [tokens] tile.
//
// Expanding E2M1 costs one conversion for two weights, little enough that each
// wavefront expands its operands in registers, from codes that lie in LDS.
//   * A workgroup has four wavefronts along the rows (32 RT each) times TW
//     along the tokens (32 NT each) times KW that share out K, and multiplies
//     with v_mfma_f32_32x32x16.
//   * A K step is 64 inputs, two blocks: lane (r, h) = (lane % 32, lane / 32)
//     takes block h of row r, 16 bytes of codes, which give the operands of
//     four instructions: instruction s multiplies codes 8 s .. 8 s + 7, so its
//     activation operand is the 16 bytes of inputs 8 s of the same block of
//     the lane's token. (The sum over K does not care which inputs meet in an
//     instruction, so no code changes lanes after its load.)
//   * Codes, scales and activations reach the wavefronts through LDS, in whole
//     128-byte lines: L2 gives about 30 TB/s in such segments, a half in ones
//     of 64 bytes, a quarter of 32, an eighth of 16, since a request costs its
//     line. (Each lane loading its own row's 16 bytes of codes and a byte of
//     scales took 190 us for 2048 x 11008 x 4096, 32-byte segments of codes
//     179, this 158.) Activations go straight to LDS three steps ahead, one of four
//     stages; codes four steps at a time, up to eight ahead, one of two;
//     scales 64 steps at a time, through registers.
//   * Chunks of 16 bytes are permuted within a row of 128 bytes on their way
//     (row_off), so that the 16 lanes of an LDS pass touch 16 distinct groups
//     of banks.
//   * Where there are few tiles K is split over workgroups too, whose float32
//     sums go to the workspace, as the accumulator registers lie, and a second
//     kernel adds them in a fixed order.
#include <algorithm>

#include "mx_tile.hpp"

namespace aqlm {
namespace {

// Byte offset of 16-byte chunk j (of 8) of row r in a stage.
__device__ __forceinline__ uint32_t row_off(int r, int j) {
  return (uint32_t)r * 128u + (uint32_t)((j ^ ((r >> 1) & 7)) << 4);
}

template <MxType T, int RT, int NT, int TW, int KW>
__global__ __launch_bounds__(64 * kRowWaves * TW * KW) void mx_tile_kernel(const TileArgs A) {
  constexpr int kWaves = kRowWaves * TW;             // of one share of K
  constexpr int kRows = kRowWaves * RT * 32;         // of W in the tile
  constexpr int kXBytes = TW * NT * 32 * 128, kWBytes = kRows * 128, kSBytes = kRows * 128;
  constexpr int kSums = tile_sums_bytes<RT, NT, TW>();
  static_assert(kWBytes * KW >= kWaves * kStoreBytes<RT>, "room for the results");
  constexpr int kArray = KW == 1 || KW * kXBytes > kSums ? KW * kXBytes : kSums;
  // one array per stage: the compiler then knows which loads into LDS a read
  // of LDS can depend on
  __shared__ __attribute__((aligned(16))) uint8_t xa0[kArray], xa1[kArray], xa2[kArray], xa3[kArray];
  __shared__ __attribute__((aligned(16))) uint8_t wa0[KW * kWBytes], wa1[KW * kWBytes];
  __shared__ __attribute__((aligned(16))) uint8_t sa[KW * kSBytes];
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

  // K goes in groups of eight steps, 16 blocks. The groups of this split, and
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
  const Rsrc xrs = make_rsrc(static_cast<const uint16_t *>(A.x) + (int64_t)tok0 * A.cols,
                             (uint32_t)tile_toks * A.cols * 2u);

  float16_t acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // Activations of step t (of group t / 8), and codes of steps 4 m .. 4 m + 3,
  // into a stage. One load of a wavefront fills 1 KiB, eight rows, in lane
  // order, so a chunk's place in its row is chosen by where the lane reads
  // from. Blocks past the last one are zeros. Wavefront w of the share makes
  // loads w, w + kWaves, .. of each kind.
  constexpr int kXLoads = NT, kWLoads = 16 * RT / kWaves;
  static_assert(16 * RT % kWaves == 0 && kXLoads <= 4 && kWLoads == 4, "loads of a wavefront");
  const int lrow = lane >> 3;
  uint32_t xoff[4], woff[4];
  int xblk[4], wblk[4];  // block of the lane's chunk, from the step's first
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * (wave + i * kWaves) + lrow, j = (lane & 7) ^ ((r >> 1) & 7);
    xblk[i] = j >> 2;
    xoff[i] = (uint32_t)r * (uint32_t)A.cols * 2u + 16u * j;
    wblk[i] = j;
    woff[i] = (uint32_t)r * half + 16u * j;
  }
  auto fill_x = [&](int t, uint8_t *a) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xrs, (__attribute__((address_space(3))) void *)(a + (kw * kXBytes + (wave + i * kWaves) * 1024)), 16,
          xoff[i] + (((t < 8 * g1) & (2 * t + xblk[i] < nb)) ? (uint32_t)t * 128u : kMxOOB), 0, 0, 0);
  };
  auto fill_w = [&](int m, auto part_c, uint8_t *a) __attribute__((always_inline)) {
    constexpr int P = decltype(part_c)::value;  // half of the loads
#pragma unroll
    for (int i = 2 * P; i < 2 * P + 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          crs, (__attribute__((address_space(3))) void *)(a + (kw * kWBytes + (wave + i * kWaves) * 1024)), 16,
          woff[i] + (((m < 2 * g1) & (8 * m + wblk[i] < nb)) ? (uint32_t)m * 128u : kMxOOB), 0, 0, 0);
  };
  const int my_rows = tile_rows - rw * 32 * RT;  // of this wavefront, where there are any
  const int tid = wave * 64 + lane;              // of the share
  ScaleStage<kRows, 64 * kWaves, 8> scales(A.scales, row0, tile_rows, nb);

  // (places of the lane's operands in a stage: 32 rows further on the
  // permutation is the same)
  uint32_t wbase[4], xbase[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    wbase[s] = kw * kWBytes + row_off(rw * 32 * RT + l32, 2 * s + h);
    xbase[s] = kw * kXBytes + row_off(tw * 32 * NT + l32, 4 * h + s);
  }
  auto w_of = [&](const uint8_t *a, int u, int i) __attribute__((always_inline)) {
    return *reinterpret_cast<const uint4 *>(a + (wbase[u] + 4096u * i));
  };
  auto x_of = [&](const uint8_t *a, int j, int s) __attribute__((always_inline)) {
    return *reinterpret_cast<const uint4 *>(a + (xbase[s] + 4096u * j));
  };

  // Step t, the U-th of its group, from stage `a`; `next` is the stage of step
  // t + 1 and `far` the one that the step before read, filled for step t + 3.
  // The codes of steps U = 0 .. 3 lie in wa0, of 4 .. 7 in wa1; each is filled
  // for four steps further on by the first two steps that read the other.
  // A step begins with its codes and first activation operands in registers:
  // they are read at the end of the step before, so that products go on right
  // after the barrier. Before the barrier the wavefront waits until at most
  // its loads of this step are under way: loads complete in order, so behind
  // the barrier all that was asked for in the steps before lies in LDS:
  // activations of step t + 2, codes of step t + 2 too. The operand reads of
  // this step have returned, since products used them.
  uint4 sc[RT];
  uint4 w[2][RT], b[2][NT];
  auto step = [&](auto wide_c, int t, auto u_c, const uint8_t *a, const uint8_t *next, uint8_t *far)
                  __attribute__((always_inline)) {
    constexpr bool WIDE = decltype(wide_c)::value;
    constexpr int U = decltype(u_c)::value;
    uint8_t *const wother = U < 4 ? wa1 : wa0;
    const uint8_t *const wnext = U < 3 || U == 7 ? wa0 : wa1;
    fill_x(t + 3, far);
    if constexpr (U % 4 < 2) fill_w((t >> 2) + 1, std::integral_constant<int, U % 4>{}, wother);
    __builtin_amdgcn_sched_barrier(0);
    float sv[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const uint32_t word = U < 2 ? sc[i].x : U < 4 ? sc[i].y : U < 6 ? sc[i].z : sc[i].w;
      sv[i] = mx_scale((word >> (16 * (U & 1) + 8 * h)) & 0xFFu);
    }
    if constexpr (WIDE) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint4 hi, lo;
          split_f16(x_of(a, j, s), hi, lo);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const uint32_t ww[4] = {w[U & 1][i].x, w[U & 1][i].y, w[U & 1][i].z, w[U & 1][i].w};
            const uint4 av = mx_decode8<MxType::kBF16>(ww[s], sv[i]);
            acc[i][j] = mx_mfma32<MxType::kBF16>(av, hi, acc[i][j]);
            acc[i][j] = mx_mfma32<MxType::kBF16>(finite_bf16(av), lo, acc[i][j]);
          }
        }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s == 3) {
#pragma unroll
        for (int i = 0; i < RT; ++i) w[(U + 1) & 1][i] = w_of(wnext, (U + 1) & 3, i);
      }
      if (s == 3 || !WIDE) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
          b[(s + 1) & 1][j] = s < 3 ? x_of(a, j, s + 1) : x_of(next, j, 0);
      }
      if constexpr (!WIDE) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const uint32_t ww[4] = {w[U & 1][i].x, w[U & 1][i].y, w[U & 1][i].z, w[U & 1][i].w};
          const uint4 av = mx_decode8<T>(ww[s], sv[i]);
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = mx_mfma32<T>(av, b[s & 1][j], acc[i][j]);
        }
        // the next instruction's operands are read before this one's products
        if (s == 3) __builtin_amdgcn_sched_group_barrier(0x100, NT + RT, 0);
        else __builtin_amdgcn_sched_group_barrier(0x100, NT, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, RT * NT, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0)" : : "i"(kXLoads + (U % 4 < 2 ? 2 : 0)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  scales.load(16 * g0, tid);
  fill_w(2 * g0, std::integral_constant<int, 0>{}, wa0);
  fill_w(2 * g0, std::integral_constant<int, 1>{}, wa0);
  fill_x(8 * g0, xa0);
  fill_x(8 * g0 + 1, xa1);
  __builtin_amdgcn_sched_barrier(0);
  fill_x(8 * g0 + 2, xa2);
  scales.store(sa + kw * kSBytes, tid);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "i"(kXLoads) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
  scales.load(16 * g0 + 128, tid);
#pragma unroll
  for (int i = 0; i < RT; ++i) w[0][i] = w_of(wa0, 0, i);
#pragma unroll
  for (int j = 0; j < NT; ++j) b[0][j] = x_of(xa0, j, 0);
  // a group's scales, every eighth time from new ones in LDS
  auto group_scales = [&](int g) __attribute__((always_inline)) {
    if (g > g0 && ((g - g0) & 7) == 0) {
      scales.store(sa + kw * kSBytes, tid);
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" : : : "memory");
      scales.load(16 * g + 128, tid);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
      sc[i] = scales.read(sa + kw * kSBytes, rw * 32 * RT + 32 * i + l32, (g - g0) & 7);
  };
  auto group = [&](auto wide_c, int g) __attribute__((always_inline)) {
    const int t = 8 * g;
    step(wide_c, t, std::integral_constant<int, 0>{}, xa0, xa1, xa3);
    step(wide_c, t + 1, std::integral_constant<int, 1>{}, xa1, xa2, xa0);
    step(wide_c, t + 2, std::integral_constant<int, 2>{}, xa2, xa3, xa1);
    step(wide_c, t + 3, std::integral_constant<int, 3>{}, xa3, xa0, xa2);
    step(wide_c, t + 4, std::integral_constant<int, 4>{}, xa0, xa1, xa3);
    step(wide_c, t + 5, std::integral_constant<int, 5>{}, xa1, xa2, xa0);
    step(wide_c, t + 6, std::integral_constant<int, 6>{}, xa2, xa3, xa1);
    step(wide_c, t + 7, std::integral_constant<int, 7>{}, xa3, xa0, xa2);
  };
  int g = g0;
  for (; g < gend; ++g) {
    group_scales(g);
    if constexpr (T == MxType::kF16) {
      u16x2_t m = {0, 0};
#pragma unroll
      for (int i = 0; i < RT; ++i) m = __builtin_elementwise_max(m, mx_above_f16(sc[i]));
      const bool f = (m.x <= 36) & (m.y <= 36);
      if (!__all(f) & (my_rows > 0)) break;
    }
    group(std::false_type{}, g);
  }
  // From the wavefront's first group with a scale that float16 weights cannot
  // take: the same product in bfloat16, which holds every weight, with x split
  // exactly in two. The barriers are those of the other loop, one a step, so
  // wavefronts in either meet.
  if constexpr (T == MxType::kF16)
    for (bool again = false; g < gend; ++g, again = true) {
      if (again) group_scales(g);
      group(std::true_type{}, g);
    }
  // the zeros past the last group are in LDS before it is used again
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  __syncthreads();

  if (add_shares<RT, NT, TW, KW>(acc, kw, wave, lane, xa0, xa1, xa2, xa3)) return;
  store_tile<T, RT, NT, TW>(A, acc, job, at, wave, lane, wa0);
}

// Fitted, with the constants of plan_tiles, to 4096 x 4096, 4096 x 11008, 11008 x
// 4096 and 28672 x 8192 from 24 to 2048 rows, each shape measured at each: at
// 64 x 11008 x 4096 the three take 28.6, 16.1 and 12.7 us, at 400 x 4096 x 4096
// 41.5, 18.4 and 23.3, at 2048 x 11008 x 4096 155, 198 and 246.
constexpr TileShape kShapes[] = {
    {2, 2, 2, 1, 3.96, 2.17}, {1, 2, 1, 2, 2.83, 1.55}, {1, 1, 1, 2, 2.07, 0.73}};

TilePlan plan_of(const MxDesc &W, int64_t batch, bool split) {
  return plan_tiles(kShapes, W.rows, batch, (W.cols / 32 + 15) / 16, split ? 8 : 1);
}

template <MxType T, int RT, int NT, int TW, int KW>
hipError_t launch_tile(const TileArgs &A, hipStream_t stream) {
  const unsigned tiles = (unsigned)(A.row_tiles * A.tok_tiles);
  hipLaunchKernelGGL((mx_tile_kernel<T, RT, NT, TW, KW>), dim3(tiles * A.splits),
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

double mx_gemm_tile_us(const MxDesc &W, int64_t batch, bool split) {
  return std::max(plan_of(W, batch, split).us, mx_read_us(W));
}

int64_t mx_gemm_tile_ws_bytes(const MxDesc &W, int64_t batch) { return plan_of(W, batch, true).ws_bytes(); }

hipError_t launch_mx_gemm_tile(const MxDesc &W, const void *x, int64_t batch, void *y, MxType type,
                               bool split, void *ws, hipStream_t stream) {
  const TilePlan p = plan_of(W, batch, split);
  const TileArgs A = tile_args(p, W, x, nullptr, batch, y, ws);
  return type == MxType::kF16 ? tile_as<MxType::kF16>(p.shape, A, stream)
                              : tile_as<MxType::kBF16>(p.shape, A, stream);
}

}  // namespace aqlm
