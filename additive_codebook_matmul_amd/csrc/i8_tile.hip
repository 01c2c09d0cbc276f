// Products of int8 layers and gated blocks for many tokens: one workgroup per
// [rows of W] x [tokens] tile.
//
// v_mfma_i32_32x32x32_i8: lane (r, h) = (lane % 32, lane / 32) gives the 16 bytes
// h of row r of a 32-input chunk, W and x alike, as they lie in memory.
//   * A K step is 128 inputs, four chunks: 128-byte rows, whole lines of L2. Both
//     sides go from memory straight to LDS, one or two steps ahead; 16-byte chunk c
//     of row r lies at chunk c ^ ((r >> 1) & 7), so that the 16 lanes of an LDS pass
//     touch 16 distinct groups of banks.
//   * A wavefront computes 32 RT x 32 NT of the tile; per 32 inputs it reads RT + NT
//     KiB from LDS for RT NT instructions of 32 cycles.
//   * GATED: of a wavefront's 32 RT rows the first half are the gate's, the second
//     the same ones of up, so that both products of a result meet in a lane.
// What bounds it: with many tokens the card's power and the wait for a step's loads at
// its barrier. A 256 x 256 tile's step takes 1.15 us where its instructions need 1.09,
// alone; with every CU at work the clock falls (2048 x 8192 x 28672 takes 322 us with
// zeros for data, 410 to 495 with codes, 2.0 to 2.35 POP/s) and the matrix cores are busy
// for 57 % of the cycles, LDS for 24 to 30. 1999 x 4096 x 11008 takes 85 us, 2048 x 11008 x
// 4096 gated 186. With few tokens the reading of W: 19 x 28672 x 8192 gated 72 us, 6.5
// TB/s.
#include "i8_gemm.hpp"
#include "i8_tile.hpp"
#include "mx_tile.hpp"

namespace aqlm {
namespace {

struct I8TileArgs {
  I8Args a;
  int4_vt *part;  // [splits][tiles][RT * NT * 4][64 RW TW], or null
  int row_tiles, tok_tiles, splits, steps_per_split;
};

// Byte offset of chunk c (of 8) of row r in its part of a stage.
__device__ __forceinline__ uint32_t row_off(int r, int c) {
  return (uint32_t)r * 128u + (uint32_t)((c ^ ((r >> 1) & 7)) << 4);
}

// ONCE: the tile's rows are read by this workgroup alone (one tile of tokens), past
// the caches.
template <MxType T, bool GATED, class S, bool ONCE>
__global__ __launch_bounds__(S::kThreads *S::KW) void i8_tile_kernel(const I8TileArgs B) {
  constexpr int RT = S::RT, NT = S::NT, TW = S::TW, KW = S::KW, kWaves = S::kWaves;
  constexpr int kStage = S::kStage, kWBytes = S::kWBytes;
  constexpr int M = GATED ? 2 : 1, OT = RT / M;     // matrices, 32-row tiles of results
  constexpr int kOut = S::kRows / M;                // result rows of the tile
  constexpr int kArray = KW * kStage > (KW > 1 ? S::kSums : 0) ? KW * kStage : S::kSums;
  constexpr int kStore = OT * 2048 > 4096 ? OT * 2048 : 4096;  // of LDS a wavefront, for its results
  static_assert(RT % M == 0 && kArray >= kWaves * kStore && S::kRows <= 1024 && S::kRows <= S::kThreads * KW,
                "room for the results and the scales");
  const I8Args &A = B.a;
  // one array per stage: the compiler then knows which loads into LDS a read
  // of LDS can depend on
  __shared__ __attribute__((aligned(16))) uint8_t s0[kArray], s1[kArray], s2[S::STAGES > 2 ? kArray : 4096];
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = KW == 1 ? 0 : wave_all / kWaves, wave = KW == 1 ? wave_all : wave_all % kWaves;
  const int rw = wave / TW, tw = wave % TW;
  const int l32 = lane & 31, h = lane >> 5;
  const int tiles = B.row_tiles * B.tok_tiles;
  const int job = xcd_job((int)blockIdx.x, tiles * B.splits);
  const int split = __builtin_amdgcn_readfirstlane(job / tiles);
  const TilePlace at = tile_place(job - split * tiles, B.row_tiles, B.tok_tiles);
  const int row0 = at.row_tile * kOut, tok0 = at.tok_tile * S::kToks;
  const uint32_t cols = (uint32_t)A.cols;

  // The steps of this split, and of those the wavefront's: each of the KW shares
  // takes as many as the largest (past its end with zeros), so that all meet at
  // every barrier.
  const int t0 = split * B.steps_per_split, t1 = min((A.cols + 127) >> 7, t0 + B.steps_per_split);
  const int share = (t1 - t0 + KW - 1) / KW;
  const int g0 = t0 + kw * share, g1 = min(t1, g0 + share), gend = g0 + share;

  // resources that end with the tile's last row: rows past it read zero
  const int tile_rows = __builtin_amdgcn_readfirstlane(min(kOut, A.rows - row0));
  const int tile_toks = __builtin_amdgcn_readfirstlane(min(S::kToks, A.batch - tok0));
  const Rsrc xrs = make_rsrc(A.x + (int64_t)tok0 * cols, (uint32_t)tile_toks * cols);

  int16_vt acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  // the tile's scales, on their way early: a channel's by its thread, the lane's tokens'
  const int wrow0 = row0 + rw * 32 * OT, wtok0 = tok0 + tw * 32 * NT;
  float channel = 0.f, token[NT];
  if ((int)threadIdx.x < S::kRows)
    channel = A.ws[threadIdx.x / kOut][min(row0 + (int)threadIdx.x % kOut, A.rows - 1)];
#pragma unroll
  for (int j = 0; j < NT; ++j) token[j] = A.xs[min(wtok0 + 32 * j + l32, A.batch - 1)];

  // Step t into a stage. One load of a wavefront fills 1 KiB, eight rows, in lane
  // order, so a chunk's place in its row is chosen by where the lane reads from
  // (chunk jb, or jb ^ 4 in every other one of a lane's loads where those are an odd
  // number of eights apart). Wavefront w of the share makes loads w, w + kWaves, ..
  // of each side.
  constexpr int kWLoads = S::kRows / 8 / kWaves, kXLoads = S::kToks / 8 / kWaves;
  static_assert(S::kRows % (8 * kWaves) == 0 && S::kToks % (8 * kWaves) == 0, "loads");
  static_assert(kWLoads <= 8 && kXLoads <= 8, "places of a lane's loads");
  uint32_t woff[8], xoff[8];
  const int8_t *wfrom[8];
  const int lr = lane >> 3, jb = (lane & 7) ^ ((4 * wave + (lr >> 1)) & 7);
#pragma unroll
  for (int i = 0; i < kWLoads; ++i) {
    const int r8 = 8 * (wave + i * kWaves);  // uniform
    int row = r8;
    const int8_t *of = A.w[0];
    if constexpr (GATED) {
      const int in = r8 % (32 * RT);
      of = in >= 16 * RT ? A.w[1] : A.w[0];
      row = r8 / (32 * RT) * (16 * RT) + in % (16 * RT);
    }
    wfrom[i] = of + (int64_t)row0 * cols;
    woff[i] = (uint32_t)(row + lr) * cols + 16u * (jb ^ (4 * (i * kWaves & 1)));
  }
#pragma unroll
  for (int i = 0; i < kXLoads; ++i) xoff[i] = (uint32_t)(8 * (wave + i * kWaves) + lr) * cols + 16u * (jb ^ (4 * (i * kWaves & 1)));
  typedef __attribute__((address_space(3))) void *LdsPtr;
  // ONCE: each row of tiles begins elsewhere in its share of K (whole numbers: any
  // order gives the same sum). Rows of W are often a power of two apart, and so may the
  // two matrices be: workgroups at the same place of K then ask the same channels of
  // memory (19 tokens of 28672 x 8192 gated 101 us, or 90 with other addresses, and
  // 72 this way).
  const int shift = ONCE && g1 > g0 ? __builtin_amdgcn_readfirstlane(at.row_tile % (g1 - g0)) : 0;
  auto fill = [&](int step_t, uint8_t *a) __attribute__((always_inline)) {
    int t = step_t;
    if constexpr (ONCE) {
      t += shift;
      if (t >= g1) t -= g1 - g0;
    }
    const uint32_t k0 = ((step_t < g1) & (128 * t + 16 * jb < A.cols)) ? (uint32_t)t * 128u : kMxOOB;
    const uint32_t k1 = ((step_t < g1) & (128 * t + 16 * (jb ^ 4) < A.cols)) ? (uint32_t)t * 128u : kMxOOB;
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(wfrom[i], (uint32_t)tile_rows * cols), (LdsPtr)(a + (kw * kStage + (wave + i * kWaves) * 1024)), 16,
                                               woff[i] + (i * kWaves & 1 ? k1 : k0), 0, 0, ONCE ? 2 : 0);
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xrs,
                                               (LdsPtr)(a + (kw * kStage + kWBytes + (wave + i * kWaves) * 1024)), 16,
                                               xoff[i] + (i * kWaves & 1 ? k1 : k0), 0, 0, 0);
  };

  // (places of the lane's operands in a stage: 32 rows further on the
  // permutation is the same)
  uint32_t wbase[4], xbase[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    wbase[s] = kw * kStage + row_off(rw * 32 * RT + l32, 2 * s + h);
    xbase[s] = kw * kStage + kWBytes + row_off(tw * 32 * NT + l32, 2 * s + h);
  }
  // Operands of chunk s of a step, and its products. Those of a step's last chunk
  // come in the next step, while its first reads are under way behind the barrier.
  // (The first step's are zeros.)
  uint4 w[2][RT], b[2][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i) w[1][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < NT; ++j) b[1][j] = make_uint4(0, 0, 0, 0);
  auto reads = [&](const uint8_t *a, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NT; ++j) b[s & 1][j] = *reinterpret_cast<const uint4 *>(a + (xbase[s] + 4096u * j));
#pragma unroll
    for (int i = 0; i < RT; ++i) w[s & 1][i] = *reinterpret_cast<const uint4 *>(a + (wbase[s] + 4096u * i));
  };
  auto products = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = i8_mfma32(w[s & 1][i], b[s & 1][j], acc[i][j]);
  };
  // Step t from stage `a`. `far` is the stage that the step before read, filled for
  // step t + STAGES - 1: every wavefront's reads of it have returned before the
  // barrier. Before the barrier the wavefront waits for its own reads and until at
  // most STAGES - 2 steps' loads are under way: loads complete in order, so behind it
  // step t + 1 lies in LDS.
  auto step = [&](int t, const uint8_t *a, uint8_t *far) __attribute__((always_inline)) {
    fill(t + S::STAGES - 1, far);
    __builtin_amdgcn_sched_barrier(0);
    reads(a, 0);
    products(3);
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      reads(a, s + 1);
      products(s);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      __builtin_amdgcn_sched_group_barrier(0x100, RT + NT, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, RT * NT, 0);
    }
    // (keeps the products in their step: nothing else ties them to a place)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j][0] = held(acc[i][j][0]);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "i"((S::STAGES - 2) * (kWLoads + kXLoads)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  fill(g0, s0);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (S::STAGES > 2) {
    fill(g0 + 1, s1);
    __builtin_amdgcn_sched_barrier(0);
  }
  asm volatile("s_waitcnt vmcnt(%0)" : : "i"((S::STAGES - 2) * (kWLoads + kXLoads)) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
  // (whole turns of the stages: with a way out after each step the compiler keeps
  // the sums in two sets of registers and moves them)
  int g = g0;
  for (; g + S::STAGES <= gend; g += S::STAGES) {
    step(g, s0, S::STAGES > 2 ? s2 : s1);
    step(g + 1, s1, s0);
    if constexpr (S::STAGES > 2) step(g + 2, s2, s1);
  }
  if (g < gend) step(g, s0, S::STAGES > 2 ? s2 : s1);
  if constexpr (S::STAGES > 2)
    if (g + 1 < gend) step(g + 1, s1, s0);
  products(3);
  // what is under way past the last step is in LDS before it is used again
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  __syncthreads();
  float *const scales = reinterpret_cast<float *>(s2);  // [M][kOut]
  if ((int)threadIdx.x < S::kRows) scales[threadIdx.x] = channel;
  if constexpr (KW == 1) __syncthreads();

  if (i8_join_shares<S>(acc, kw, wave, lane, s0)) return;  // (whole numbers: any order gives the same)
  if (B.splits > 1) return i8_store_part<S>(acc, B.part, job, wave, lane, wtok0, A.batch);

  // 32 tokens of the wavefront at a time
  uint8_t *const mine = s1 + wave * kStore;
  const bool lines = (A.rows & 7) == 0;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int tokj = wtok0 + 32 * j;
    float4_t out[OT][4], v[M][OT][4];
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const float4_t c = *reinterpret_cast<const float4_t *>(scales + m * kOut + rw * 32 * OT + 32 * i + 8 * q + 4 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[m][i][q][e] = i8_value(acc[i + m * OT][j][4 * q + e], c[e], token[j]);
        }
        if constexpr (GATED) {
#pragma unroll
          for (int e = 0; e < 4; ++e) out[i][q][e] = materialize(act_value(A.act, v[0][i][q][e]) * v[M - 1][i][q][e]);
        } else {
          out[i][q] = v[0][i][q];
        }
      }
    if (lines) {
      // (i8_store_lines, here in place: as a call it costs the gated 256 x 256 tile spills)
      constexpr int kChunks = 4 * OT;  // of 16 bytes, eight rows, for a token
#pragma unroll
      for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = (4 * i + q) ^ (l32 & (kChunks - 1));
          const float4_t &o = out[i][q];
          *reinterpret_cast<uint2 *>(mine + (l32 * kChunks + c) * 16 + 8 * h) =
              make_uint2(f2t<T>(o[0]) | (f2t<T>(o[1]) << 16), f2t<T>(o[2]) | (f2t<T>(o[3]) << 16));
        }
      wave_exchange();
#pragma unroll
      for (int k = 0; k < kChunks / 2; ++k) {
        const int id = 64 * k + lane, tt = id / kChunks, c = id % kChunks;
        const uint4 r = *reinterpret_cast<const uint4 *>(mine + (tt * kChunks + (c ^ (tt & (kChunks - 1)))) * 16);
        const int tok = tokj + tt, row = wrow0 + 8 * c;
        if (tok < A.batch && row < A.rows) *reinterpret_cast<uint4 *>(A.y + (int64_t)tok * A.rows + row) = r;
      }
      wave_exchange();
    } else if (tokj + l32 < A.batch) {
#pragma unroll
      for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          store4<T>(A.y + (int64_t)(tokj + l32) * A.rows, wrow0 + 32 * i + 8 * q + 4 * h, A.rows, out[i][q],
                    (A.rows & 3) == 0);
    }
    if constexpr (GATED) {
      if (A.g == nullptr) continue;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        float *const to = m == 0 ? A.g : A.u;
#pragma unroll
        for (int i = 0; i < OT; ++i) {
          if (lines) {  // 128 bytes, 32 rows, a token
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<float4_t *>(mine + l32 * 128 + (((2 * q + h) ^ (l32 & 7)) << 4)) = v[m][i][q];
            wave_exchange();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int tt = 8 * k + (lane >> 3), c = lane & 7;
              const float4_t r = *reinterpret_cast<const float4_t *>(mine + tt * 128 + ((c ^ (tt & 7)) << 4));
              const int tok = tokj + tt, row = wrow0 + 32 * i + 4 * c;
              if (tok < A.batch && row < A.rows)
                *reinterpret_cast<float4_t *>(to + (int64_t)tok * A.rows + row) = r;
            }
            wave_exchange();
          } else if (tokj + l32 < A.batch) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int row = wrow0 + 32 * i + 8 * q + 4 * h + e;
                if (row < A.rows) to[(int64_t)(tokj + l32) * A.rows + row] = v[m][i][q][e];
              }
          }
        }
      }
    }
  }
}

// Sums of the split parts, and the results.
template <MxType T, bool GATED, class S>
__global__ __launch_bounds__(S::kThreads) void i8_tile_sum_kernel(const I8TileArgs B) {
  constexpr int NT = S::NT, M = GATED ? 2 : 1, OT = S::RT / M;
  const I8Args &A = B.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles = B.row_tiles * B.tok_tiles;
  const int slot = (int)blockIdx.x % (OT * NT * 4), tile = (int)blockIdx.x / (OT * NT * 4);
  const int q = slot & 3, j = (slot >> 2) % NT, i = (slot >> 2) / NT;
  const TilePlace at = tile_place(tile, B.row_tiles, B.tok_tiles);
  const int tok = at.tok_tile * S::kToks + (wave % S::TW) * 32 * NT + 32 * j + (lane & 31);
  const int row = at.row_tile * (S::kRows / M) + (wave / S::TW) * 32 * OT + 32 * i + 8 * q + 4 * (lane >> 5);
  if (tok >= A.batch || row >= A.rows) return;
  const int64_t stride = (int64_t)tiles * (S::RT * NT * 4) * S::kThreads;
  int4_vt v[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int4_vt *p = B.part + ((int64_t)tile * (S::RT * NT * 4) + ((i + m * OT) * NT + j) * 4 + q) * S::kThreads + tid;
    v[m] = i8_sum_parts(p, stride, B.splits);
  }
  i8_store4<T, GATED>(A, tok, row, v);
}

template <MxType T, bool GATED, class S> hipError_t launch_shape(const I8TileArgs &B, hipStream_t stream) {
  const unsigned tiles = (unsigned)(B.row_tiles * B.tok_tiles);
  const dim3 grid(tiles * B.splits), block(S::kThreads * S::KW);
  // (19 tokens of 28672 x 8192 gated 97 us through the caches, 87 past them)
  if (B.tok_tiles == 1) hipLaunchKernelGGL((i8_tile_kernel<T, GATED, S, true>), grid, block, 0, stream, B);
  else hipLaunchKernelGGL((i8_tile_kernel<T, GATED, S, false>), grid, block, 0, stream, B);
  if (B.splits > 1)
    hipLaunchKernelGGL((i8_tile_sum_kernel<T, GATED, S>), dim3(tiles * (S::RT / (GATED ? 2 : 1)) * S::NT * 4),
                       dim3(S::kThreads), 0, stream, B);
  return hipGetLastError();
}

template <MxType T, bool GATED> hipError_t tile_as(int shape, const I8TileArgs &B, hipStream_t stream) {
  using namespace i8_tile;  // (in the order of its costs)
  if (shape == 0) return launch_shape<T, GATED, Large>(B, stream);
  if (shape == 1) return launch_shape<T, GATED, Wide>(B, stream);
  if (shape == 2) return launch_shape<T, GATED, Middle>(B, stream);
  if (shape == 3) return launch_shape<T, GATED, Half>(B, stream);
  if (shape == 4) return launch_shape<T, GATED, Small>(B, stream);
  if (shape == 5) return launch_shape<T, GATED, Slim>(B, stream);
  return launch_shape<T, GATED, Least>(B, stream);
}

}  // namespace

hipError_t launch_i8_tile(const I8Args &A, const I8Plan &p, MxType type, bool gated, void *ws, hipStream_t stream) {
  const I8TileArgs B = {A, static_cast<int4_vt *>(ws), (int)p.across, (int)p.tok_tiles, p.splits, p.steps_per_split};
  if (type == MxType::kF16)
    return gated ? tile_as<MxType::kF16, true>(p.shape, B, stream) : tile_as<MxType::kF16, false>(p.shape, B, stream);
  return gated ? tile_as<MxType::kBF16, true>(p.shape, B, stream) : tile_as<MxType::kBF16, false>(p.shape, B, stream);
}

}  // namespace aqlm
