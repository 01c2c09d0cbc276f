// Product of half activations with microscaled weights for many rows of
// activations: y = x . W^T with one workgroup per [rows of W] x [tokens] tile.
//
// Expanding E2M1 costs one conversion for two weights, little enough that each
// wavefront expands its own rows straight from the codes in registers: the
// weights never pass through LDS, where only the activations lie, shared by
// the workgroup's wavefronts.
//   * Wavefront w owns rows 32 RT w .. + 32 RT - 1 of the tile and all of its
//     32 NT tokens: RT x NT tiles of v_mfma_f32_32x32x16.
//   * K goes in groups of four steps, eight blocks of 32 inputs: lane (r, h) =
//     (lane % 32, lane / 32) takes blocks 4 h .. 4 h + 3 of the group, whose
//     scales are one word, and step u multiplies block 4 h + u: its 16 bytes of
//     codes give the operands of four instructions, s taking codes 8 s .. 8 s +
//     7, so that the activation operand is the 16 bytes of inputs 8 s of the
//     same block of the lane's token. (The sum over K does not care which
//     inputs meet in an instruction, so no code ever changes lanes.)
//   * Activations go from memory straight to LDS three steps ahead, into one
//     of four stages, codes to registers two steps ahead. LDS rows are 128
//     bytes (blocks u and 4 + u) and 16-byte chunk j of row t lies at chunk
//     j ^ ((t >> 1) & 7), so that the 16 lanes of an LDS pass touch 16
//     distinct groups of banks.
//   * Where there are few tiles the K steps are split over workgroups whose
//     float32 sums go to the workspace, as the accumulator registers lie, and
//     a second kernel adds them in a fixed order.
#include <algorithm>

#include "mx_device.hpp"

namespace aqlm {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;

// Byte offset of 16-byte chunk j of activation row t in an LDS buffer.
__device__ __forceinline__ uint32_t x_off(int t, int j) {
  return (uint32_t)t * 128u + (uint32_t)((j ^ ((t >> 1) & 7)) << 4);
}

struct TileArgs {
  const uint8_t *codes;
  const uint8_t *scales;
  const uint16_t *x;
  uint16_t *y;
  float4_t *part;  // [splits][tiles][RT * NT * 4][threads], or null
  int rows, cols, batch;
  int row_tiles, tok_tiles, splits, groups_per_split;
};

// Workgroup -> tile. Workgroups go round the 8 XCDs in turn, each with an L2
// of its own: give every XCD one run of consecutive tiles, tokens fastest, so
// that the workgroups at work on an XCD share rows of W and steps of x.
__device__ __forceinline__ int xcd_tile(int b, int n) {
  const int per = n >> 3, rest = n & 7, xcd = b & 7, i = b >> 3;
  return xcd * per + min(xcd, rest) + i;
}

template <MxType T, int RT, int NT>
__global__ __launch_bounds__(kThreads, 2) void mx_tile_kernel(const TileArgs A) {
  // one array per stage: the compiler then knows which loads into LDS a read
  // of LDS can depend on
  __shared__ __attribute__((aligned(16))) uint8_t xt0[NT * 32 * 128], xt1[NT * 32 * 128],
      xt2[NT * 32 * 128], xt3[NT * 32 * 128];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int tiles = A.row_tiles * A.tok_tiles;
  const int job = xcd_tile((int)blockIdx.x, tiles * A.splits);
  // (uniform, but divisions run on the vector unit: back to scalar registers)
  const int split = __builtin_amdgcn_readfirstlane(job / tiles), tile = job - split * tiles;
  const int row_tile = __builtin_amdgcn_readfirstlane(tile / A.tok_tiles);
  const int tok0 = (tile - row_tile * A.tok_tiles) * (32 * NT);
  const int row0 = (row_tile * kWaves + wave) * (32 * RT);
  const int nb = A.cols >> 5;
  const int g0 = split * A.groups_per_split;
  const int g1 = min((nb + 7) >> 3, g0 + A.groups_per_split);

  // resources that end with the tile's last row: rows past it read zero
  const uint32_t half = (uint32_t)A.cols >> 1;
  const int wave_rows = __builtin_amdgcn_readfirstlane(max(0, min(32 * RT, A.rows - row0)));
  const int tile_toks = __builtin_amdgcn_readfirstlane(min(32 * NT, A.batch - tok0));
  const Rsrc crs = make_rsrc(A.codes + (int64_t)row0 * half, (uint32_t)wave_rows * half);
  const Rsrc srs = make_rsrc(A.scales + (int64_t)row0 * nb, (uint32_t)wave_rows * nb);
  const Rsrc xrs = make_rsrc(A.x + (int64_t)tok0 * A.cols, (uint32_t)tile_toks * A.cols * 2u);

  float16_t acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // A step's activations, straight into LDS: each load of a wavefront fills 1
  // KiB (eight rows) in lane order, so a chunk's place in its row is chosen by
  // where the lane reads from. Chunks past the last block are zeros.
  const int xrow = tid >> 3, xj = (tid & 7) ^ ((tid >> 4) & 7);
  auto load_x = [&](int g, int u, uint8_t *dst) __attribute__((always_inline)) {
    const int blk = 8 * g + u + (xj & 4);
    const bool in = (g < g1) & (blk < nb);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint32_t off = (uint32_t)(xrow + 32 * i) * (uint32_t)A.cols * 2u + (uint32_t)blk * 64u +
                           16u * (xj & 3);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xrs, (__attribute__((address_space(3))) void *)(dst + i * 4096 + wave * 1024), 16,
          in ? off : kMxOOB, 0, 0, 0);
    }
  };
  auto load_w = [&](int g, int u, uint4 (&wv)[RT]) __attribute__((always_inline)) {
    const int blk = 8 * g + 4 * h + u;
    const bool in = (g < g1) & (blk < nb);
#pragma unroll
    for (int i = 0; i < RT; ++i)
      wv[i] = buf_load16(crs, in ? (32u * i + l32) * half + (uint32_t)blk * 16u : kMxOOB);
  };
  // The four scale bytes of a group. Past the last row or block the codes are
  // zeros and the byte is that of the last one there is, so that it is one of
  // this row (or of a row that is not stored) and needs no care: only a NaN
  // would show, in a row that is NaN already.
  uint32_t srow[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) srow[i] = (uint32_t)max(0, min(32 * i + l32, wave_rows - 1)) * nb;
  const bool whole = (nb & 7) == 0;  // whole groups: every word aligned and inside its row
  auto load_s = [&](int g, uint32_t (&sv)[RT]) __attribute__((always_inline)) {
    const int blk = 8 * min(g, g1 - 1) + 4 * h;
    if (whole) {
#pragma unroll
      for (int i = 0; i < RT; ++i) sv[i] = buf_load4(srs, srow[i] + (uint32_t)blk);
    } else {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        uint32_t v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = buf_load_u8(srs, srow[i] + (uint32_t)min(blk + u, nb - 1));
        sv[i] = v[0] | (v[1] << 8) | (v[2] << 16) | (v[3] << 24);
      }
    }
  };

  // One step. `X` holds its activations; `far` is the stage that the step
  // before read and the third one from here reads. Before the barrier the
  // wavefront waits for the next step's codes `w1` (the empty asm uses them):
  // loads return in order, and those were asked for a step after the next
  // step's activations, so these lie in LDS. The operand reads of this step
  // have long returned, since products used them.
  auto step = [&](auto wide_c, int g, auto u_c, const uint8_t *X, uint8_t *far,
                  const uint4 (&wv)[RT], const uint32_t (&sv)[RT], uint4 (&w1)[RT], uint4 (&w2)[RT])
                  __attribute__((always_inline)) {
    constexpr bool WIDE = decltype(wide_c)::value;
    constexpr int U = decltype(u_c)::value;
    load_w(U < 2 ? g : g + 1, (U + 2) & 3, w2);
    load_x(U < 1 ? g : g + 1, (U + 3) & 3, far);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (!WIDE) {
      uint4 b[2][NT];
      auto reads = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
          b[s & 1][j] = *reinterpret_cast<const uint4 *>(X + x_off(32 * j + l32, 4 * h + s));
      };
      reads(0);
      __builtin_amdgcn_sched_group_barrier(0x100, NT, 0);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s < 3) reads(s + 1);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const uint32_t ww[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
          const uint4 a = mx_decode8<T>(ww[s], mx_scale((sv[i] >> (8 * U)) & 0xFFu));
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = mx_mfma32<T>(a, b[s & 1][j], acc[i][j]);
        }
        if (s < 3) {  // the next instruction's operands are read before this one's products
          __builtin_amdgcn_sched_group_barrier(0x100, NT, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, RT * NT, 0);
        }
      }
    } else {
#pragma unroll 1
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint4 hi, lo;
          split_f16(*reinterpret_cast<const uint4 *>(X + x_off(32 * j + l32, 4 * h + s)), hi, lo);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const uint32_t word = s == 0 ? wv[i].x : s == 1 ? wv[i].y : s == 2 ? wv[i].z : wv[i].w;
            const uint4 a =
                mx_decode8<MxType::kBF16>(word, mx_scale((sv[i] >> (8 * U)) & 0xFFu));
            acc[i][j] = mx_mfma32<MxType::kBF16>(a, hi, acc[i][j]);
            acc[i][j] = mx_mfma32<MxType::kBF16>(a, lo, acc[i][j]);
          }
        }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < RT; ++i) asm volatile("" : "+v"(w1[i].x) : : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  uint4 w[4][RT];
  uint32_t sc[RT], sn[RT];
  load_s(g0, sc);
  load_x(g0, 0, xt0);
  __builtin_amdgcn_sched_barrier(0);
  load_w(g0, 0, w[0]);
  load_x(g0, 1, xt1);
  __builtin_amdgcn_sched_barrier(0);
  load_w(g0, 1, w[1]);
  load_x(g0, 2, xt2);
#pragma unroll
  for (int i = 0; i < RT; ++i) asm volatile("" : "+v"(w[0][i].x) : : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
  typedef std::integral_constant<int, 0> U0;
  typedef std::integral_constant<int, 1> U1;
  typedef std::integral_constant<int, 2> U2;
  typedef std::integral_constant<int, 3> U3;
  auto group = [&](auto wide_c, int g) __attribute__((always_inline)) {
    load_s(g + 1, sn);
    step(wide_c, g, U0{}, xt0, xt3, w[0], sc, w[1], w[2]);
    step(wide_c, g, U1{}, xt1, xt0, w[1], sc, w[2], w[3]);
    step(wide_c, g, U2{}, xt2, xt1, w[2], sc, w[3], w[0]);
    step(wide_c, g, U3{}, xt3, xt2, w[3], sc, w[0], w[1]);
#pragma unroll
    for (int i = 0; i < RT; ++i) sc[i] = sn[i];
  };
  int g = g0;
  for (; g < g1; ++g) {
    if constexpr (T == MxType::kF16) {
      bool f = true;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) f = f & mx_fits_f16((sc[i] >> (8 * u)) & 0xFFu);
      if (!__all(f) & (wave_rows > 0)) break;
    }
    group(std::false_type{}, g);
  }
  // From the wavefront's first group with a scale that float16 weights cannot
  // take: the same product in bfloat16, which holds every weight, with x split
  // exactly in two. The barriers are those of the other loop, one a step, so
  // wavefronts in either meet.
  if constexpr (T == MxType::kF16)
    for (; g < g1; ++g) group(std::true_type{}, g);
  // the zeros past the last group are in LDS before the wavefront can end
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");

  // register 4 g + e of a 32 x 32 tile: row 8 g + 4 h + e, token l32
  if (A.splits > 1) {
    float4_t *p = A.part + (int64_t)job * (RT * NT * 4 * kThreads) + tid;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          p[((i * NT + j) * 4 + g) * kThreads] = float4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1],
                                                          acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
    return;
  }
  const bool packed = (A.rows & 3) == 0;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int tok = tok0 + 32 * j + l32;
    if (tok >= A.batch) continue;
    uint16_t *row = A.y + (int64_t)tok * A.rows;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        store4<T>(row, row0 + 32 * i + 8 * g + 4 * h, A.rows,
                  float4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                           acc[i][j][4 * g + 3]},
                  packed);
  }
}

// Sums of the split parts, in order of the split, rounded and stored.
template <MxType T, int RT, int NT>
__global__ __launch_bounds__(kThreads) void mx_tile_sum_kernel(const TileArgs A) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles = A.row_tiles * A.tok_tiles;
  const int slot = (int)blockIdx.x % (RT * NT * 4), tile = (int)blockIdx.x / (RT * NT * 4);
  const float4_t *p = A.part + ((int64_t)tile * (RT * NT * 4) + slot) * kThreads + tid;
  const int64_t stride = (int64_t)tiles * (RT * NT * 4) * kThreads;
  float4_t v = p[0];
  for (int s = 1; s < A.splits; ++s) v += p[s * stride];
  const int g = slot & 3, j = (slot >> 2) % NT, i = (slot >> 2) / NT;
  const int row_tile = tile / A.tok_tiles;
  const int tok = (tile - row_tile * A.tok_tiles) * (32 * NT) + 32 * j + (lane & 31);
  const int row = (row_tile * kWaves + wave) * (32 * RT) + 32 * i + 8 * g + 4 * (lane >> 5);
  if (tok < A.batch) store4<T>(A.y + (int64_t)tok * A.rows, row, A.rows, v, (A.rows & 3) == 0);
}

// Tile of a product: rows of W per wavefront in units of 32, tokens in units
// of 32, workgroups K is split over.
struct Plan {
  int rt, nt, splits, groups_per_split;
  int64_t row_tiles, tok_tiles;
};

Plan plan_of(int64_t rows, int64_t cols, int64_t batch) {
  Plan p;
  p.nt = batch <= 32 ? 1 : batch <= 64 ? 2 : batch <= 96 ? 3 : 4;
  p.rt = 2;
  p.tok_tiles = (batch + 32 * p.nt - 1) / (32 * p.nt);
  p.row_tiles = (rows + 32 * kWaves * p.rt - 1) / (32 * kWaves * p.rt);
  if (p.row_tiles * p.tok_tiles < 256) {
    p.rt = 1;
    p.row_tiles = (rows + 32 * kWaves - 1) / (32 * kWaves);
  }
  const int64_t groups = (cols / 32 + 7) / 8, tiles = p.row_tiles * p.tok_tiles;
  // about two workgroups per CU, at least two groups of K steps each
  int64_t s = std::max<int64_t>(1, std::min<int64_t>(512 / tiles, groups / 2));
  if (tiles >= 192) s = 1;
  p.groups_per_split = (int)((groups + s - 1) / s);
  p.splits = (int)((groups + p.groups_per_split - 1) / p.groups_per_split);
  return p;
}

template <MxType T, int RT, int NT>
hipError_t launch_tile(const TileArgs &A, hipStream_t stream) {
  const unsigned tiles = (unsigned)(A.row_tiles * A.tok_tiles);
  hipLaunchKernelGGL((mx_tile_kernel<T, RT, NT>), dim3(tiles * A.splits), dim3(kThreads), 0, stream,
                     A);
  if (A.splits > 1)
    hipLaunchKernelGGL((mx_tile_sum_kernel<T, RT, NT>), dim3(tiles * RT * NT * 4), dim3(kThreads), 0,
                       stream, A);
  return hipGetLastError();
}

template <MxType T> hipError_t tile_as(const Plan &p, const TileArgs &A, hipStream_t stream) {
  switch (p.rt * 8 + p.nt) {
    case 9: return launch_tile<T, 1, 1>(A, stream);
    case 10: return launch_tile<T, 1, 2>(A, stream);
    case 11: return launch_tile<T, 1, 3>(A, stream);
    case 12: return launch_tile<T, 1, 4>(A, stream);
    case 17: return launch_tile<T, 2, 1>(A, stream);
    case 18: return launch_tile<T, 2, 2>(A, stream);
    case 19: return launch_tile<T, 2, 3>(A, stream);
    default: return launch_tile<T, 2, 4>(A, stream);
  }
}

}  // namespace

int64_t mx_gemm_tile_ws_bytes(const MxDesc &W, int64_t batch) {
  const Plan p = plan_of(W.rows, W.cols, batch);
  if (p.splits == 1) return 0;
  return p.row_tiles * p.tok_tiles * p.splits * (int64_t)(p.rt * p.nt * 4 * kThreads) *
         (int64_t)sizeof(float4_t);
}

hipError_t launch_mx_gemm_tile(const MxDesc &W, const void *x, int64_t batch, void *y, MxType type,
                               void *ws, hipStream_t stream) {
  const Plan p = plan_of(W.rows, W.cols, batch);
  TileArgs A;
  A.codes = W.codes;
  A.scales = W.scales;
  A.x = static_cast<const uint16_t *>(x);
  A.y = static_cast<uint16_t *>(y);
  A.part = static_cast<float4_t *>(ws);
  A.rows = (int)W.rows;
  A.cols = (int)W.cols;
  A.batch = (int)batch;
  A.row_tiles = (int)p.row_tiles;
  A.tok_tiles = (int)p.tok_tiles;
  A.splits = p.splits;
  A.groups_per_split = p.groups_per_split;
  return type == MxType::kF16 ? tile_as<MxType::kF16>(p, A, stream)
                              : tile_as<MxType::kBF16>(p, A, stream);
}

}  // namespace aqlm
