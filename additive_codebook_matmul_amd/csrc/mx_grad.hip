// Input gradient of a microscaled layer: dx = dy . W, one workgroup per
// [columns of W] x [tokens] tile (mx_tile.hpp, its rows being W's columns).
//
// The sum runs over the rows of W, along which neither codes nor scales are
// contiguous, while a matrix instruction wants eight consecutive terms of the
// sum in a lane.
//   * A K step is 64 rows of W. Each thread loads one block of one row (16
//     bytes of codes, its scale byte), expands it with one conversion for two
//     weights and writes 32 halves to LDS, row by row: every weight of a tile
//     is expanded once.
//   * ds_read_b64_tr_b16 transposes on the way back: 16 lanes give the places
//     of 4 rows x 16 columns and each receives four rows of one column, so two
//     reads make an operand of v_mfma_f32_32x32x16. Rows are 64 bytes longer
//     than their 256 RT of weights, which spreads four rows x 32 columns over
//     all banks; the threads that write take the four chunks of a block in
//     different orders, so that eight of them hit all banks.
//   * dy goes from memory straight to LDS three steps ahead, into one of four
//     stages of 128-byte rows, permuted as in the other tile kernels.
//   * float16: a workgroup that meets a scale that float16 weights cannot take
//     starts again, expanding to bfloat16, which holds every weight, and with
//     dy split exactly in two.
// dy's rows must be whole 16-byte chunks: with rows % 8 != 0 they are first
// copied into the workspace with zeros behind them.
#include <algorithm>

#include "mx_tile.hpp"

namespace aqlm {
namespace {

// Byte offset of 16-byte chunk j (of 8) of token t in a stage of dy.
__device__ __forceinline__ uint32_t row_off(int t, int j) {
  return (uint32_t)t * 128u + (uint32_t)((j ^ ((t >> 1) & 7)) << 4);
}

typedef short short4_vt __attribute__((ext_vector_type(4)));

// A.rows: columns of W (the result's); A.cols: rows of W (the sum's length);
// A.x: dy, [batch][dy_stride].
template <MxType T, int RT, int NT, int TW, int KW>
__global__ __launch_bounds__(64 * kRowWaves * TW * KW) void mx_grad_tile_kernel(const TileArgs A,
                                                                                const int dy_stride) {
  constexpr int kWaves = kRowWaves * TW, kThreads = 64 * kWaves;  // of one share of K
  constexpr int kCols = kRowWaves * RT * 32;                      // of W in the tile
  constexpr int kRowBytes = kCols * 2 + 64;
  constexpr int kXBytes = TW * NT * 32 * 128, kWBytes = 64 * kRowBytes;
  constexpr int kSums = tile_sums_bytes<RT, NT, TW>();
  constexpr int kArray = KW == 1 || KW * kXBytes > kSums ? KW * kXBytes : kSums;
  static_assert(64 * kCols / 32 == kThreads, "one block a thread and step");
  static_assert(KW * kWBytes >= kWaves * kStoreBytes<RT>, "room for the results");
  // one array per stage: the compiler then knows which loads into LDS a read
  // of LDS can depend on
  __shared__ __attribute__((aligned(16))) uint8_t xa0[kArray], xa1[kArray], xa2[kArray], xa3[kArray];
  __shared__ __attribute__((aligned(16))) uint8_t wa0[KW * kWBytes], wa1[KW * kWBytes];
  __shared__ uint32_t flags[kWaves * KW];
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = KW == 1 ? 0 : wave_all / kWaves, wave = KW == 1 ? wave_all : wave_all % kWaves;
  const int rw = wave / TW, tw = wave % TW;
  const int l32 = lane & 31, h = lane >> 5;
  const int tiles = A.row_tiles * A.tok_tiles;
  const int job = xcd_job((int)blockIdx.x, tiles * A.splits);
  const int split = __builtin_amdgcn_readfirstlane(job / tiles);
  const TilePlace at = tile_place(job - split * tiles, A.row_tiles, A.tok_tiles);
  const int col0 = at.row_tile * kCols, tok0 = at.tok_tile * (32 * NT * TW);
  const int out = A.cols, cols = A.rows;

  // K goes in groups of four steps, 256 rows of W. The groups of this split,
  // and of those the wavefront's: each of the KW shares takes as many turns as
  // the largest (past its end with zeros), so that all meet at every barrier.
  const int s0 = split * A.groups_per_split, s1 = min((out + 255) >> 8, s0 + A.groups_per_split);
  const int share = (s1 - s0 + KW - 1) / KW;
  const int g0 = s0 + kw * share, g1 = min(s1, g0 + share), gend = g0 + share;
  const int oend = min(out, 256 * g1);  // the share's rows end here

  const int tile_toks = __builtin_amdgcn_readfirstlane(min(32 * NT * TW, A.batch - tok0));
  const Rsrc xrs = make_rsrc(static_cast<const uint16_t *>(A.x) + (int64_t)tok0 * dy_stride,
                             (uint32_t)tile_toks * (uint32_t)dy_stride * 2u);

  float16_t acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // dy of step t (of group t / 4), rows 64 t .. 64 t + 63 of W, into a stage
  constexpr int kXLoads = NT;
  static_assert(kXLoads <= 4, "places of a lane's loads");
  uint32_t xoff[4];
  int xo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * (wave + i * kWaves) + (lane >> 3), j = (lane & 7) ^ ((r >> 1) & 7);
    xo[i] = 8 * j;
    xoff[i] = (uint32_t)r * (uint32_t)dy_stride * 2u + 16u * j;
  }
  auto fill_x = [&](int t, uint8_t *a) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xrs, (__attribute__((address_space(3))) void *)(a + (kw * kXBytes + (wave + i * kWaves) * 1024)), 16,
          xoff[i] + (64 * t + xo[i] < oend ? (uint32_t)t * 128u : kMxOOB), 0, 0, 0);
  };

  // the thread's block of step t: row 64 t + wo, block wb of the tile's columns
  const int tid = wave * 64 + lane, wo = tid / (kCols / 32), wb = tid % (kCols / 32);
  const uint32_t half = (uint32_t)cols >> 1, nb = (uint32_t)cols >> 5;
  const uint32_t cplace = col0 + 32 * wb < cols ? wo * half + (uint32_t)(col0 >> 1) + 16u * wb : kMxOOB;
  const uint32_t splace = col0 + 32 * wb < cols ? wo * nb + (uint32_t)(col0 >> 5) + wb : kMxOOB;
  struct Block {
    uint4 c;
    uint32_t s;
  };
  auto load_w = [&](int t, Block &b) __attribute__((always_inline)) {
    // resources of the step's rows: past the last they read zero
    const int64_t o = 64 * (int64_t)t;
    const int rows = __builtin_amdgcn_readfirstlane(max(0, min(64, oend - 64 * t)));
    b.c = buf_load16(make_rsrc(A.codes + (rows > 0 ? o * half : 0), (uint32_t)rows * half), cplace);
    b.s = buf_load_u8(make_rsrc(A.scales + (rows > 0 ? o * nb : 0), (uint32_t)rows * nb), splace);
  };
  // (A write takes the chunks of eight lanes at once, which are to lie in eight
  // places of 128 bytes: lanes two blocks apart write their four chunks in
  // another order, turned by `turn`; the words change places first.)
  const int turn = kCols == 256 ? (wb >> 1) & 3 : ((wb >> 1) & 1) | ((wo & 1) << 1);
  const uint32_t turn1 = turn & 1 ? ~0u : 0u, turn2 = turn & 2 ? ~0u : 0u;
  const uint32_t wplace = kw * kWBytes + wo * kRowBytes + wb * 64;
  auto put_w = [&](const Block &b, uint8_t *a, auto wide_c) __attribute__((always_inline)) {
    constexpr MxType E = decltype(wide_c)::value ? MxType::kBF16 : T;
    uint32_t w[4] = {b.c.x, b.c.y, b.c.z, b.c.w}, v[4], u[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = (w[c ^ 1] & turn1) | (w[c] & ~turn1);
#pragma unroll
    for (int c = 0; c < 4; ++c) u[c] = (v[c ^ 2] & turn2) | (v[c] & ~turn2);
    const float s = mx_scale(b.s);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      *reinterpret_cast<uint4 *>(a + (wplace + 16u * (c ^ turn))) = mx_decode8<E>(u[c], s);
    }
  };

  auto unfit = [&](int t, const Block &b) __attribute__((always_inline)) {
    return !mx_fits_f16(b.s) & (64 * t + wo < oend) & (cplace != kMxOOB);
  };

  // places of the lane's operands
  const int e16 = lane & 15;
  const uint32_t wbase = kw * kWBytes + (8 * h + (e16 >> 2)) * kRowBytes +
                         (rw * 32 * RT + 16 * ((lane >> 4) & 1) + 4 * (e16 & 3)) * 2;
  uint32_t xbase[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) xbase[s] = kw * kXBytes + row_off(tw * 32 * NT + l32, 2 * s + h);
  auto w_of = [&](const uint8_t *a, int i, int s) __attribute__((always_inline)) {
    typedef __attribute__((address_space(3))) short4_vt *LdsPtr;
    const short4_vt lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(a + (wbase + (16 * s) * kRowBytes + 64u * i)));
    const short4_vt hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(a + (wbase + (16 * s + 4) * kRowBytes + 64u * i)));
    const uint2 l = __builtin_bit_cast(uint2, lo), u = __builtin_bit_cast(uint2, hi);
    return make_uint4(l.x, l.y, u.x, u.y);
  };
  auto x_of = [&](const uint8_t *a, int j, int s) __attribute__((always_inline)) {
    return *reinterpret_cast<const uint4 *>(a + (xbase[s] + 4096u * j));
  };

  // All of K. Step t, the U-th of its group, reads stage U of dy and stage U %
  // 2 of W; the stage of dy that the step before read is filled for step t + 3,
  // the other of W with step t + 1's rows, whose blocks were loaded two steps
  // before. Before the barrier the wavefront waits for its own writes and until
  // at most its loads of this step and the one before are under way: loads
  // complete in order, so behind the barrier step t + 1 lies in LDS.
  // False (for the whole workgroup, with the sums of no use) where float16
  // cannot take a scale.
  auto run = [&](auto wide_c) __attribute__((always_inline)) -> bool {
    constexpr bool WIDE = decltype(wide_c)::value;
    constexpr bool kLook = T == MxType::kF16 && !WIDE;
    Block blk[4];
    bool bad = false;
    // Operands of instruction s of a step, and its products. Those of a step's
    // last instruction come in the next step, while its first reads are under
    // way behind the barrier. (The first step's are zeros.)
    uint4 wv[2][RT], b[2][NT];
#pragma unroll
    for (int i = 0; i < RT; ++i) wv[1][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < NT; ++j) b[1][j] = make_uint4(0, 0, 0, 0);
    auto reads = [&](int s, const uint8_t *a, const uint8_t *w) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < RT; ++i) wv[s & 1][i] = w_of(w, i, s);
#pragma unroll
      for (int j = 0; j < NT; ++j) b[s & 1][j] = x_of(a, j, s);
    };
    auto products = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if constexpr (WIDE && T == MxType::kF16) {
            uint4 hi, lo;
            split_f16(b[s & 1][j], hi, lo);
            acc[i][j] = mx_mfma32<MxType::kBF16>(wv[s & 1][i], hi, acc[i][j]);
            acc[i][j] = mx_mfma32<MxType::kBF16>(finite_bf16(wv[s & 1][i]), lo, acc[i][j]);
          } else {
            acc[i][j] = mx_mfma32<T>(wv[s & 1][i], b[s & 1][j], acc[i][j]);
          }
        }
    };
    auto step = [&](int t, auto u_c, uint8_t *a, uint8_t *far, uint8_t *w, uint8_t *wfar)
                    __attribute__((always_inline)) {
      constexpr int U = decltype(u_c)::value;
      fill_x(t + 3, far);
      load_w(t + 3, blk[(U + 3) & 3]);
      __builtin_amdgcn_sched_barrier(0);
      reads(0, a, w);
      products(3);
      put_w(blk[(U + 1) & 3], wfar, wide_c);
      if constexpr (kLook) {
        bad = bad | unfit(t + 1, blk[(U + 1) & 3]);
        if (U == 3) {
          const uint64_t any = __ballot(bad);
          if (lane == 0) flags[wave_all] = any != 0;
        }
      }
      if constexpr (!WIDE || T != MxType::kF16) {
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * RT + NT, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, (RT * NT + 1) / 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, RT * NT - (RT * NT + 1) / 2, 0);
      }
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        reads(s + 1, a, w);
        products(s);
        // the next instruction's operands are read before this one's products,
        // a chunk of the next rows written between them
        if constexpr (!WIDE || T != MxType::kF16) {
          __builtin_amdgcn_sched_group_barrier(0x100, 2 * RT + NT, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, (RT * NT + 1) / 2, 0);
          __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, RT * NT - (RT * NT + 1) / 2, 0);
        }
      }
      // (keeps the products in their step: nothing else ties them to a place)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j][0] = materialize(acc[i][j][0]);
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "i"(2 * (kXLoads + 2)) : "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" : : : "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    fill_x(4 * g0, xa0);
    load_w(4 * g0, blk[0]);
    __builtin_amdgcn_sched_barrier(0);
    fill_x(4 * g0 + 1, xa1);
    load_w(4 * g0 + 1, blk[1]);
    __builtin_amdgcn_sched_barrier(0);
    fill_x(4 * g0 + 2, xa2);
    load_w(4 * g0 + 2, blk[2]);
    __builtin_amdgcn_sched_barrier(0);
    put_w(blk[0], wa0, wide_c);
    if constexpr (kLook) bad = unfit(4 * g0, blk[0]);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "i"(2 * (kXLoads + 2)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
    bool good = true;
    for (int g = g0; g < gend; ++g) {
      const int t = 4 * g;
      step(t, std::integral_constant<int, 0>{}, xa0, xa3, wa0, wa1);
      step(t + 1, std::integral_constant<int, 1>{}, xa1, xa0, wa1, wa0);
      step(t + 2, std::integral_constant<int, 2>{}, xa2, xa1, wa0, wa1);
      step(t + 3, std::integral_constant<int, 3>{}, xa3, xa2, wa1, wa0);
      if constexpr (kLook) {
        uint32_t f = 0;
#pragma unroll
        for (int i = 0; i < kWaves * KW; ++i) f |= flags[i];
        good = __builtin_amdgcn_readfirstlane(f) == 0;
        if (!good) break;
      }
    }
    products(3);
    // what is under way has arrived before LDS is used again
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    __syncthreads();
    return good;
  };
  if (!run(std::integral_constant<bool, T != MxType::kF16>{})) {
    if constexpr (T == MxType::kF16) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
      run(std::true_type{});
    }
  }

  if (add_shares<RT, NT, TW, KW>(acc, kw, wave, lane, xa0, xa1, xa2, xa3)) return;
  store_tile<T, RT, NT, TW>(A, acc, job, at, wave, lane, wa0);
}

// dy with its rows moved to a stride of whole 16-byte chunks, zeros behind them.
__global__ __launch_bounds__(256) void mx_pad_rows_kernel(const uint16_t *__restrict__ in,
                                                          uint4 *__restrict__ to, int cols, int chunks) {
  const int c = (int)blockIdx.x * 256 + threadIdx.x;
  if (c >= chunks) return;
  const uint16_t *p = in + (int64_t)blockIdx.y * cols + 8 * c;
  uint32_t v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 8 * c + e < cols ? p[e] : 0u;
  to[(int64_t)blockIdx.y * chunks + c] = make_uint4(v[0] | (v[1] << 16), v[2] | (v[3] << 16),
                                                    v[4] | (v[5] << 16), v[6] | (v[7] << 16));
}

// Fitted, with the constants of plan_tiles, to 4096 x 4096, 4096 x 11008, 11008 x
// 4096 and 28672 x 8192 from 24 to 2048 rows, each shape measured at each: at
// 24 x 4096 x 4096 the three take 18.2, 12.3 and 10.8 us, at 100 x 11008 x 4096
// 29.3, 25.0 and 31.3, at 2048 x 11008 x 4096 164, 256 and 396.
constexpr TileShape kShapes[] = {
    {2, 2, 2, 1, 2.60, 0.89}, {1, 2, 1, 2, 2.38, 0.68}, {1, 1, 1, 2, 2.01, 0.43}};

TilePlan plan_of(const MxDesc &W, int64_t batch) {
  return plan_tiles(kShapes, W.cols, batch, (W.rows + 255) / 256);
}

// Bytes of the copy of dy that ragged rows need.
int64_t pad_bytes(const MxDesc &W, int64_t batch) {
  return W.rows % 8 == 0 ? 0 : batch * ((W.rows + 7) / 8) * 16;
}

template <MxType T, int RT, int NT, int TW, int KW>
hipError_t launch_tile(const TileArgs &A, int stride, hipStream_t stream) {
  const unsigned tiles = (unsigned)(A.row_tiles * A.tok_tiles);
  hipLaunchKernelGGL((mx_grad_tile_kernel<T, RT, NT, TW, KW>), dim3(tiles * A.splits),
                     dim3(64 * kRowWaves * TW * KW), 0, stream, A, stride);
  if (A.splits > 1)
    hipLaunchKernelGGL((mx_tile_sum_kernel<T, RT, NT, TW>), dim3(tiles * RT * NT * 4),
                       dim3(64 * kRowWaves * TW), 0, stream, A);
  return hipGetLastError();
}

template <MxType T>
hipError_t tile_as(const TileShape &c, const TileArgs &A, int stride, hipStream_t stream) {
  if (c.rt == 2) return launch_tile<T, 2, 2, 2, 1>(A, stride, stream);
  if (c.nt == 2) return launch_tile<T, 1, 2, 1, 2>(A, stride, stream);
  return launch_tile<T, 1, 1, 1, 2>(A, stride, stream);
}

}  // namespace

int64_t mx_grad_ws_bytes(const MxDesc &W, int64_t batch) {
  return plan_of(W, batch).ws_bytes() + pad_bytes(W, batch);
}

hipError_t launch_mx_grad(const MxDesc &W, const void *dy, int64_t batch, void *dx, MxType type, void *ws,
                          hipStream_t stream) {
  const TilePlan p = plan_of(W, batch);
  int64_t stride = W.rows;
  if (W.rows % 8 != 0) {  // behind the split sums
    stride = (W.rows + 7) / 8 * 8;
    uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(ws) + p.ws_bytes());
    const int chunks = (int)(stride / 8);
    for (int64_t b = 0; b < batch; b += 65535) {  // grid.y holds the tokens
      const unsigned n = (unsigned)std::min<int64_t>(batch - b, 65535);
      hipLaunchKernelGGL(mx_pad_rows_kernel, dim3((unsigned)(chunks + 255) / 256, n), dim3(256), 0, stream,
                         static_cast<const uint16_t *>(dy) + b * W.rows, to + b * chunks, (int)W.rows, chunks);
    }
    dy = to;
  }
  TileArgs A = tile_args(p, W, dy, nullptr, batch, dx, ws);
  A.rows = (int)W.cols;
  A.cols = (int)W.rows;
  return type == MxType::kF16 ? tile_as<MxType::kF16>(p.shape, A, (int)stride, stream)
                              : tile_as<MxType::kBF16>(p.shape, A, (int)stride, stream);
}

}  // namespace aqlm
