// Gradients of int8 layers and gated blocks with respect to the activations:
// dx = D . C, where C are the codes and D, [batch][rows] (GATED: both matrices'
// one after the other), the gradient of each product times its channel's scale:
//   a layer  D = dy w
//   gated    D = (dh u act'(g) w_gate, dh act(g) w_up)
// A term is float32 and a matrix instruction takes float16, so a term goes there as the
// sum of two. i8_grad_rows_kernel writes D once, each term times a power of two of the
// token's own that takes the largest magnitude to [2^14, 2^15): its nearest float16, and
// 2^11 times what that leaves, its nearest float16 too. The first is off by 2^-11 of the
// term at most, so the second leaves 2^-23 of it (or 2^-36, a 2^-50th of the token's
// largest, where it is subnormal): float32's own roundings are no smaller. The kernels
// after it multiply the first by the codes and the second by the codes times 2^-11, both of
// which float16 holds exactly, sum in float32 and take the power of two back. (One float16
// a term spares half of the instructions, 2048 x 11008 x 4096 193 to 203 us, and loses 2^-11
// of every term.)
// What bounds the product of many tokens is the card's power, as for the int8 products:
// with its terms' launch 2048 x 11008 x 4096 takes 335 to 355 us, and 239 with zeros for
// codes and gradients (gated 700 and 516): 1.1 PFLOP/s of float16 instructions. (The
// library's product of float16 matrices, half as many, 211.)
#include <algorithm>

#include "i8_tile.hpp"
#include "mx_tile.hpp"

namespace aqlm {
namespace {

struct I8GradRowsArgs {
  const void *dy;
  const float *g, *u;
  const float *ws[2];
  uint16_t *d;   // [batch][ld]: matrix m's part begins at 2 m part; 64 terms' first halves, then
                 // their second ones, zeros behind its rows
  int *power;    // [batch]
  int rows, part, ld;
  I8Act act;
};

// The terms of one row of the matrix (both matrices), before their power of two.
template <bool GATED>
__device__ __forceinline__ void grad_terms(const I8GradRowsArgs &A, float dy, float g, float u, float wg, float wu,
                                           float (&v)[GATED ? 2 : 1]) {
  if constexpr (GATED) {
    float a, slope;
    act_and_slope(A.act, g, a, slope);
    v[0] = dy * u * slope * wg;
    v[1] = dy * a * wu;
  } else {
    v[0] = dy * wg;
  }
}

template <MxType T> __device__ __forceinline__ float half_value(uint32_t h) {
  return T == MxType::kF16 ? h2f(h) : __builtin_bit_cast(float, h << 16);
}

// Bits of the largest finite magnitude.
__device__ __forceinline__ uint32_t finite_max(uint32_t top, float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? max(top, b) : top;
}

// Maximum over a workgroup of WAVES wavefronts; the power of two that takes it to
// [2^14, 2^15).
template <int WAVES> __device__ __forceinline__ int power_of(uint32_t top, uint32_t *tops) {
  top = wave_max(top);
  __syncthreads();  // the token before is done with `tops`
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES; ++w) top = max(top, tops[w]);
  return top == 0 ? 0 : 15 - __builtin_amdgcn_frexp_expf(__builtin_bit_cast(float, top));
}

// The two float16 numbers of a term, v times 2^power. (Infinity and NaN are the first's.)
__device__ __forceinline__ void split_term(float v, int power, uint32_t &first, uint32_t &second) {
  const float scaled = __builtin_amdgcn_ldexpf(v, power);
  first = f2h(scaled);
  second = (first & 0x7C00u) == 0x7C00u ? 0u : f2h((scaled - h2f(first)) * 0x1p11f);
}

// Where row i's first half lies in its matrix's part; the second is 64 further on.
__device__ __forceinline__ int term_at(int i) { return 2 * (i & ~63) + (i & 63); }

// A token a workgroup, 8 rows of the matrix a thread and round, the terms in
// registers between their maximum and their rounding: everything is read and written
// once, 16 bytes at a time. (rows a multiple of 8)
template <MxType T, bool GATED, int WAVES, int ROUNDS>
__global__ __launch_bounds__(WAVES * 64) void i8_grad_rows_kernel(const I8GradRowsArgs A, int64_t batch) {
  constexpr int M = GATED ? 2 : 1, kThreads = WAVES * 64;
  __shared__ uint32_t tops[WAVES];
  for (int64_t tok = blockIdx.x; tok < batch; tok += gridDim.x) {
    const int64_t at = tok * A.rows;
    float v[ROUNDS][M][8];
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const int i = 8 * ((int)threadIdx.x + r * kThreads);
      if (i < A.rows) {
        const uint4 h = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(A.dy) + at + i);
        const uint32_t w[4] = {h.x, h.y, h.z, h.w};
        float c[M][8], gu[2][8] = {};
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<float4_t *>(&c[m][4 * k]) = *reinterpret_cast<const float4_t *>(A.ws[m] + i + 4 * k);
        if constexpr (GATED) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            *reinterpret_cast<float4_t *>(&gu[0][4 * k]) = *reinterpret_cast<const float4_t *>(A.g + at + i + 4 * k);
            *reinterpret_cast<float4_t *>(&gu[1][4 * k]) = *reinterpret_cast<const float4_t *>(A.u + at + i + 4 * k);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float t[M];
          grad_terms<GATED>(A, half_value<T>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu), gu[0][e], gu[1][e], c[0][e],
                            c[M - 1][e], t);
#pragma unroll
          for (int m = 0; m < M; ++m) {
            v[r][m][e] = t[m];
            top = finite_max(top, t[m]);
          }
        }
      } else {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[r][m][e] = 0.f;
      }
    }
    const int e2 = power_of<WAVES>(top, tops);
    if (threadIdx.x == 0) A.power[tok] = -e2;
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const int i = 8 * ((int)threadIdx.x + r * kThreads);
      if (i < A.part) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
          uint32_t o[2][8];
#pragma unroll
          for (int e = 0; e < 8; ++e) split_term(v[r][m][e], e2, o[0][e], o[1][e]);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<uint4 *>(A.d + tok * A.ld + 2 * m * A.part + term_at(i) + 64 * k) =
                make_uint4(o[k][0] | (o[k][1] << 16), o[k][2] | (o[k][3] << 16), o[k][4] | (o[k][5] << 16),
                           o[k][6] | (o[k][7] << 16));
        }
      }
    }
  }
}

// Ragged rows, whose tokens begin anywhere, and more rows than registers hold: one row
// of the matrix a thread, computed twice.
template <MxType T, bool GATED>
__global__ __launch_bounds__(1024) void i8_grad_any_rows_kernel(const I8GradRowsArgs A, int64_t batch) {
  constexpr int M = GATED ? 2 : 1;
  __shared__ uint32_t tops[16];
  for (int64_t tok = blockIdx.x; tok < batch; tok += gridDim.x) {
    const int64_t at = tok * A.rows;
    auto terms = [&](int i, float(&v)[M]) __attribute__((always_inline)) {
      const float dy = half_value<T>(static_cast<const uint16_t *>(A.dy)[at + i]);
      grad_terms<GATED>(A, dy, GATED ? A.g[at + i] : 0.f, GATED ? A.u[at + i] : 0.f, A.ws[0][i], A.ws[M - 1][i], v);
    };
    uint32_t top = 0;
    for (int i = threadIdx.x; i < A.rows; i += 1024) {
      float v[M];
      terms(i, v);
#pragma unroll
      for (int m = 0; m < M; ++m) top = finite_max(top, v[m]);
    }
    const int e2 = power_of<16>(top, tops);
    if (threadIdx.x == 0) A.power[tok] = -e2;
    for (int i = threadIdx.x; i < A.part; i += 1024) {
      float v[M] = {};
      if (i < A.rows) terms(i, v);
#pragma unroll
      for (int m = 0; m < M; ++m) {
        uint32_t first, second;
        split_term(v[m], e2, first, second);
        uint16_t *const to = A.d + tok * A.ld + 2 * m * A.part + term_at(i);
        to[0] = (uint16_t)first;
        to[64] = (uint16_t)second;
      }
    }
  }
}

template <MxType T, bool GATED> void launch_terms(const I8GradRowsArgs &R, int64_t batch, hipStream_t stream) {
  const dim3 grid((unsigned)std::min<int64_t>(batch, 1 << 20));
  if (R.rows % 8 != 0 || R.part > 32768)
    hipLaunchKernelGGL((i8_grad_any_rows_kernel<T, GATED>), grid, dim3(1024), 0, stream, R, batch);
  else if (R.part <= 2048)
    hipLaunchKernelGGL((i8_grad_rows_kernel<T, GATED, 4, 1>), grid, dim3(256), 0, stream, R, batch);
  else if (R.part <= 4096)
    hipLaunchKernelGGL((i8_grad_rows_kernel<T, GATED, 4, 2>), grid, dim3(256), 0, stream, R, batch);
  else if (R.part <= 8192)
    hipLaunchKernelGGL((i8_grad_rows_kernel<T, GATED, 8, 2>), grid, dim3(512), 0, stream, R, batch);
  else if (R.part <= 16384)
    hipLaunchKernelGGL((i8_grad_rows_kernel<T, GATED, 16, 2>), grid, dim3(1024), 0, stream, R, batch);
  else
    hipLaunchKernelGGL((i8_grad_rows_kernel<T, GATED, 16, 4>), grid, dim3(1024), 0, stream, R, batch);
}

// The product D . C: one workgroup per [columns of C] x [tokens] tile. The sum runs
// over the rows of C, along which codes are not contiguous, while a matrix
// instruction wants eight consecutive terms of the sum in a lane.
//   * A K step is 64 rows of one matrix. Codes and D go from memory straight to LDS,
//     one or two steps ahead. 16-byte chunk c of row r of the codes lies at chunk
//     c ^ turn(r), so that the 32 lanes that read 8 rows x 32 columns at once touch
//     all banks; D's 128-byte rows, first halves and second, are permuted as in the other
//     tile kernels.
//   * ds_read_b64_tr_b8 transposes on the way out of LDS: 16 lanes give the places of
//     8 rows x 16 columns and each receives eight rows of one column, which is one
//     side of v_mfma_f32_32x32x16_f16 but for the type.
//   * A code becomes float16 in registers: its bits with the sign bit turned, below
//     the exponent of 1024, are 1152 more than it, exactly; times 2^-11 it is one still.
//     14 instructions for the eight terms of a lane, between the products of the chunk
//     before.
struct I8GradArgs {
  const int8_t *w[2];
  const uint16_t *d;  // [batch][ld]
  const int *power;
  uint16_t *dx;       // [batch][cols]
  float4_t *part;     // [splits][tiles][RT * NT * 4][64 RW TW], or null
  int rows, part_rows, ld, cols, batch, matrices;
  int col_tiles, tok_tiles, splits, steps_per_split;
};

// Where chunk c of row r of the codes lies: c ^ turn.
template <int COLS> __device__ __forceinline__ int turn_of(int r) {
  static_assert(COLS == 256 || COLS == 128, "16 or 8 chunks a row");
  return COLS == 256 ? 2 * (r & 7) : 2 * ((r >> 1) & 3);
}

// Eight codes as float16, and times 2^-11.
__device__ __forceinline__ void codes_to_f16(const uint2 &c, uint4 &whole, uint4 &small) {
  const uint32_t in[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
  const half2_t off = {(_Float16)-1152.0f, (_Float16)-1152.0f}, by = {(_Float16)0x1p-11f, (_Float16)0x1p-11f};
  uint32_t r[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = __builtin_amdgcn_perm(0x64646464u, in[i >> 1], i & 1 ? 0x04030402u : 0x04010400u);
    const half2_t code = __builtin_bit_cast(half2_t, v) + off;
    r[i] = __builtin_bit_cast(uint32_t, code);
    s[i] = __builtin_bit_cast(uint32_t, code * by);
  }
  whole = make_uint4(r[0], r[1], r[2], r[3]);
  small = make_uint4(s[0], s[1], s[2], s[3]);
}

template <MxType T, class S>
__global__ __launch_bounds__(S::kThreads *S::KW) void i8_grad_kernel(const I8GradArgs A) {
  constexpr int RT = S::RT, NT = S::NT, TW = S::TW, KW = S::KW, kWaves = S::kWaves, kCols = S::kCols;
  constexpr int kStage = S::kStage, kWBytes = S::kWBytes, kXBytes = S::kXBytes;
  constexpr int kArray = S::kArray;
  // one array per stage: the compiler then knows which loads into LDS a read
  // of LDS can depend on
  __shared__ __attribute__((aligned(16))) uint8_t s0[kArray], s1[kArray], s2[S::STAGES > 2 ? kArray : 16];
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = KW == 1 ? 0 : wave_all / kWaves, wave = KW == 1 ? wave_all : wave_all % kWaves;
  const int rw = wave / TW, tw = wave % TW;
  const int l32 = lane & 31, h = lane >> 5;
  const int tiles = A.col_tiles * A.tok_tiles;
  const int job = xcd_job((int)blockIdx.x, tiles * A.splits);
  const int split = __builtin_amdgcn_readfirstlane(job / tiles);
  const TilePlace at = tile_place(job - split * tiles, A.col_tiles, A.tok_tiles);
  const int col0 = at.row_tile * kCols, tok0 = at.tok_tile * S::kToks;
  const uint32_t cols = (uint32_t)A.cols;

  // The steps of this split, and of those the wavefront's: each of the KW shares
  // takes as many as the largest (past its end with zeros), so that all meet at
  // every barrier. Steps go through the first matrix, then the second.
  const int per = A.part_rows >> 6;  // steps of a matrix
  const int t0 = split * A.steps_per_split, t1 = min(per * A.matrices, t0 + A.steps_per_split);
  const int share = (t1 - t0 + KW - 1) / KW;
  const int g0 = t0 + kw * share, g1 = min(t1, g0 + share), gend = g0 + share;

  const int tile_toks = __builtin_amdgcn_readfirstlane(min(S::kToks, A.batch - tok0));
  const Rsrc xrs = make_rsrc(A.d + (int64_t)tok0 * A.ld, (uint32_t)tile_toks * (uint32_t)A.ld * 2u);

  float16_t acc[RT][NT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const int wcol0 = col0 + rw * 32 * RT, wtok0 = tok0 + tw * 32 * NT;
  int power[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) power[j] = A.power[min(wtok0 + 32 * j + l32, A.batch - 1)];

  // Step t into a stage: loads of a wavefront fill 1 KiB in lane order, 1024 /
  // kCols rows of codes or eight tokens.
  constexpr int kWLoads = 64 * kCols / 1024 / kWaves, kXLoads = S::kToks / 8 / kWaves;  // (of each half)
  constexpr int kLoads = kWLoads + 2 * kXLoads;
  constexpr int kLoadRows = 1024 / kCols, kRowLanes = kCols / 16;
  static_assert(64 * kCols % (1024 * kWaves) == 0 && S::kToks % (8 * kWaves) == 0, "loads");
  static_assert(kWLoads <= 8 && kXLoads <= 8, "places of a lane's loads");
  uint32_t woff[8], xoff[8];
#pragma unroll
  for (int i = 0; i < kWLoads; ++i) {
    const int r = (wave + i * kWaves) * kLoadRows + lane / kRowLanes;
    const int c = (lane % kRowLanes) ^ turn_of<kCols>(r);
    woff[i] = col0 + 16 * c < A.cols ? (uint32_t)r * cols + (uint32_t)(col0 + 16 * c) : kMxOOB;
  }
#pragma unroll
  for (int i = 0; i < kXLoads; ++i) {
    const int r = 8 * (wave + i * kWaves) + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
    xoff[i] = (uint32_t)r * (uint32_t)A.ld * 2u + 16u * c;
  }
  typedef __attribute__((address_space(3))) void *LdsPtr;
  auto fill = [&](int t, uint8_t *a) __attribute__((always_inline)) {
    // a resource of the step's rows: past the last they read zero
    const bool second = t >= per;
    const int o = 64 * (second ? t - per : t);
    const int rows = __builtin_amdgcn_readfirstlane(t < g1 ? max(0, min(64, A.rows - o)) : 0);
    const int8_t *const base = second ? A.w[1] : A.w[0];
    const Rsrc wrs = make_rsrc(base + (rows > 0 ? (int64_t)o * cols : 0), (uint32_t)rows * cols);
    const uint32_t k = t < g1 ? (uint32_t)t * 256u : kMxOOB;
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wrs, (LdsPtr)(a + (kw * kStage + (wave + i * kWaves) * 1024)), 16,
                                               woff[i], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            xrs, (LdsPtr)(a + (kw * kStage + kWBytes + p * kXBytes + (wave + i * kWaves) * 1024)), 16,
            xoff[i] + k + 128u * p, 0, 0, 0);
  };

  // places of the lane's operands: 16 further rows of codes, 32 further columns or
  // tokens are at the same permutation but for the columns' chunk
  const int e16 = lane & 15, er = 8 * h + (e16 >> 1);  // row (of 16), and the lane's half chunk
  uint32_t wbase[4], xbase[4];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int c = (rw * 32 * RT + 32 * i) / 16 + ((lane >> 4) & 1);
    wbase[i] = kw * kStage + er * kCols + ((c ^ turn_of<kCols>(er)) << 4) + 8 * (e16 & 1);
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int t = tw * 32 * NT + l32;
    xbase[s] = kw * kStage + kWBytes + t * 128 + (((2 * s + h) ^ ((t >> 1) & 7)) << 4);
  }
  static_assert(RT <= 4, "places of the operands");
  uint2 raw[2][RT];
  uint4 w[2][2][RT], b[2][2][NT];  // [chunk's parity][first or second halves]
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int i = 0; i < RT; ++i) w[1][p][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < NT; ++j) b[1][p][j] = make_uint4(0, 0, 0, 0);
  }
  auto read_w = [&](const uint8_t *a, int s) __attribute__((always_inline)) {
    typedef int int2_vt __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) int2_vt *TrPtr;
#pragma unroll
    for (int i = 0; i < RT; ++i)
      raw[s & 1][i] = __builtin_bit_cast(
          uint2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((TrPtr)(a + (wbase[i] + (uint32_t)(16 * s * kCols)))));
  };
  auto read_x = [&](const uint8_t *a, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        b[s & 1][p][j] = *reinterpret_cast<const uint4 *>(a + (xbase[s] + (uint32_t)(p * kXBytes) + 4096u * j));
  };
  auto convert = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RT; ++i) codes_to_f16(raw[s & 1][i], w[s & 1][0][i], w[s & 1][1][i]);
  };
  auto products = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mx_mfma32<MxType::kF16>(w[s & 1][p][i], b[s & 1][p][j], acc[i][j]);
  };
  // Step t from stage `a`. `far` is the stage that the step before read, filled for
  // step t + STAGES - 1. Codes are read two chunks ahead and converted one ahead; the
  // products of a step's last chunk come behind the barrier, while the first reads of
  // the next step are under way. (The first step's are zeros.) Before the barrier the
  // wavefront waits for its own reads and until at most STAGES - 2 steps' loads are
  // under way: loads complete in order, so behind it step t + 1 lies in LDS.
  auto step = [&](int t, const uint8_t *a, uint8_t *far) __attribute__((always_inline)) {
    fill(t + S::STAGES - 1, far);
    __builtin_amdgcn_sched_barrier(0);
    read_w(a, 0);
    read_w(a, 1);
    products(3);
    read_x(a, 0);
    convert(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      read_x(a, s + 1);
      if (s < 2) read_w(a, s + 2);
      products(s);
      convert(s + 1);
      __builtin_amdgcn_sched_group_barrier(0x100, 2 * NT, 0);
      if (s < 2) __builtin_amdgcn_sched_group_barrier(0x100, RT, 0);
#pragma unroll
      for (int k = 0; k < 2 * RT * NT; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, (14 + 2 * NT - 1) / (2 * NT), 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // (keeps the products in their step: nothing else ties them to a place)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j][0] = materialize(acc[i][j][0]);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "i"((S::STAGES - 2) * kLoads) : "memory");
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
  asm volatile("s_waitcnt vmcnt(%0)" : : "i"((S::STAGES - 2) * kLoads) : "memory");
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

  if (i8_join_shares<S>(acc, kw, wave, lane, s0)) return;
  if (A.splits > 1) return i8_store_part<S>(acc, A.part, job, wave, lane, wtok0, A.batch);

  // 32 tokens of the wavefront at a time (columns are a multiple of 16)
  uint8_t *const mine = S::STAGES == 2 ? s1 + wave * S::kStore
                                       : (wave & 1 ? s2 : s1) + (wave >> 1) * S::kStore;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    float4_t out[RT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) out[i][q][e] = materialize(__builtin_amdgcn_ldexpf(acc[i][j][4 * q + e], power[j]));
    i8_store_lines<T>(out, mine, lane, A.dx, wtok0 + 32 * j, wcol0, A.batch, A.cols);
  }
}

// Sums of the split parts, in order of the split, and the results.
template <MxType T, class S>
__global__ __launch_bounds__(S::kThreads) void i8_grad_sum_kernel(const I8GradArgs A) {
  constexpr int RT = S::RT, NT = S::NT;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles = A.col_tiles * A.tok_tiles;
  const int slot = (int)blockIdx.x % (RT * NT * 4), tile = (int)blockIdx.x / (RT * NT * 4);
  const int q = slot & 3, j = (slot >> 2) % NT, i = (slot >> 2) / NT;
  const TilePlace at = tile_place(tile, A.col_tiles, A.tok_tiles);
  const int tok = at.tok_tile * S::kToks + (wave % S::TW) * 32 * NT + 32 * j + (lane & 31);
  const int col = at.row_tile * S::kCols + (wave / S::TW) * 32 * RT + 32 * i + 8 * q + 4 * (lane >> 5);
  if (tok >= A.batch || col >= A.cols) return;
  const float4_t *p = A.part + ((int64_t)tile * (RT * NT * 4) + slot) * S::kThreads + tid;
  const int64_t stride = (int64_t)tiles * (RT * NT * 4) * S::kThreads;
  float4_t v = i8_sum_parts(p, stride, A.splits);
  const int power = A.power[tok];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = materialize(__builtin_amdgcn_ldexpf(v[e], power));
  store4<T>(A.dx + (int64_t)tok * A.cols, col, A.cols, v, true);
}

template <MxType T, class S> hipError_t launch_shape(const I8GradArgs &A, hipStream_t stream) {
  const unsigned tiles = (unsigned)(A.col_tiles * A.tok_tiles);
  hipLaunchKernelGGL((i8_grad_kernel<T, S>), dim3(tiles * A.splits), dim3(S::kThreads * S::KW), 0, stream, A);
  if (A.splits > 1)
    hipLaunchKernelGGL((i8_grad_sum_kernel<T, S>), dim3(tiles * S::RT * S::NT * 4), dim3(S::kThreads), 0, stream, A);
  return hipGetLastError();
}

template <MxType T> hipError_t grad_as(const I8Grad &p, const I8Plan &g, void *ws, hipStream_t stream) {
  const int part = (int)i8_term_rows(p.W.rows), ld = 2 * part * (p.gated() ? 2 : 1);
  int *const power = static_cast<int *>(ws);
  uint16_t *const d = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(ws) + i8_terms_at(p.batch));
  const I8GradRowsArgs R = {p.dy, p.g, p.u, {p.W.scales, p.up.scales}, d, power, (int)p.W.rows, part, ld, p.act};
  if (p.gated()) launch_terms<T, true>(R, p.batch, stream);
  else launch_terms<T, false>(R, p.batch, stream);
  float4_t *const sums = reinterpret_cast<float4_t *>(static_cast<uint8_t *>(ws) + i8_grad_sums_at(p.W.rows, p.gated(), p.batch));
  const I8GradArgs A = {{p.W.codes, p.up.codes}, d, power, static_cast<uint16_t *>(p.dx), sums, (int)p.W.rows, part, ld,
                        (int)p.W.cols, (int)p.batch, p.gated() ? 2 : 1, (int)g.across, (int)g.tok_tiles, g.splits,
                        g.steps_per_split};
  using namespace i8_grad;  // (in the order of its costs)
  if (g.shape == 0) return launch_shape<T, Large>(A, stream);
  if (g.shape == 1) return launch_shape<T, Half>(A, stream);
  if (g.shape == 2) return launch_shape<T, Small>(A, stream);
  return launch_shape<T, Deep>(A, stream);
}

}  // namespace

hipError_t launch_i8_grad(const I8Grad &p, const I8Plan &plan, void *ws, hipStream_t stream) {
  return p.type == MxType::kF16 ? grad_as<MxType::kF16>(p, plan, ws, stream)
                                : grad_as<MxType::kBF16>(p, plan, ws, stream);
}

}  // namespace aqlm
