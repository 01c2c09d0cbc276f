// Products of int8 layers for up to four tokens and of gated blocks for up to eight:
// whole rows of W by a wavefront.
//
// Reading W bounds these (one token: a multiply and add for every byte), so that all
// serves a steady stream: a wavefront takes two rows at a time (GATED: a row of the
// gate and the same one of up, whose results meet there), its lanes 16 bytes each of
// 1 KiB of a row, two such chunks ahead, and v_dot4_i32_i8 adds them up beside the
// tokens' codes from LDS. The lanes' sums meet at a row's end.
// (One token: 28672 x 8192 gated 76 us, 6.2 TB/s, 8192 x 28672 39 with the token's
// quantisation, 6.0 TB/s, 11008 x 4096 gated 15.8, 5.7 TB/s.)
// HOLD > 0: x is halves, which every workgroup quantises on their way into LDS, while
// its threads hold HOLD octets of each token (i8_rows_quantize).
#include <algorithm>

#include "i8_gemm.hpp"

namespace aqlm {
namespace {

constexpr int kThreads = kI8RowThreads, kWaves = kThreads / 64;
constexpr int kMostLds = 65536;  // bytes of codes in LDS

// Bytes of codes of a token in LDS: all of them in whole chunks where they fit.
__host__ __device__ constexpr int segment_bytes(int cols, int b) {
  return (cols + 1023) / 1024 * 1024 <= kMostLds / b ? (cols + 1023) / 1024 * 1024 : kMostLds / b;
}

__device__ __forceinline__ int dot16(const uint4 &a, const uint4 &b, int c) {
  c = __builtin_amdgcn_sdot4((int)a.x, (int)b.x, c, false);
  c = __builtin_amdgcn_sdot4((int)a.y, (int)b.y, c, false);
  c = __builtin_amdgcn_sdot4((int)a.z, (int)b.z, c, false);
  return __builtin_amdgcn_sdot4((int)a.w, (int)b.w, c, false);
}

// Sum over the wavefront, in lane 63.
__device__ __forceinline__ int lanes_sum(int v) {
  auto step = [&](auto ctrl, auto rows) __attribute__((always_inline)) {
    v += __builtin_amdgcn_update_dpp(0, v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
  };
  step(std::integral_constant<int, kDppQuadXor1>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, kDppQuadXor2>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, kDppRowHalfMirror>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, kDppRowMirror>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, kDppRowBcast15>{}, std::integral_constant<int, 0xA>{});
  step(std::integral_constant<int, kDppRowBcast31>{}, std::integral_constant<int, 0xC>{});
  return v;
}

template <MxType T, bool GATED, int B, int HOLD>
__global__ __launch_bounds__(kThreads) void i8_rows_kernel(const I8Args A, const void *__restrict__ x) {
  constexpr int S = 2, kRows = GATED ? 1 : 2;  // streams, and rows of results, of a wavefront
  constexpr bool QUANT = HOLD > 0;
  extern __shared__ __attribute__((aligned(16))) uint8_t codes[];  // [B][seg]
  __shared__ uint32_t tops[B][kWaves];
  const int seg = segment_bytes(A.cols, B);
  const uint32_t cols = (uint32_t)A.cols;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row0 = ((int)blockIdx.x * kWaves + wave) * kRows;
  // resources of the wavefront's rows: past W's last they read zero
  const int8_t *const w0 = A.w[0] + (int64_t)min(row0, A.rows - 1) * cols;
  const int8_t *const w1 = GATED ? A.w[1] + (int64_t)min(row0, A.rows - 1) * cols
                                 : A.w[0] + (int64_t)min(row0 + 1, A.rows - 1) * cols;
  const Rsrc rs0 = make_rsrc(w0, row0 < A.rows ? cols : 0u);
  const Rsrc rs1 = make_rsrc(w1, row0 + (GATED ? 0 : 1) < A.rows ? cols : 0u);

  int acc[S][B];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int b = 0; b < B; ++b) acc[s][b] = 0;
  // chunks c and c + 1 of both rows (a resource ends with its row)
  uint4 w[2][2][S];
  auto load = [&](int c, uint4 (&v)[2][S]) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t at = (uint32_t)(c + k) * 1024u + 16u * lane;
      v[k][0] = buf_load16_nt(rs0, at);
      v[k][1] = buf_load16_nt(rs1, at);
    }
  };
  const int chunks = (A.cols + 1023) >> 10;

  const int octets = A.cols >> 3;
  RowScale rs[QUANT ? B : 1];
  Octet<T> held[QUANT ? B : 1][QUANT ? HOLD : 1];
  if constexpr (QUANT) {
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int u = 0; u < HOLD; ++u) {
        const int i = threadIdx.x + u * kThreads;
        if (i < octets) held[b][u] = load_octet<T, false>(x, (int64_t)min(b, A.batch - 1) * octets + i);
        else held[b][u] = {};
      }
  }
  load(0, w[0]);
  if constexpr (QUANT) {  // the tokens' scales
#pragma unroll
    for (int b = 0; b < B; ++b) {
      uint32_t m = 0;
#pragma unroll
      for (int u = 0; u < HOLD; ++u) m = max(m, octet_max<T>(held[b][u]));
      m = wave_max(m);
      if (lane == 0) tops[b][wave] = m;
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < B; ++b) {
      uint32_t t = tops[b][0];
#pragma unroll
      for (int k = 1; k < kWaves; ++k) t = max(t, tops[b][k]);
      rs[b] = row_scale(max_bits<T>(t));
    }
  }

  int k0 = 0;
  do {  // a segment of the tokens (QUANT: all of them)
    if (k0 > 0) __syncthreads();
    const int here = min(seg, A.cols - k0);
    if constexpr (QUANT) {
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int u = 0; u < HOLD; ++u) {
          const int i = threadIdx.x + u * kThreads;
          if (i < octets) *reinterpret_cast<uint2 *>(codes + b * seg + 8 * i) = encode_octet<T>(held[b][u], rs[b]);
        }
    } else {
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int8_t *const from = A.x + (int64_t)min(b, A.batch - 1) * cols + k0;
        for (int i = threadIdx.x; 16 * i < here; i += kThreads)
          *reinterpret_cast<uint4 *>(codes + b * seg + 16 * i) = *reinterpret_cast<const uint4 *>(from + 16 * i);
      }
    }
    __syncthreads();
    const int c0 = k0 >> 10, c1 = min(chunks, c0 + (seg >> 10));
    // (past the row's end the codes of W are zeros, whatever lies in LDS)
    auto turn = [&](int c, uint4 (&now)[2][S], uint4 (&next)[2][S]) __attribute__((always_inline)) {
      load(c + 2, next);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = min(c + k - c0, (seg >> 10) - 1) * 1024 + 16 * lane;
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const uint4 xv = *reinterpret_cast<const uint4 *>(codes + b * seg + at);
#pragma unroll
          for (int s = 0; s < S; ++s) acc[s][b] = dot16(now[k][s], xv, acc[s][b]);
        }
      }
    };
    for (int c = c0; c < c1; c += 4) {
      turn(c, w[0], w[1]);
      if (c + 2 < c1) turn(c + 2, w[1], w[0]);
      else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int s = 0; s < S; ++s) w[0][k][s] = w[1][k][s];
      }
    }
    k0 += seg;
  } while (!QUANT && k0 < A.cols);

  // lane b takes token b
  int sum[S] = {0, 0};
  float token = 0.f;
#pragma unroll
  for (int b = 0; b < B; ++b) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int v = __builtin_amdgcn_readlane(lanes_sum(acc[s][b]), 63);
      sum[s] = lane == b ? v : sum[s];
    }
    if constexpr (QUANT) token = lane == b ? rs[b].scale : token;
  }
  if (lane >= A.batch || row0 >= A.rows) return;
  if constexpr (!QUANT) token = A.xs[lane];
  const int64_t at = (int64_t)lane * A.rows + row0;
  if constexpr (GATED) {
    const float g = i8_value(sum[0], A.ws[0][row0], token), u = i8_value(sum[1], A.ws[1][row0], token);
    A.y[at] = (uint16_t)f2t<T>(materialize(act_value(A.act, g) * u));
    if (A.g) {
      A.g[at] = g;
      A.u[at] = u;
    }
  } else {
    A.y[at] = (uint16_t)f2t<T>(i8_value(sum[0], A.ws[0][row0], token));
    if (row0 + 1 < A.rows) A.y[at + 1] = (uint16_t)f2t<T>(i8_value(sum[1], A.ws[0][row0 + 1], token));
  }
}

template <MxType T, bool GATED, int B> void launch_b(const I8Args &A, const void *x, hipStream_t stream) {
  constexpr int kRows = kWaves * (GATED ? 1 : 2);
  const dim3 grid((unsigned)((A.rows + kRows - 1) / kRows));
  const unsigned lds = (unsigned)(B * segment_bytes(A.cols, B));
  if constexpr (B <= 4)
    if (x) {
      // (twice the octets cost registers: one token of 11008 x 4096 gated 17.2 us with
      // four and 18.0 with eight)
      constexpr int kHold = 4 / B;
      if (A.cols / 8 <= kHold * kThreads) {
        hipLaunchKernelGGL((i8_rows_kernel<T, GATED, B, kHold>), grid, dim3(kThreads), lds, stream, A, x);
        return;
      }
      if constexpr (B <= 2) {
        hipLaunchKernelGGL((i8_rows_kernel<T, GATED, B, 2 * kHold>), grid, dim3(kThreads), lds, stream, A, x);
        return;
      }
    }
  hipLaunchKernelGGL((i8_rows_kernel<T, GATED, B, 0>), grid, dim3(kThreads), lds, stream, A, x);
}

template <MxType T, bool GATED> hipError_t rows_as(const I8Args &A, const void *x, hipStream_t stream) {
  if (A.batch == 1) launch_b<T, GATED, 1>(A, x, stream);
  else if (A.batch == 2) launch_b<T, GATED, 2>(A, x, stream);
  else if (!GATED || A.batch <= 4) launch_b<T, GATED, 4>(A, x, stream);
  else if constexpr (GATED) launch_b<T, GATED, 8>(A, x, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_rows(const I8Args &A, const void *x, MxType type, bool gated, hipStream_t stream) {
  if (type == MxType::kF16)
    return gated ? rows_as<MxType::kF16, true>(A, x, stream) : rows_as<MxType::kF16, false>(A, x, stream);
  return gated ? rows_as<MxType::kBF16, true>(A, x, stream) : rows_as<MxType::kBF16, false>(A, x, stream);
}

}  // namespace aqlm
