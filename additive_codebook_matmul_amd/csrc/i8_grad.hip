// Gradients of int8 layers and gated blocks with respect to the activations:
// dx = D . C, where C are the codes and D, [batch][rows] (GATED: both matrices'
// one after the other), the gradient of each product times its channel's scale:
//   a layer  D = dy w
//   gated    D = (dh u act'(g) w_gate, dh act(g) w_up)
// i8_grad_rows_kernel writes D once, as float16 times a power of two of the token's
// own that takes its largest magnitude to [2^14, 2^15), and the kernels after it
// multiply by the codes, which float16 holds exactly, sum in float32 and take the
// power of two back. A code is 8 bits and float16 has 11, so this rounding to 2^-12
// of the value is the only one before the last (bfloat16 gradients times float32
// scales would lose 2^-9 in bfloat16).
#include <algorithm>

#include "i8_device.hpp"

namespace aqlm {
namespace {

struct I8GradRowsArgs {
  const void *dy;
  const float *g, *u;
  const float *ws[2];
  uint16_t *d;   // [batch][ld]: matrix m's part begins at m * part, zeros behind its rows
  int *power;    // [batch]
  int rows, part, ld;
  I8Act act;
};

// D of row `i` of the matrix (both matrices), before its power of two.
template <MxType T, bool GATED>
__device__ __forceinline__ void grad_terms(const I8GradRowsArgs &A, int64_t at, int i, float (&v)[GATED ? 2 : 1]) {
  const uint16_t h = static_cast<const uint16_t *>(A.dy)[at + i];
  const float dy = T == MxType::kF16 ? h2f(h) : __builtin_bit_cast(float, (uint32_t)h << 16);
  if constexpr (GATED) {
    float a, slope;
    act_and_slope(A.act, A.g[at + i], a, slope);
    v[0] = dy * A.u[at + i] * slope * A.ws[0][i];
    v[1] = dy * a * A.ws[1][i];
  } else {
    v[0] = dy * A.ws[0][i];
  }
}

template <MxType T, bool GATED>
__global__ __launch_bounds__(256) void i8_grad_rows_kernel(const I8GradRowsArgs A, int64_t batch) {
  constexpr int M = GATED ? 2 : 1;
  __shared__ uint32_t tops[4];
  for (int64_t tok = blockIdx.x; tok < batch; tok += gridDim.x) {
    const int64_t at = tok * A.rows;
    uint32_t top = 0;  // of the finite ones
    for (int i = threadIdx.x; i < A.rows; i += 256) {
      float v[M];
      grad_terms<T, GATED>(A, at, i, v);
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v[m]) & 0x7FFFFFFFu;
        if (b < 0x7F800000u) top = max(top, b);
      }
    }
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    // largest = f 2^e, 1/2 <= f < 1: taken to [2^14, 2^15)
    int e = 0;
    if (top != 0) {
      const float f = __builtin_bit_cast(float, top);
      e = 15 - (__builtin_amdgcn_frexp_expf(f));
    }
    if (threadIdx.x == 0) A.power[tok] = -e;
    for (int i = threadIdx.x; i < A.part; i += 256) {
      float v[M] = {};
      if (i < A.rows) grad_terms<T, GATED>(A, at, i, v);
#pragma unroll
      for (int m = 0; m < M; ++m)
        A.d[tok * A.ld + m * A.part + i] = (uint16_t)f2h(__builtin_amdgcn_ldexpf(v[m], e));
    }
    __syncthreads();
  }
}

struct I8GradArgs {
  const int8_t *w[2];
  const uint16_t *d;  // [batch][ld]
  const int *power;
  uint16_t *dx;       // [batch][cols]
  int rows, part, ld, cols, batch, matrices;
};

// One workgroup: 64 columns of W by 64 tokens, 32 rows of W a step.
template <MxType T>
__global__ __launch_bounds__(256) void i8_grad_kernel(const I8GradArgs A) {
  __shared__ __attribute__((aligned(16))) uint16_t wt[64][40], xt[64][40];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col0 = (int)blockIdx.x * 64, tok0 = (int)blockIdx.y * 64;
  const int toks = __builtin_amdgcn_readfirstlane(min(64, A.batch - tok0));
  const Rsrc xrs = make_rsrc(A.d + (int64_t)tok0 * A.ld, (uint32_t)toks * (uint32_t)A.ld * 2u);
  float16_t acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
  for (int m = 0; m < A.matrices; ++m)
    for (int o0 = 0; o0 < A.part; o0 += 32) {
      const int rows = __builtin_amdgcn_readfirstlane(max(0, min(32, A.rows - o0)));
      const Rsrc wrs = make_rsrc(A.w[m] + (rows > 0 ? (int64_t)o0 * A.cols : 0), (uint32_t)rows * (uint32_t)A.cols);
      const int o = tid >> 3, c = 8 * (tid & 7);
      const uint2 b = buf_load8(wrs, col0 + c < A.cols ? (uint32_t)o * A.cols + col0 + c : kMxOOB);
      const uint4 d = buf_load16(xrs, (uint32_t)(tid >> 2) * A.ld * 2u + (uint32_t)(m * A.part + o0) * 2u + 16u * (tid & 3));
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e)
        wt[c + e][o] = (uint16_t)f2h((float)(int8_t)((e < 4 ? b.x : b.y) >> (8 * (e & 3))));
      *reinterpret_cast<uint4 *>(&xt[tid >> 2][8 * (tid & 3)]) = d;
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int k = 16 * s + 8 * (lane >> 5);
        const uint4 wv = *reinterpret_cast<const uint4 *>(&wt[32 * (wave & 1) + (lane & 31)][k]);
        const uint4 xv = *reinterpret_cast<const uint4 *>(&xt[32 * (wave >> 1) + (lane & 31)][k]);
        acc = mx_mfma32<MxType::kF16>(wv, xv, acc);
      }
    }
  const int tok = tok0 + 32 * (wave >> 1) + (lane & 31);
  if (tok >= A.batch) return;
  const int power = A.power[tok];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float4_t v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __builtin_amdgcn_ldexpf(acc[4 * q + e], power);
    store4<T>(A.dx + (int64_t)tok * A.cols, col0 + 32 * (wave & 1) + 8 * q + 4 * (lane >> 5), A.cols, v, true);
  }
}

// Rows of one matrix in D: whole steps.
int64_t part_of(const I8Desc &W) { return (W.rows + 63) / 64 * 64; }
// Workspace: the powers, then D, from multiples of 256 bytes on.
int64_t terms_at(int64_t batch) { return (batch * 4 + 255) / 256 * 256; }

template <MxType T> hipError_t grad_as(const I8Grad &p, void *ws, hipStream_t stream) {
  const int part = (int)part_of(p.W), ld = part * (p.gated() ? 2 : 1);
  int *const power = static_cast<int *>(ws);
  uint16_t *const d = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(ws) + terms_at(p.batch));
  const I8GradRowsArgs R = {p.dy, p.g, p.u, {p.W.scales, p.up.scales}, d, power, (int)p.W.rows, part, ld, p.act};
  const dim3 grid((unsigned)std::min<int64_t>(p.batch, 1 << 20));
  if (p.gated()) hipLaunchKernelGGL((i8_grad_rows_kernel<T, true>), grid, dim3(256), 0, stream, R, p.batch);
  else hipLaunchKernelGGL((i8_grad_rows_kernel<T, false>), grid, dim3(256), 0, stream, R, p.batch);
  const I8GradArgs A = {{p.W.codes, p.up.codes}, d, power, static_cast<uint16_t *>(p.dx), (int)p.W.rows, part, ld,
                        (int)p.W.cols, (int)p.batch, p.gated() ? 2 : 1};
  hipLaunchKernelGGL((i8_grad_kernel<T>), dim3((unsigned)((p.W.cols + 63) / 64), (unsigned)((p.batch + 63) / 64)),
                     dim3(256), 0, stream, A);
  return hipGetLastError();
}

}  // namespace

int64_t i8_grad_ws_bytes(const I8Desc &W, bool gated, int64_t batch) {
  return terms_at(batch) + batch * part_of(W) * (gated ? 2 : 1) * 2;
}

hipError_t launch_i8_grad(const I8Grad &p, void *ws, hipStream_t stream) {
  return p.type == MxType::kF16 ? grad_as<MxType::kF16>(p, ws, stream) : grad_as<MxType::kBF16>(p, ws, stream);
}

}  // namespace aqlm
