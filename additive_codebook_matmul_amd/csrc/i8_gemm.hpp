// What the kernels of int8 products share.
#pragma once

#include "i8_device.hpp"

namespace aqlm {

struct I8Args {
  const int8_t *w[2];     // the layer, or gate and up
  const float *ws[2];
  const int8_t *x;        // [batch][cols]
  const float *xs;
  uint16_t *y;
  float *g, *u;           // or null
  int rows, cols, batch;
  I8Act act;
};

// Results of four consecutive rows, from `row` on, of token `tok`.
template <MxType T, bool GATED>
__device__ __forceinline__ void i8_store4(const I8Args &A, int tok, int row, const int4_vt (&sums)[GATED ? 2 : 1]) {
  const float token = A.xs[tok];
  const int64_t at = (int64_t)tok * A.rows;
  float v[GATED ? 2 : 1][4], out[4];
#pragma unroll
  for (int m = 0; m < (GATED ? 2 : 1); ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[m][e] = i8_value(sums[m][e], A.ws[m][min(row + e, A.rows - 1)], token);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (GATED) out[e] = materialize(act_value(A.act, v[0][e]) * v[1][e]);
    else out[e] = v[0][e];
  }
  if constexpr (GATED) {
    if (A.g) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (row + e < A.rows) {
          A.g[at + row + e] = v[0][e];
          A.u[at + row + e] = v[1][e];
        }
    }
  }
  store4<T>(A.y + at, row, A.rows, float4_t{out[0], out[1], out[2], out[3]}, (A.rows & 3) == 0);
}

// Few tokens by whole rows of W (i8_rows.hip), up to four of a layer and kI8RowTokens
// of a gated block; x: halves to be quantised on
// the way, for sizes that i8_rows_quantize takes, or null where A.x and A.xs are given.
hipError_t launch_i8_rows(const I8Args &A, const void *x, MxType type, bool gated, hipStream_t stream);

// The tile kernels (i8_tile.hip).
hipError_t launch_i8_tile(const I8Args &A, const I8Plan &p, MxType type, bool gated, void *ws, hipStream_t stream);

}  // namespace aqlm
