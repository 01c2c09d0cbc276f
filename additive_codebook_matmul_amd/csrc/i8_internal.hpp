// Internal declarations of the int8 translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "i8_plan.hpp"
#include "mx_internal.hpp"

namespace aqlm {

// Dense element types are MxType's (aqlm_i8_type has the same values).

// Values of aqlm_i8_act.
enum class I8Act : int { kSilu = 0, kGelu = 1, kGeluTanh = 2 };

struct I8Desc {
  int64_t rows, cols;   // cols a multiple of 16
  const int8_t *codes;  // [rows][cols]
  const float *scales;  // [rows]
};

hipError_t launch_i8_quantize(const void *x, MxType type, int64_t rows, int64_t cols, int8_t *codes,
                              float *scales, hipStream_t stream);
hipError_t launch_i8_dequant(const I8Desc &m, MxType type, void *W, hipStream_t stream);

// A product of one layer, or the two of a gated block (up.codes not null).
struct I8Product {
  I8Desc W;   // the layer, or the gate
  I8Desc up;  // sizes of W's, or none
  I8Act act;
  const void *x;           // halves to be quantised, or null where the codes are given
  const int8_t *xcodes;    // given codes [batch][cols]
  const float *xscales;
  int64_t batch;
  void *y;                 // [batch][rows]
  float *g, *u;            // [batch][rows] or null
  MxType type;
  bool gated() const { return up.codes != nullptr; }
};
hipError_t launch_i8_product(const I8Product &p, const I8Route &route, void *ws, hipStream_t stream);

// The gradient with respect to the activations: of a layer (up.codes null, g
// and u unused) or a gated block.
struct I8Grad {
  I8Desc W, up;
  I8Act act;
  const float *g, *u;
  const void *dy;  // [batch][rows]
  int64_t batch;
  void *dx;        // [batch][cols]
  MxType type;
  bool gated() const { return up.codes != nullptr; }
};
hipError_t launch_i8_grad(const I8Grad &p, const I8Plan &plan, void *ws, hipStream_t stream);

}  // namespace aqlm
