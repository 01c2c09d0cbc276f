// Internal declarations of the int8 translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

// How a tile kernel does a product or a gradient.
struct I8Plan {
  int shape, splits, steps_per_split;
  int64_t across, tok_tiles;  // tiles of W's rows (a gradient: of its columns), and of tokens
  int64_t sums;               // bytes of the split parts' sums in the workspace
  double us;                  // modelled duration
};

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
// The kernels of a product (`quant`: x is halves), by its sizes: chosen once a call,
// since a choice takes the host a microsecond.
struct I8Route {
  enum Kind { kRows, kSkinny, kTiles } kind;
  bool inside;  // the product's own workgroups quantise x
  I8Plan plan;  // kTiles
  int64_t ws_bytes;
};
I8Route i8_route(const I8Desc &W, bool gated, int64_t batch, bool quant);
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
I8Plan i8_grad_plan(const I8Desc &W, bool gated, int64_t batch);
int64_t i8_grad_ws_bytes(const I8Desc &W, bool gated, int64_t batch, const I8Plan &plan);
hipError_t launch_i8_grad(const I8Grad &p, const I8Plan &plan, void *ws, hipStream_t stream);

}  // namespace aqlm
