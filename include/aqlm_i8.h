/*
 * aqlm_i8.h - C ABI of the 8-bit integer (int8) linear layers and gated
 * feed-forward blocks in libaqlm_mi355x.so: a third weight format beside the
 * codebook one of aqlm.h and the 4-bit floats of aqlm_mx.h, for layers that are
 * to lose less than those do. Weights and activations are both whole numbers with
 * one scale for each output channel and each token, which the integer matrix
 * instructions of gfx950 multiply and add without any rounding.
 *
 * Format. A matrix [rows][cols], cols a multiple of 16, is
 *   codes   [rows][cols] int8
 *   scales  [rows] float32
 *   value[r][c] = codes[r][c] * scales[r]
 * A layer's rows are its output channels, those of activations are tokens.
 *
 * Element types of dense operands: AQLM_I8_F16, AQLM_I8_BF16 and, for
 * quantisation and expansion, AQLM_I8_F32.
 *
 * A product's sum of codes is exact (in 32-bit integers, which is why cols is
 * limited to AQLM_I8_MAX_COLS); it is then taken to float32, multiplied by the
 * channel's scale and by the token's, and rounded once, to nearest even, to the
 * type of the result. The gradients sum in float32 in a fixed order. A scale that is
 * NaN makes its whole row or column of the result NaN, one that is an infinity
 * infinities, and NaN where the sum is zero.
 *
 * Pointers, streams and errors as in aqlm.h: every pointer is a device pointer
 * on the current HIP device (the structs are host memory), 16-byte aligned,
 * owned by the caller and dense row-major; arguments are validated on the host
 * before anything is enqueued; calls enqueue on `stream` and return without
 * synchronising; nothing is allocated and no state is kept. Outputs must not
 * overlap inputs, workspaces or each other. Results are deterministic: the same
 * call gives the same bits. Status codes are aqlm.h's (AQLM_ERR_TYPE for an
 * unknown element type or activation).
 *
 * Workspaces: at least the bytes that the entry point's *_workspace_size gives
 * for the same sizes, NULL where that is 0; overwritten. Calls that may overlap
 * in time need workspaces of their own. AQLM_ERR_WORKSPACE if workspace_bytes is
 * too small, AQLM_ERR_NULL if a workspace is needed and NULL.
 */
#ifndef AQLM_I8_H
#define AQLM_I8_H

#include <stdint.h>

#include "aqlm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest rows and batch of the products. */
#define AQLM_I8_MAX_DIM (1ll << 21)

/* Largest cols of the products: 2^14 a term, codes of -128 on both sides, stays
 * below 2^31 in the sum. */
#define AQLM_I8_MAX_COLS ((1ll << 17) - 16)

typedef enum aqlm_i8_type { AQLM_I8_F16 = 0, AQLM_I8_BF16 = 1, AQLM_I8_F32 = 2 } aqlm_i8_type;

/*
 * Activations of a gated block:
 *   SILU       g / (1 + e^-g)
 *   GELU       g Phi(g), Phi the normal distribution function
 *   GELU_TANH  g / (1 + e^-2z), z = sqrt(2/pi) (g + 0.044715 g^3), which is
 *              g (1 + tanh z) / 2
 */
typedef enum aqlm_i8_act { AQLM_I8_SILU = 0, AQLM_I8_GELU = 1, AQLM_I8_GELU_TANH = 2 } aqlm_i8_act;

/* An int8 matrix: sizes plus device pointers. */
typedef struct aqlm_i8_matrix {
  int64_t rows;        /* >= 1 (a layer's out_features) */
  int64_t cols;        /* >= 16, multiple of 16 (a layer's in_features) */
  const int8_t *codes; /* device, [rows][cols] */
  const float *scales; /* device, [rows] */
} aqlm_i8_matrix;

/*
 * aqlm_i8_quantize: codes and scales of the dense matrix x [rows][cols] of
 * `type`. With A the largest magnitude of a row, its scale is A / 127 (rounded
 * to float32) and a value's code the whole number nearest to 127 v / A, ties to
 * the even one, as if computed without error; codes lie in [-127, 127]. A row
 * of zeros has scale 0 and codes 0, a row that holds an infinity or a NaN scale
 * NaN and codes 0. rows == 0 is a no-op. rows < 2^31, cols < 2^31, rows * cols
 * < 2^40.
 */
AQLM_API int aqlm_i8_quantize(const void *x, int32_t type, int64_t rows, int64_t cols, int8_t *codes,
                              float *scales, void *stream);

/* aqlm_i8_dequant: the dense matrix W [rows][cols] of `type`: each code times
 * its scale in float32, rounded once more where the type needs it. */
AQLM_API int aqlm_i8_dequant(const aqlm_i8_matrix *m, int32_t type, void *W, void *stream);

/*
 * aqlm_i8_gemm: y [x->rows][W->rows] = x . W^T of two int8 matrices (x->cols ==
 * W->cols), y of `type` (F16 or BF16). x->rows may be 0 (no-op).
 */
AQLM_API int aqlm_i8_gemm_workspace_size(const aqlm_i8_matrix *W, int64_t batch, int64_t *bytes);
AQLM_API int aqlm_i8_gemm(const aqlm_i8_matrix *W, const aqlm_i8_matrix *x, void *y, int32_t type,
                          void *workspace, int64_t workspace_bytes, void *stream);

/*
 * aqlm_i8_gemm_quant: y [batch][rows] = Q(x) . W^T with x [batch][cols] of
 * `type` (F16 or BF16) quantised on the way, y of the same type: the bits of
 * aqlm_i8_quantize and aqlm_i8_gemm, in one call. batch == 0 is a no-op.
 */
AQLM_API int aqlm_i8_gemm_quant_workspace_size(const aqlm_i8_matrix *W, int64_t batch, int64_t *bytes);
AQLM_API int aqlm_i8_gemm_quant(const aqlm_i8_matrix *W, const void *x, int64_t batch, void *y,
                                int32_t type, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * aqlm_i8_gated: h [batch][rows] = act(g) * u with g = Q(x) . gate^T and u =
 * Q(x) . up^T, the first half of a gated feed-forward block in one pass: both
 * products, the activation and their product stay in float32 and are rounded
 * once, to `type`. gate and up have the same sizes. g and u, both given or both
 * NULL, receive the float32 products [batch][rows], for aqlm_i8_gated_grad.
 * batch == 0 is a no-op.
 */
AQLM_API int aqlm_i8_gated_workspace_size(const aqlm_i8_matrix *gate, const aqlm_i8_matrix *up,
                                          int64_t batch, int64_t *bytes);
AQLM_API int aqlm_i8_gated(const aqlm_i8_matrix *gate, const aqlm_i8_matrix *up, const void *x,
                           int64_t batch, int32_t act, void *h, float *g, float *u, int32_t type,
                           void *workspace, int64_t workspace_bytes, void *stream);

/*
 * aqlm_i8_grad_input: dx [batch][cols] = dy [batch][rows] . W, the gradient of
 * aqlm_i8_gemm_quant with respect to x through the (constant) weights and
 * straight through the quantisation; dy and dx of `type` (F16 or BF16). The terms,
 * each token's gradients times the channels' scales, are float32 and enter the
 * matrix instructions as the sum of two float16 numbers, relative to a power of two
 * of the token's own: off by at most 2^-23 of the term, or 2^-50 of the token's
 * largest one, whatever its magnitude.
 * rows need not be a multiple of anything; batch == 0 is a no-op.
 */
AQLM_API int aqlm_i8_grad_input_workspace_size(const aqlm_i8_matrix *W, int64_t batch, int64_t *bytes);
AQLM_API int aqlm_i8_grad_input(const aqlm_i8_matrix *W, const void *dy, int64_t batch, void *dx,
                                int32_t type, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * aqlm_i8_gated_grad: dx [batch][cols] = (dh u act'(g)) . gate + (dh act(g)) .
 * up, the gradient of aqlm_i8_gated with respect to x, from the g and u it gave
 * and dh [batch][rows]; dh and dx of `type` (F16 or BF16). Arithmetic as in
 * aqlm_i8_grad_input. batch == 0 is a no-op.
 */
AQLM_API int aqlm_i8_gated_grad_workspace_size(const aqlm_i8_matrix *gate, const aqlm_i8_matrix *up,
                                               int64_t batch, int64_t *bytes);
AQLM_API int aqlm_i8_gated_grad(const aqlm_i8_matrix *gate, const aqlm_i8_matrix *up, const float *g,
                                const float *u, const void *dh, int64_t batch, int32_t act, void *dx,
                                int32_t type, void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* AQLM_I8_H */
