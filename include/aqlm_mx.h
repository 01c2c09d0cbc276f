/*
 * aqlm_mx.h - C ABI of the microscaled 4-bit (MXFP4) linear layers in
 * libaqlm_mi355x.so: a second weight format beside the codebook one of aqlm.h.
 * Where a codebook layer spends a learned codebook and an encoder's search on
 * each matrix, this one rounds every weight by itself to a 4-bit float, at 4.25
 * bits a weight, which the matrix instructions of gfx950 take as it is.
 *
 * Format ("OCP Microscaling Formats (MX) Specification", version 1.0, MXFP4).
 * A matrix [rows][cols], cols a multiple of 32, is
 *   codes   [rows][cols/2] uint8: two E2M1 codes a byte, the even column in
 *           bits 0..3, the odd one in bits 4..7. Bit 3 of a code is the sign,
 *           bits 0..2 select 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   scales  [rows][cols/32] uint8: one E8M0 byte for each 32 consecutive
 *           columns of a row; byte s stands for 2^(s - 127), and 255 for NaN.
 *   value[r][c] = e2m1(code[r][c]) * 2^(scales[r][c/32] - 127)
 * and every value of a block whose byte is 255 is NaN (zeros too).
 *
 * Element types of dense operands: AQLM_MX_F16, AQLM_MX_BF16 and, for
 * quantisation and expansion, AQLM_MX_F32.
 *
 * Products accumulate in float32 in a fixed order and round once, to nearest
 * even, to the type of the result. A weight enters a product as the value
 * above, exactly, whatever its scale (with float16 activations too, whose
 * type cannot hold every such value). In the products with half activations
 * and in the gradient magnitudes from 2^128 on are infinities (scale bytes 253
 * and 254; aqlm_mx_quantize writes 253 by its CEIL rule alone, for blocks that
 * reach above 6 * 2^125, and 254 never); where both sides are microscaled they
 * keep their value, and only a sum can overflow.
 * NaN and infinities propagate as in a dense product, also from activations.
 *
 * Pointers, streams and errors as in aqlm.h: every pointer is a device pointer
 * on the current HIP device (the arrays of pointers and structs are host
 * memory), 16-byte aligned, owned by the caller and dense row-major; arguments
 * are validated on the host before anything is enqueued; calls enqueue on
 * `stream` and return without synchronising; nothing is allocated and no state
 * is kept. Outputs must not overlap inputs, workspaces or each other. Results
 * are deterministic: the same call gives the same bits. Status codes are
 * aqlm.h's (AQLM_ERR_TYPE for an unknown element type or scale rule).
 */
#ifndef AQLM_MX_H
#define AQLM_MX_H

#include <stdint.h>

#include "aqlm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Values that share one scale. */
#define AQLM_MX_BLOCK 32

/* Largest rows, cols and batch of the products. */
#define AQLM_MX_MAX_DIM (1ll << 21)

typedef enum aqlm_mx_type { AQLM_MX_F16 = 0, AQLM_MX_BF16 = 1, AQLM_MX_F32 = 2 } aqlm_mx_type;

/*
 * How aqlm_mx_quantize chooses a block's power of two from its largest
 * magnitude A:
 *   FLOOR  2^(floor(log2 A) - 2), the specification's rule: A / scale lies in
 *          [4, 8), and what exceeds 6 there is held as 6
 *   CEIL   the smallest power of two with A / scale <= 6: nothing is clipped
 */
typedef enum aqlm_mx_rule { AQLM_MX_SCALE_FLOOR = 0, AQLM_MX_SCALE_CEIL = 1 } aqlm_mx_rule;

/* A microscaled matrix: sizes plus device pointers. */
typedef struct aqlm_mx_matrix {
  int64_t rows;          /* >= 1 (a layer's out_features) */
  int64_t cols;          /* >= 32, multiple of 32 (a layer's in_features) */
  const uint8_t *codes;  /* device, [rows][cols/2] */
  const uint8_t *scales; /* device, [rows][cols/32] */
} aqlm_mx_matrix;

/*
 * aqlm_mx_quantize: codes and scales of the dense matrix x [rows][cols] of
 * `type`. Each value goes to the nearest E2M1 multiple of its block's scale,
 * ties to the even code, the sign kept (of zeros too), magnitudes above 6
 * scales to 6. A block of zeros has byte 127 (2^0), a block that holds an
 * infinity or a NaN byte 255 and codes 0; scales below 2^-127 are held as
 * 2^-127. rows == 0 is a no-op. rows * cols must stay below 2^40.
 */
AQLM_API int aqlm_mx_quantize(const void *x, int32_t type, int64_t rows, int64_t cols,
                              int32_t rule, uint8_t *codes, uint8_t *scales, void *stream);

/*
 * aqlm_mx_dequant: the dense matrix W [rows][cols] of `type`, each value
 * rounded once to nearest even (exact for float32 and bfloat16 but for
 * overflow to infinity; float16 also rounds below 2^-24).
 */
AQLM_API int aqlm_mx_dequant(const aqlm_mx_matrix *m, int32_t type, void *W, void *stream);

/*
 * aqlm_mx_gemv_batched: y[i] = x[i] . W_i^T for num_layers layers in one call,
 * 0 <= batch <= 8 activation rows each. W, x and y are HOST arrays of
 * num_layers entries (at most 4096); x[i] is [batch][cols_i] and y[i]
 * [batch][rows_i], both of `type` (F16 or BF16). x[i] may be shared. Up to 16
 * layers go into one launch, but large ones that a tile kernel serves better
 * (from three rows on) into one each. Results are bit-identical to calls with one
 * layer.
 */
AQLM_API int aqlm_mx_gemv_batched(const aqlm_mx_matrix *W, const void *const *x, void *const *y,
                                  int32_t num_layers, int64_t batch, int32_t type, void *stream);

/*
 * aqlm_mx_gemm: y [batch][rows] = x [batch][cols] . W^T for any batch
 * (0: no-op), x and y of `type` (F16 or BF16). Up to 2 rows it gives
 * aqlm_mx_gemv_batched's bits; from 3 on it may split K over workgroups, which
 * that entry point, without a workspace, does not. Weights are expanded in
 * registers on their way to the matrix instructions and never written.
 *   workspace  at least aqlm_mx_gemm_workspace_size bytes (NULL where that is
 *              0): float32 partial sums where K is split over workgroups;
 *              overwritten. Calls that may overlap in time need workspaces of
 *              their own.
 * Returns AQLM_ERR_WORKSPACE if workspace_bytes is too small, AQLM_ERR_NULL if
 * a workspace is needed and NULL.
 */
AQLM_API int aqlm_mx_gemm_workspace_size(const aqlm_mx_matrix *W, int64_t batch, int64_t *bytes);
AQLM_API int aqlm_mx_gemm(const aqlm_mx_matrix *W, const void *x, int64_t batch, void *y,
                          int32_t type, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * aqlm_mx_gemm_mx: y [x->rows][W->rows] = x . W^T where both sides are
 * microscaled (x->cols == W->cols), on the block-scaled matrix instructions,
 * y of `type` (F16 or BF16). x->rows may be 0 (no-op). Workspace as above.
 */
AQLM_API int aqlm_mx_gemm_mx_workspace_size(const aqlm_mx_matrix *W, int64_t batch,
                                            int64_t *bytes);
AQLM_API int aqlm_mx_gemm_mx(const aqlm_mx_matrix *W, const aqlm_mx_matrix *x, void *y,
                             int32_t type, void *workspace, int64_t workspace_bytes,
                             void *stream);

/*
 * aqlm_mx_gemm_quant: y [batch][rows] = Q(x) . W^T with x [batch][cols] of
 * `type` (F16 or BF16) quantised by aqlm_mx_quantize's `rule` on the way, y of
 * the same type: aqlm_mx_quantize and aqlm_mx_gemm_mx in one call, with
 * their bits but at 3 to 5 rows, where the sums may be added in another order.
 * batch == 0 is a no-op. Workspace as above, the activations' codes and scales
 * among it where they are written.
 */
AQLM_API int aqlm_mx_gemm_quant_workspace_size(const aqlm_mx_matrix *W, int64_t batch,
                                               int64_t *bytes);
AQLM_API int aqlm_mx_gemm_quant(const aqlm_mx_matrix *W, const void *x, int64_t batch,
                                int32_t rule, void *y, int32_t type, void *workspace,
                                int64_t workspace_bytes, void *stream);

/*
 * aqlm_mx_grad_input: dx [batch][cols] = dy [batch][rows] . W, the gradient of
 * y = x . W^T with respect to x through the (constant) weights; dy and dx of
 * `type` (F16 or BF16). It is also the straight-through gradient of
 * aqlm_mx_gemm_mx with respect to the activations before their quantisation.
 * rows need not be a multiple of anything; batch == 0 is a no-op. Workspace
 * as above.
 */
AQLM_API int aqlm_mx_grad_input_workspace_size(const aqlm_mx_matrix *W, int64_t batch,
                                               int64_t *bytes);
AQLM_API int aqlm_mx_grad_input(const aqlm_mx_matrix *W, const void *dy, int64_t batch, void *dx,
                                int32_t type, void *workspace, int64_t workspace_bytes,
                                void *stream);

#ifdef __cplusplus
}
#endif

#endif /* AQLM_MX_H */
