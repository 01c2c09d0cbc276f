// C entry points of aqlm_mx.h: argument validation on the host, then kernel
// launches on the caller's stream. Nothing here allocates or synchronises.
#include "../../include/aqlm_mx.h"
#include "mx_internal.hpp"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int from_hip(hipError_t e) { return e == hipSuccess ? AQLM_OK : AQLM_ERR_HIP; }

// Row and column limits of quantisation and expansion (flat 64-bit indexing).
bool flat_shape_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows < (int64_t(1) << 31) && cols >= AQLM_MX_BLOCK &&
         cols < (int64_t(1) << 31) && cols % AQLM_MX_BLOCK == 0 &&
         (rows == 0 || cols < (int64_t(1) << 40) / rows);
}

int check_matrix(const aqlm_mx_matrix *m, aqlm::MxDesc *d, bool product, bool may_be_empty) {
  if (!m) return AQLM_ERR_NULL;
  if (!flat_shape_ok(m->rows, m->cols)) return AQLM_ERR_SHAPE;
  if (m->rows < 1 && !may_be_empty) return AQLM_ERR_SHAPE;
  if (product && (m->rows > AQLM_MX_MAX_DIM || m->cols > AQLM_MX_MAX_DIM)) return AQLM_ERR_SHAPE;
  *d = {m->rows, m->cols, m->codes, m->scales};
  if (m->rows == 0) return AQLM_OK;
  if (!m->codes || !m->scales) return AQLM_ERR_NULL;
  if (!aligned16(m->codes) || !aligned16(m->scales)) return AQLM_ERR_ALIGN;
  return AQLM_OK;
}

bool half_type(int32_t type) { return type == AQLM_MX_F16 || type == AQLM_MX_BF16; }

int check_io(const void *in, const void *out) {
  if (!in || !out) return AQLM_ERR_NULL;
  if (!aligned16(in) || !aligned16(out)) return AQLM_ERR_ALIGN;
  return AQLM_OK;
}

int check_workspace(int64_t need, const void *workspace, int64_t bytes) {
  if (need == 0) return AQLM_OK;
  if (!workspace) return AQLM_ERR_NULL;
  if (!aligned16(workspace)) return AQLM_ERR_ALIGN;
  return bytes < need ? AQLM_ERR_WORKSPACE : AQLM_OK;
}

typedef int64_t (*WsBytes)(const aqlm::MxDesc &, int64_t);

int workspace_size(WsBytes f, const aqlm_mx_matrix *W, int64_t batch, int64_t *bytes) {
  if (!bytes) return AQLM_ERR_NULL;
  *bytes = 0;
  aqlm::MxDesc d;
  const int st = check_matrix(W, &d, true, false);
  if (st != AQLM_OK) return st;
  if (batch < 0 || batch > AQLM_MX_MAX_DIM) return AQLM_ERR_BATCH;
  if (batch > 0) *bytes = f(d, batch);
  return AQLM_OK;
}

}  // namespace

extern "C" {

int aqlm_mx_quantize(const void *x, int32_t type, int64_t rows, int64_t cols, int32_t rule,
                     uint8_t *codes, uint8_t *scales, void *stream) {
  if (type < AQLM_MX_F16 || type > AQLM_MX_F32) return AQLM_ERR_TYPE;
  if (rule != AQLM_MX_SCALE_FLOOR && rule != AQLM_MX_SCALE_CEIL) return AQLM_ERR_TYPE;
  if (!flat_shape_ok(rows, cols)) return AQLM_ERR_SHAPE;
  if (rows == 0) return AQLM_OK;
  if (!x || !codes || !scales) return AQLM_ERR_NULL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return AQLM_ERR_ALIGN;
  return from_hip(aqlm::launch_mx_quantize(x, static_cast<aqlm::MxType>(type), rows, cols,
                                           rule == AQLM_MX_SCALE_CEIL, codes, scales,
                                           static_cast<hipStream_t>(stream)));
}

int aqlm_mx_dequant(const aqlm_mx_matrix *m, int32_t type, void *W, void *stream) {
  aqlm::MxDesc d;
  const int st = check_matrix(m, &d, false, true);
  if (st != AQLM_OK) return st;
  if (type < AQLM_MX_F16 || type > AQLM_MX_F32) return AQLM_ERR_TYPE;
  if (d.rows == 0) return AQLM_OK;
  if (!W) return AQLM_ERR_NULL;
  if (!aligned16(W)) return AQLM_ERR_ALIGN;
  return from_hip(aqlm::launch_mx_dequant(d, static_cast<aqlm::MxType>(type), W,
                                          static_cast<hipStream_t>(stream)));
}

int aqlm_mx_gemv_batched(const aqlm_mx_matrix *W, const void *const *x, void *const *y,
                         int32_t num_layers, int64_t batch, int32_t type, void *stream) {
  if (num_layers < 0 || num_layers > 4096) return AQLM_ERR_SHAPE;
  if (batch < 0 || batch > 8) return AQLM_ERR_BATCH;
  if (!half_type(type)) return AQLM_ERR_TYPE;
  if (num_layers == 0 || batch == 0) return AQLM_OK;
  if (!W || !x || !y) return AQLM_ERR_NULL;
  aqlm::MxDesc d[aqlm::kMxGroup];
  for (int i = 0; i < num_layers; ++i) {  // every layer before anything is launched
    int st = check_matrix(&W[i], &d[0], true, false);
    if (st == AQLM_OK) st = check_io(x[i], y[i]);
    if (st != AQLM_OK) return st;
  }
  for (int i = 0; i < num_layers; i += aqlm::kMxGroup) {
    const int n = num_layers - i < aqlm::kMxGroup ? num_layers - i : aqlm::kMxGroup;
    for (int k = 0; k < n; ++k) check_matrix(&W[i + k], &d[k], true, false);
    const int st = from_hip(aqlm::launch_mx_gemv_batched(d, x + i, y + i, n, (int)batch,
                                                         static_cast<aqlm::MxType>(type),
                                                         static_cast<hipStream_t>(stream)));
    if (st != AQLM_OK) return st;
  }
  return AQLM_OK;
}

int aqlm_mx_gemm_workspace_size(const aqlm_mx_matrix *W, int64_t batch, int64_t *bytes) {
  return workspace_size(aqlm::mx_gemm_ws_bytes, W, batch, bytes);
}

int aqlm_mx_gemm(const aqlm_mx_matrix *W, const void *x, int64_t batch, void *y, int32_t type,
                 void *workspace, int64_t workspace_bytes, void *stream) {
  aqlm::MxDesc d;
  int st = check_matrix(W, &d, true, false);
  if (st != AQLM_OK) return st;
  if (!half_type(type)) return AQLM_ERR_TYPE;
  if (batch < 0 || batch > AQLM_MX_MAX_DIM) return AQLM_ERR_BATCH;
  if (batch == 0) return AQLM_OK;
  st = check_io(x, y);
  if (st == AQLM_OK) st = check_workspace(aqlm::mx_gemm_ws_bytes(d, batch), workspace, workspace_bytes);
  if (st != AQLM_OK) return st;
  return from_hip(aqlm::launch_mx_gemm(d, x, batch, y, static_cast<aqlm::MxType>(type), workspace,
                                       static_cast<hipStream_t>(stream)));
}

int aqlm_mx_gemm_mx_workspace_size(const aqlm_mx_matrix *W, int64_t batch, int64_t *bytes) {
  return workspace_size(aqlm::mx_gemm_mx_ws_bytes, W, batch, bytes);
}

int aqlm_mx_gemm_mx(const aqlm_mx_matrix *W, const aqlm_mx_matrix *x, void *y, int32_t type,
                    void *workspace, int64_t workspace_bytes, void *stream) {
  aqlm::MxDesc d, dx;
  int st = check_matrix(W, &d, true, false);
  if (st == AQLM_OK) st = check_matrix(x, &dx, true, true);
  if (st != AQLM_OK) return st;
  if (d.cols != dx.cols) return AQLM_ERR_SHAPE;
  if (!half_type(type)) return AQLM_ERR_TYPE;
  if (dx.rows == 0) return AQLM_OK;
  if (!y) return AQLM_ERR_NULL;
  if (!aligned16(y)) return AQLM_ERR_ALIGN;
  st = check_workspace(aqlm::mx_gemm_mx_ws_bytes(d, dx.rows), workspace, workspace_bytes);
  if (st != AQLM_OK) return st;
  return from_hip(aqlm::launch_mx_gemm_mx(d, dx, y, static_cast<aqlm::MxType>(type), workspace,
                                          static_cast<hipStream_t>(stream)));
}

int aqlm_mx_gemm_quant_workspace_size(const aqlm_mx_matrix *W, int64_t batch, int64_t *bytes) {
  return workspace_size(aqlm::mx_gemm_quant_ws_bytes, W, batch, bytes);
}

int aqlm_mx_gemm_quant(const aqlm_mx_matrix *W, const void *x, int64_t batch, int32_t rule, void *y,
                       int32_t type, void *workspace, int64_t workspace_bytes, void *stream) {
  aqlm::MxDesc d;
  int st = check_matrix(W, &d, true, false);
  if (st != AQLM_OK) return st;
  if (!half_type(type)) return AQLM_ERR_TYPE;
  if (rule != AQLM_MX_SCALE_FLOOR && rule != AQLM_MX_SCALE_CEIL) return AQLM_ERR_TYPE;
  if (batch < 0 || batch > AQLM_MX_MAX_DIM) return AQLM_ERR_BATCH;
  if (batch == 0) return AQLM_OK;
  st = check_io(x, y);
  if (st == AQLM_OK)
    st = check_workspace(aqlm::mx_gemm_quant_ws_bytes(d, batch), workspace, workspace_bytes);
  if (st != AQLM_OK) return st;
  return from_hip(aqlm::launch_mx_gemm_quant(d, x, batch, rule == AQLM_MX_SCALE_CEIL, y,
                                             static_cast<aqlm::MxType>(type), workspace,
                                             static_cast<hipStream_t>(stream)));
}

int aqlm_mx_grad_input_workspace_size(const aqlm_mx_matrix *W, int64_t batch, int64_t *bytes) {
  return workspace_size(aqlm::mx_grad_ws_bytes, W, batch, bytes);
}

int aqlm_mx_grad_input(const aqlm_mx_matrix *W, const void *dy, int64_t batch, void *dx,
                       int32_t type, void *workspace, int64_t workspace_bytes, void *stream) {
  aqlm::MxDesc d;
  int st = check_matrix(W, &d, true, false);
  if (st != AQLM_OK) return st;
  if (!half_type(type)) return AQLM_ERR_TYPE;
  if (batch < 0 || batch > AQLM_MX_MAX_DIM) return AQLM_ERR_BATCH;
  if (batch == 0) return AQLM_OK;
  st = check_io(dy, dx);
  if (st == AQLM_OK) st = check_workspace(aqlm::mx_grad_ws_bytes(d, batch), workspace, workspace_bytes);
  if (st != AQLM_OK) return st;
  return from_hip(aqlm::launch_mx_grad(d, dy, batch, dx, static_cast<aqlm::MxType>(type), workspace,
                                       static_cast<hipStream_t>(stream)));
}

}  // extern "C"
