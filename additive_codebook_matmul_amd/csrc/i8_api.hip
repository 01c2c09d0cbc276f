// C entry points of aqlm_i8.h: argument validation on the host, then kernel
// launches on the caller's stream. Nothing here allocates or synchronises.
#include "../../include/aqlm_i8.h"
#include "i8_internal.hpp"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int from_hip(hipError_t e) { return e == hipSuccess ? AQLM_OK : AQLM_ERR_HIP; }

// Row and column limits of quantisation and expansion (flat 64-bit indexing).
bool flat_shape_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows < (int64_t(1) << 31) && cols >= 16 && cols < (int64_t(1) << 31) && cols % 16 == 0 &&
         (rows == 0 || cols < (int64_t(1) << 40) / rows);
}

int check_matrix(const aqlm_i8_matrix *m, aqlm::I8Desc *d, bool product, bool may_be_empty) {
  if (!m) return AQLM_ERR_NULL;
  if (!flat_shape_ok(m->rows, m->cols)) return AQLM_ERR_SHAPE;
  if (m->rows < 1 && !may_be_empty) return AQLM_ERR_SHAPE;
  if (product && (m->rows > AQLM_I8_MAX_DIM || m->cols > AQLM_I8_MAX_COLS)) return AQLM_ERR_SHAPE;
  *d = {m->rows, m->cols, m->codes, m->scales};
  if (m->rows == 0) return AQLM_OK;
  if (!m->codes || !m->scales) return AQLM_ERR_NULL;
  if (!aligned16(m->codes) || !aligned16(m->scales)) return AQLM_ERR_ALIGN;
  return AQLM_OK;
}

// The two layers of a gated block.
int check_pair(const aqlm_i8_matrix *gate, const aqlm_i8_matrix *up, aqlm::I8Desc *g, aqlm::I8Desc *u) {
  int st = check_matrix(gate, g, true, false);
  if (st == AQLM_OK) st = check_matrix(up, u, true, false);
  if (st != AQLM_OK) return st;
  return g->rows == u->rows && g->cols == u->cols ? AQLM_OK : AQLM_ERR_SHAPE;
}

bool half_type(int32_t type) { return type == AQLM_I8_F16 || type == AQLM_I8_BF16; }
bool act_ok(int32_t act) { return act >= AQLM_I8_SILU && act <= AQLM_I8_GELU_TANH; }
bool batch_ok(int64_t batch) { return batch >= 0 && batch <= AQLM_I8_MAX_DIM; }

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

// Sizes of a workspace query; `up` null where there is one layer.
template <class F>
int workspace_size(const aqlm_i8_matrix *W, const aqlm_i8_matrix *up, bool pair, int64_t batch, int64_t *bytes, F f) {
  if (!bytes) return AQLM_ERR_NULL;
  *bytes = 0;
  aqlm::I8Desc d, u;
  const int st = pair ? check_pair(W, up, &d, &u) : check_matrix(W, &d, true, false);
  if (st != AQLM_OK) return st;
  if (!batch_ok(batch)) return AQLM_ERR_BATCH;
  if (batch > 0) *bytes = f(d);
  return AQLM_OK;
}

constexpr aqlm::I8Desc kNone = {0, 0, nullptr, nullptr};

}  // namespace

extern "C" {

int aqlm_i8_quantize(const void *x, int32_t type, int64_t rows, int64_t cols, int8_t *codes, float *scales,
                     void *stream) {
  if (type < AQLM_I8_F16 || type > AQLM_I8_F32) return AQLM_ERR_TYPE;
  if (!flat_shape_ok(rows, cols)) return AQLM_ERR_SHAPE;
  if (rows == 0) return AQLM_OK;
  if (!x || !codes || !scales) return AQLM_ERR_NULL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return AQLM_ERR_ALIGN;
  return from_hip(aqlm::launch_i8_quantize(x, static_cast<aqlm::MxType>(type), rows, cols, codes, scales,
                                           static_cast<hipStream_t>(stream)));
}

int aqlm_i8_dequant(const aqlm_i8_matrix *m, int32_t type, void *W, void *stream) {
  aqlm::I8Desc d;
  const int st = check_matrix(m, &d, false, true);
  if (st != AQLM_OK) return st;
  if (type < AQLM_I8_F16 || type > AQLM_I8_F32) return AQLM_ERR_TYPE;
  if (d.rows == 0) return AQLM_OK;
  if (!W) return AQLM_ERR_NULL;
  if (!aligned16(W)) return AQLM_ERR_ALIGN;
  return from_hip(
      aqlm::launch_i8_dequant(d, static_cast<aqlm::MxType>(type), W, static_cast<hipStream_t>(stream)));
}

int aqlm_i8_gemm_workspace_size(const aqlm_i8_matrix *W, int64_t batch, int64_t *bytes) {
  return workspace_size(W, nullptr, false, batch, bytes,
                        [&](const aqlm::I8Desc &d) {
                          return aqlm::i8_route(d.rows, d.cols, false, batch, false).ws_bytes;
                        });
}

int aqlm_i8_gemm(const aqlm_i8_matrix *W, const aqlm_i8_matrix *x, void *y, int32_t type, void *workspace,
                 int64_t workspace_bytes, void *stream) {
  aqlm::I8Desc d, dx;
  int st = check_matrix(W, &d, true, false);
  if (st == AQLM_OK) st = check_matrix(x, &dx, true, true);
  if (st != AQLM_OK) return st;
  if (d.cols != dx.cols) return AQLM_ERR_SHAPE;
  if (!half_type(type)) return AQLM_ERR_TYPE;
  if (dx.rows == 0) return AQLM_OK;
  if (!y) return AQLM_ERR_NULL;
  if (!aligned16(y)) return AQLM_ERR_ALIGN;
  const aqlm::I8Route route = aqlm::i8_route(d.rows, d.cols, false, dx.rows, false);
  st = check_workspace(route.ws_bytes, workspace, workspace_bytes);
  if (st != AQLM_OK) return st;
  const aqlm::I8Product p = {d, kNone, aqlm::I8Act::kSilu, nullptr, dx.codes, dx.scales, dx.rows,
                             y, nullptr, nullptr, static_cast<aqlm::MxType>(type)};
  return from_hip(aqlm::launch_i8_product(p, route, workspace, static_cast<hipStream_t>(stream)));
}

int aqlm_i8_gemm_quant_workspace_size(const aqlm_i8_matrix *W, int64_t batch, int64_t *bytes) {
  return workspace_size(W, nullptr, false, batch, bytes,
                        [&](const aqlm::I8Desc &d) {
                          return aqlm::i8_route(d.rows, d.cols, false, batch, true).ws_bytes;
                        });
}

int aqlm_i8_gemm_quant(const aqlm_i8_matrix *W, const void *x, int64_t batch, void *y, int32_t type,
                       void *workspace, int64_t workspace_bytes, void *stream) {
  aqlm::I8Desc d;
  int st = check_matrix(W, &d, true, false);
  if (st != AQLM_OK) return st;
  if (!half_type(type)) return AQLM_ERR_TYPE;
  if (!batch_ok(batch)) return AQLM_ERR_BATCH;
  if (batch == 0) return AQLM_OK;
  st = check_io(x, y);
  if (st != AQLM_OK) return st;
  const aqlm::I8Route route = aqlm::i8_route(d.rows, d.cols, false, batch, true);
  st = check_workspace(route.ws_bytes, workspace, workspace_bytes);
  if (st != AQLM_OK) return st;
  const aqlm::I8Product p = {d, kNone, aqlm::I8Act::kSilu, x, nullptr, nullptr, batch,
                             y, nullptr, nullptr, static_cast<aqlm::MxType>(type)};
  return from_hip(aqlm::launch_i8_product(p, route, workspace, static_cast<hipStream_t>(stream)));
}

int aqlm_i8_gated_workspace_size(const aqlm_i8_matrix *gate, const aqlm_i8_matrix *up, int64_t batch,
                                 int64_t *bytes) {
  return workspace_size(gate, up, true, batch, bytes,
                        [&](const aqlm::I8Desc &d) {
                          return aqlm::i8_route(d.rows, d.cols, true, batch, true).ws_bytes;
                        });
}

int aqlm_i8_gated(const aqlm_i8_matrix *gate, const aqlm_i8_matrix *up, const void *x, int64_t batch, int32_t act,
                  void *h, float *g, float *u, int32_t type, void *workspace, int64_t workspace_bytes,
                  void *stream) {
  aqlm::I8Desc d, e;
  int st = check_pair(gate, up, &d, &e);
  if (st != AQLM_OK) return st;
  if (!half_type(type) || !act_ok(act)) return AQLM_ERR_TYPE;
  if (!batch_ok(batch)) return AQLM_ERR_BATCH;
  if (batch == 0) return AQLM_OK;
  st = check_io(x, h);
  if (st != AQLM_OK) return st;
  if (!g != !u) return AQLM_ERR_NULL;
  if (!aligned16(g) || !aligned16(u)) return AQLM_ERR_ALIGN;
  const aqlm::I8Route route = aqlm::i8_route(d.rows, d.cols, true, batch, true);
  st = check_workspace(route.ws_bytes, workspace, workspace_bytes);
  if (st != AQLM_OK) return st;
  const aqlm::I8Product p = {d, e, static_cast<aqlm::I8Act>(act), x, nullptr, nullptr, batch,
                             h, g, u, static_cast<aqlm::MxType>(type)};
  return from_hip(aqlm::launch_i8_product(p, route, workspace, static_cast<hipStream_t>(stream)));
}

int aqlm_i8_grad_input_workspace_size(const aqlm_i8_matrix *W, int64_t batch, int64_t *bytes) {
  return workspace_size(W, nullptr, false, batch, bytes,
                        [&](const aqlm::I8Desc &d) {
                          return aqlm::i8_grad_ws_bytes(d.rows, false, batch,
                                                        aqlm::i8_grad_plan(d.rows, d.cols, false, batch));
                        });
}

int aqlm_i8_grad_input(const aqlm_i8_matrix *W, const void *dy, int64_t batch, void *dx, int32_t type,
                       void *workspace, int64_t workspace_bytes, void *stream) {
  aqlm::I8Desc d;
  int st = check_matrix(W, &d, true, false);
  if (st != AQLM_OK) return st;
  if (!half_type(type)) return AQLM_ERR_TYPE;
  if (!batch_ok(batch)) return AQLM_ERR_BATCH;
  if (batch == 0) return AQLM_OK;
  st = check_io(dy, dx);
  if (st != AQLM_OK) return st;
  const aqlm::I8Plan plan = aqlm::i8_grad_plan(d.rows, d.cols, false, batch);
  st = check_workspace(aqlm::i8_grad_ws_bytes(d.rows, false, batch, plan), workspace, workspace_bytes);
  if (st != AQLM_OK) return st;
  const aqlm::I8Grad p = {d, kNone, aqlm::I8Act::kSilu, nullptr, nullptr, dy, batch, dx,
                          static_cast<aqlm::MxType>(type)};
  return from_hip(aqlm::launch_i8_grad(p, plan, workspace, static_cast<hipStream_t>(stream)));
}

int aqlm_i8_gated_grad_workspace_size(const aqlm_i8_matrix *gate, const aqlm_i8_matrix *up, int64_t batch,
                                      int64_t *bytes) {
  return workspace_size(gate, up, true, batch, bytes,
                        [&](const aqlm::I8Desc &d) {
                          return aqlm::i8_grad_ws_bytes(d.rows, true, batch,
                                                        aqlm::i8_grad_plan(d.rows, d.cols, true, batch));
                        });
}

int aqlm_i8_gated_grad(const aqlm_i8_matrix *gate, const aqlm_i8_matrix *up, const float *g, const float *u,
                       const void *dh, int64_t batch, int32_t act, void *dx, int32_t type, void *workspace,
                       int64_t workspace_bytes, void *stream) {
  aqlm::I8Desc d, e;
  int st = check_pair(gate, up, &d, &e);
  if (st != AQLM_OK) return st;
  if (!half_type(type) || !act_ok(act)) return AQLM_ERR_TYPE;
  if (!batch_ok(batch)) return AQLM_ERR_BATCH;
  if (batch == 0) return AQLM_OK;
  st = check_io(dh, dx);
  if (st == AQLM_OK) st = check_io(g, u);
  if (st != AQLM_OK) return st;
  const aqlm::I8Plan plan = aqlm::i8_grad_plan(d.rows, d.cols, true, batch);
  st = check_workspace(aqlm::i8_grad_ws_bytes(d.rows, true, batch, plan), workspace, workspace_bytes);
  if (st != AQLM_OK) return st;
  const aqlm::I8Grad p = {d, e, static_cast<aqlm::I8Act>(act), g, u, dh, batch, dx,
                          static_cast<aqlm::MxType>(type)};
  return from_hip(aqlm::launch_i8_grad(p, plan, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
