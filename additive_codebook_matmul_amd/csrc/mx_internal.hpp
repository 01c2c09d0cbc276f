// Internal declarations of the microscaled (MXFP4) translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace aqlm {

// Dense element types (values of aqlm_mx_type).
enum class MxType : int { kF16 = 0, kBF16 = 1, kF32 = 2 };

struct MxDesc {
  int64_t rows, cols;     // cols a multiple of 32
  const uint8_t *codes;   // [rows][cols/2]
  const uint8_t *scales;  // [rows][cols/32]
};

// Modelled time (us) that reading the weights takes any kernel: about 5.2 TB/s
// and what passes around that.
inline double mx_read_us(const MxDesc &W) {
  return 3.0 + (double)(W.rows * (W.cols / 2 + W.cols / 32)) / 5.2e6;
}

// Most layers of one grouped launch.
constexpr int kMxGroup = 16;

hipError_t launch_mx_quantize(const void *x, MxType type, int64_t rows, int64_t cols, bool ceil_rule,
                              uint8_t *codes, uint8_t *scales, hipStream_t stream);
hipError_t launch_mx_dequant(const MxDesc &m, MxType type, void *W, hipStream_t stream);

// Products. The *_ws_bytes functions give the device workspace of the launch
// for the same sizes (0: none).
hipError_t launch_mx_gemv_batched(const MxDesc *W, const void *const *x, void *const *y, int n,
                                  int batch, MxType type, hipStream_t stream);
int64_t mx_gemm_ws_bytes(const MxDesc &W, int64_t batch);
hipError_t launch_mx_gemm(const MxDesc &W, const void *x, int64_t batch, void *y, MxType type,
                          void *ws, hipStream_t stream);
int64_t mx_gemm_mx_ws_bytes(const MxDesc &W, int64_t batch);
hipError_t launch_mx_gemm_mx(const MxDesc &W, const MxDesc &x, void *y, MxType type, void *ws,
                             hipStream_t stream);
int64_t mx_gemm_quant_ws_bytes(const MxDesc &W, int64_t batch);
hipError_t launch_mx_gemm_quant(const MxDesc &W, const void *x, int64_t batch, bool ceil_rule, void *y,
                                MxType type, void *ws, hipStream_t stream);
// Their tile kernels (mx_gemm_tile.hip, mx_gemm_mx_tile.hip): modelled duration
// in us, workspace, launch. Without `split` K is not split over workgroups and
// no workspace needed.
double mx_gemm_tile_us(const MxDesc &W, int64_t batch, bool split);
int64_t mx_gemm_tile_ws_bytes(const MxDesc &W, int64_t batch);
hipError_t launch_mx_gemm_tile(const MxDesc &W, const void *x, int64_t batch, void *y, MxType type,
                               bool split, void *ws, hipStream_t stream);
double mx_gemm_mx_tile_us(const MxDesc &W, int64_t batch);
int64_t mx_gemm_mx_tile_ws_bytes(const MxDesc &W, int64_t batch);
hipError_t launch_mx_gemm_mx_tile(const MxDesc &W, const MxDesc &x, void *y, MxType type, void *ws,
                                  hipStream_t stream);
int64_t mx_grad_ws_bytes(const MxDesc &W, int64_t batch);
hipError_t launch_mx_grad(const MxDesc &W, const void *dy, int64_t batch, void *dx, MxType type,
                          void *ws, hipStream_t stream);

}  // namespace aqlm
