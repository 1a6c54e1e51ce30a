// train.h -- launchers of the layer norm kernels, of the products of two-level
// codes and of the orthogonalised weight update, shared with their C ABI layer.
// Host-side; arguments are already validated.
#pragma once
#include "mqconv_internal.h"

namespace mq {

// One layer norm: the rows of P pixels and N samples, C channels each.
struct LnShape {
  int P, N, C;
  float eps;
};
size_t layer_norm_workspace_bytes(const LnShape& s, int op);
// exactly one of y and yq (yq.codes) is given; residual, mean, rstd may be null; sum is given exactly where residual is
hipError_t launch_layer_norm(const LnShape& s, const float* x, const float* residual, const float* gamma,
                             const float* beta, float* sum, float* y, const MxOutView& yq, float* mean, float* rstd,
                             void* ws, hipStream_t st);
hipError_t launch_layer_norm_backward(const LnShape& s, const float* dy, const float* x, const float* gamma,
                                      const float* mean, const float* rstd, const float* dskip, float* dx,
                                      const MxOutView& dxq, float* dgamma, float* dbeta, void* ws, hipStream_t st);

// An operand of the two-level products.
struct NvfpView {
  const uint8_t *codes, *scales;
  const float* tensor;
  int fmt;
};
// whether the products' 16-bit operands stay within 32-bit offsets; op 0 forward, 1 backward data, 2 backward weight
bool nvfp_gemm_ok(const Conv& c, int op);
size_t nvfp_gemm_workspace_bytes(const Conv& c, int op, int fa);  // fa: format of the call's first operand
hipError_t launch_nvfp_forward(const Conv& c, const NvfpView& x, const NvfpView& w, float* y, void* ws, hipStream_t st);
hipError_t launch_nvfp_backward_data(const Conv& c, const NvfpView& dy, const NvfpView& w, float* dx, void* ws, hipStream_t st);
hipError_t launch_nvfp_backward_weight(const Conv& c, const NvfpView& dy, const NvfpView& x, float* dw, void* ws, hipStream_t st);

// The weight update: Newton-Schulz steps, and the optimizer around them.
constexpr int kUpdateGroup = 32;  // MQ_UPDATE_GROUP_MAX
struct UpdateSpec {
  int steps;
  float a, b, c, eps;
  float momentum, decay, lr;
  bool nesterov;
  int scale;          // MQ_SCALE_*
  const float* rate;  // device, or null
};
// whether the planes of a matrix stay within 32-bit offsets
bool newton_shape_ok(int rows, int cols);
size_t newton_workspace_bytes(int count, const int* rows, const int* cols);
// mom null: out = the orthogonalised gradient; else mom and out (the weight) are updated
hipError_t launch_newton(const UpdateSpec& u, int count, const int* rows, const int* cols, const float* const* grad,
                         float* const* mom, float* const* out, void* ws, hipStream_t st);

}  // namespace mq
