// layer_norm.h -- arguments that the layer norm's kernels share.
#pragma once
#include "block_common.h"
#include "train.h"

namespace mq {

// Row sums of the gradient over C: k1 = sum(gamma dy) / C, k2 = sum(gamma dy xh) / C.
struct LnRow {
  float k1, k2;
};

struct LnArgs {
  const float *x, *add;            // add: residual (forward) or the skip path's gradient (backward); may be null
  const float *dy, *gamma, *beta;  // gamma, beta may be null
  const float *mean_in, *rstd_in;  // backward
  float *sum, *mean, *rstd;        // forward: x + add (given exactly where add is), and the statistics (may be null)
  float* out;                      // y or dx; null: the rows' parameters instead (rows: mean, rstd or `row`)
  LnRow* row;                      // backward without dx
  float2* part;                    // backward: sums of dy and dy xh of each workgroup's rows [parts][C]
  float *dgamma, *dbeta;
  int R, C, parts;
  float eps;
  double inv;                      // 1 / C
};

hipError_t launch_layer_norm_rows(const LnArgs& a, hipStream_t st);
// dx or the rows' parameters, and `part` where it is given
hipError_t launch_layer_norm_grad_rows(const LnArgs& a, hipStream_t st);
hipError_t launch_layer_norm_columns(const LnArgs& a, hipStream_t st);
// the MX forms in one pass, for rows of C channels that one wave holds; the gradient's sets `parts` to the rows it leaves, at
// most as many as it is given
bool layer_norm_mx_one_pass(int C);
hipError_t launch_layer_norm_mx(const LnArgs& a, int N, const MxOutView& out, hipStream_t st);
hipError_t launch_layer_norm_grad_mx(LnArgs& a, int N, const MxOutView& out, hipStream_t st);
// their second pass for other rows: every value again from its row's parameters
hipError_t launch_layer_norm_mx_rows(const LnArgs& a, int N, const MxOutView& out, hipStream_t st);
hipError_t launch_layer_norm_grad_mx_rows(const LnArgs& a, int N, const MxOutView& out, hipStream_t st);

// Values that two kernels must agree on to the bit: contraction is off, and
// the fused operations are explicit.
__device__ __forceinline__ float ln_value(float x, float mean, float rstd, float gamma, float beta) {
#pragma clang fp contract(off)
  return __builtin_fmaf((x - mean) * rstd, gamma, beta);
}
__device__ __forceinline__ float ln_hat(float x, float mean, float rstd) {
#pragma clang fp contract(off)
  return (x - mean) * rstd;
}
__device__ __forceinline__ float ln_grad(float g, float xh, float k1, float k2, float rstd) {
#pragma clang fp contract(off)
  return rstd * __builtin_fmaf(-xh, k2, g - k1);
}
__device__ __forceinline__ float ln_grad(float g, float xh, float k1, float k2, float rstd, float skip) {
#pragma clang fp contract(off)
  return __builtin_fmaf(rstd, __builtin_fmaf(-xh, k2, g - k1), skip);
}

}  // namespace mq
