// block.h -- launchers of the group norm, dropout and replay cache kernels,
// shared with their C ABI layer. Host-side; arguments are already validated.
#pragma once
#include "mqconv_internal.h"

namespace mq {

struct DropArgs;  // block_common.h

// Dropout as the ABI gives it (p = 0: none).
struct DropSpec {
  float p;
  uint64_t seed;
  const uint64_t* step;
};

// One group norm: P pixels, N samples, C channels in G groups.
struct NormShape {
  int P, N, C, G, act;
  float eps;
};

size_t norm_workspace_bytes(const NormShape& s, int op);
// exactly one of y and yq (yq.codes) is given; mean, rstd may be null
hipError_t launch_group_norm(const NormShape& s, const float* x, const float* gamma, const float* beta,
                             const DropSpec& drop, float* y, const MxOutView& yq, float* mean, float* rstd, void* ws,
                             hipStream_t st);
hipError_t launch_group_norm_backward(const NormShape& s, const float* dy, const float* x, const float* gamma,
                                      const float* beta, const float* mean, const float* rstd, const DropSpec& drop,
                                      float* dx, const MxOutView& dxq, float* dgamma, float* dbeta, void* ws,
                                      hipStream_t st);

hipError_t launch_dropout(const float* x, const float* residual, int rows, int C, const DropSpec& drop, float* y,
                          hipStream_t st);
hipError_t launch_dropout_mx(const float* x, int P, int N, int C, const DropSpec& drop, const MxOutView& out,
                             hipStream_t st);

// A replay cache: slot-major lines, P pixels a slot.
struct CacheView {
  uint8_t *codes, *scales;
  int fmt, slots, P, C;
};
hipError_t launch_cache_write(const CacheView& c, const float* x, int N, int n0, int count, const int32_t* slot,
                              hipStream_t st);
hipError_t launch_cache_read(const CacheView& c, const int32_t* slot, int count, float* x, int N, int n0,
                             hipStream_t st);
hipError_t launch_cache_read_mx(const CacheView& c, const int32_t* slot, int N, const MxOutView& out, hipStream_t st);

}  // namespace mq
