// train_api.hip -- the C ABI declared in include/mqconv_train.h: argument
// checks (all before any HIP call) and hand-off to the launchers.
#include "mqconv_train.h"

#include <math.h>

#include "api_checks.h"
#include "train.h"

using namespace mq;

namespace {

const MxOutView kNoMx{nullptr, nullptr, 0, 0};

int check_layer_norm(const mq_layer_norm* ln, LnShape* s) {
  if (!ln) return MQ_ERR_NULL;
  if (!dims_ok(ln->h, ln->w, ln->n, ln->c)) return MQ_ERR_SHAPE;
  if (!(ln->eps >= 0.0f) || isinf(ln->eps)) return MQ_ERR_UNSUPPORTED;
  *s = LnShape{ln->h * ln->w, ln->n, ln->c, ln->eps};
  return MQ_OK;
}

int check_ws(const LnShape& s, int op, const void* ws, size_t ws_bytes) {
  if (!ws || ws_bytes < layer_norm_workspace_bytes(s, op)) return MQ_ERR_WORKSPACE;
  return aligned16(ws) ? MQ_OK : MQ_ERR_ALIGN;
}

int layer_norm(const mq_layer_norm* ln, const float* x, const float* residual, const float* gamma, const float* beta,
               float* sum, float* y, const mq_mx* yq, float* mean, float* rstd, void* ws, size_t ws_bytes,
               void* stream) {
  LnShape s;
  int e = check_layer_norm(ln, &s);
  if (e != MQ_OK) return e;
  if (!x || (!yq && !y) || (residual && !sum)) return MQ_ERR_NULL;
  if (sum && !residual) return MQ_ERR_UNSUPPORTED;
  if (yq && (e = check_mx(*yq, MQ_ROLE_ACT, ln->h, ln->w, ln->n, ln->c)) != MQ_OK) return e;
  if (!aligned4(x) || !aligned4(residual) || !aligned4(gamma) || !aligned4(beta) || !aligned4(sum) || !aligned4(y) ||
      !aligned4(mean) || !aligned4(rstd))
    return MQ_ERR_ALIGN;
  if (yq && (e = check_ws(s, 0, ws, ws_bytes)) != MQ_OK) return e;
  return hip_status(launch_layer_norm(s, x, residual, gamma, beta, sum, y, yq ? out_view(*yq) : kNoMx, mean, rstd, ws,
                                      (hipStream_t)stream));
}

int layer_norm_backward(const mq_layer_norm* ln, const float* dy, const float* x, const float* gamma,
                        const float* mean, const float* rstd, const float* dskip, float* dx, const mq_mx* dxq,
                        float* dgamma, float* dbeta, void* ws, size_t ws_bytes, void* stream) {
  LnShape s;
  int e = check_layer_norm(ln, &s);
  if (e != MQ_OK) return e;
  if (!dy || !x || !mean || !rstd || (!dxq && !dx)) return MQ_ERR_NULL;
  if (dxq && (e = check_mx(*dxq, MQ_ROLE_GRAD, ln->h, ln->w, ln->n, ln->c)) != MQ_OK) return e;
  if (!aligned4(dy) || !aligned4(x) || !aligned4(gamma) || !aligned4(mean) || !aligned4(rstd) || !aligned4(dskip) ||
      !aligned4(dx) || !aligned4(dgamma) || !aligned4(dbeta))
    return MQ_ERR_ALIGN;
  if ((e = check_ws(s, 1, ws, ws_bytes)) != MQ_OK) return e;
  return hip_status(launch_layer_norm_backward(s, dy, x, gamma, mean, rstd, dskip, dx, dxq ? out_view(*dxq) : kNoMx,
                                               dgamma, dbeta, ws, (hipStream_t)stream));
}

}  // namespace

extern "C" {

size_t mqconv_layer_norm_workspace_bytes(const mq_layer_norm* ln, int op) {
  LnShape s;
  if (check_layer_norm(ln, &s) != MQ_OK || op < 0 || op > 1) return 0;
  return layer_norm_workspace_bytes(s, op);
}

int mqconv_layer_norm(const mq_layer_norm* ln, const float* x, const float* residual, const float* gamma,
                      const float* beta, float* sum, float* y, float* mean, float* rstd, void* stream) {
  return layer_norm(ln, x, residual, gamma, beta, sum, y, nullptr, mean, rstd, nullptr, 0, stream);
}

int mqconv_layer_norm_mx(const mq_layer_norm* ln, const float* x, const float* residual, const float* gamma,
                         const float* beta, float* sum, mq_mx yq, float* mean, float* rstd, void* ws,
                         size_t ws_bytes, void* stream) {
  return layer_norm(ln, x, residual, gamma, beta, sum, nullptr, &yq, mean, rstd, ws, ws_bytes, stream);
}

int mqconv_layer_norm_backward(const mq_layer_norm* ln, const float* dy, const float* x, const float* gamma,
                               const float* mean, const float* rstd, const float* dskip, float* dx, float* dgamma,
                               float* dbeta, void* ws, size_t ws_bytes, void* stream) {
  return layer_norm_backward(ln, dy, x, gamma, mean, rstd, dskip, dx, nullptr, dgamma, dbeta, ws, ws_bytes, stream);
}

int mqconv_layer_norm_backward_mx(const mq_layer_norm* ln, const float* dy, const float* x, const float* gamma,
                                  const float* mean, const float* rstd, const float* dskip, mq_mx dxq, float* dgamma,
                                  float* dbeta, void* ws, size_t ws_bytes, void* stream) {
  return layer_norm_backward(ln, dy, x, gamma, mean, rstd, dskip, nullptr, &dxq, dgamma, dbeta, ws, ws_bytes, stream);
}

}  // extern "C"
