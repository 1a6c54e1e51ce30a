// train_api.hip -- the C ABI declared in include/mqconv_train.h: argument
// checks (all before any HIP call) and hand-off to the launchers.
#include "mqconv_train.h"

#include <math.h>

#include "api_checks.h"
#include "train.h"

using namespace mq;

namespace {

static_assert(kUpdateGroup == MQ_UPDATE_GROUP_MAX, "matrices of a call");

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

int check_nvfp(const mq_nvfp& t, mq_role role, int32_t d0, int32_t d1, int32_t d2, int32_t d3, NvfpView* v) {
  if (!t.codes || !t.block_scales || !t.tensor_scale) return MQ_ERR_NULL;
  if (!fmt_ok(t.fmt) || t.role != role) return MQ_ERR_FORMAT;
  if (t.d0 != d0 || t.d1 != d1 || t.d2 != d2 || t.d3 != d3) return MQ_ERR_SHAPE;
  if (!aligned16(t.codes) || !aligned4(t.tensor_scale)) return MQ_ERR_ALIGN;
  *v = NvfpView{static_cast<const uint8_t*>(t.codes), t.block_scales, t.tensor_scale, t.fmt};
  return MQ_OK;
}

int check_product(const mq_conv* cv, int op, int fa, const float* out, const void* ws, size_t ws_bytes) {
  if (!nvfp_gemm_ok(to_conv(cv), op)) return MQ_ERR_SHAPE;
  if (!out) return MQ_ERR_NULL;
  if (!aligned4(out)) return MQ_ERR_ALIGN;
  if (!ws || ws_bytes < nvfp_gemm_workspace_bytes(to_conv(cv), op, fa)) return MQ_ERR_WORKSPACE;
  return aligned16(ws) ? MQ_OK : MQ_ERR_ALIGN;
}

// Whether the steps stay where the stored values are in range (newton.hip):
// |x| and |x|^2 below 2, the factor of a step below 4, with room for rounding.
bool newton_in_range(const mq_newton& p) {
  const double a = p.a, b = p.b, c = p.c;
  double top = 1.0;  // of the singular values before the step
  for (int s = 0; s < p.steps; s++) {
    const double y1 = top * top * 1.002;
    if (!(y1 < 1.99)) return false;
    // extremes over y = x^2 in [0, y1]: the ends and the stationary points
    double most_f = fmax(fabs(a), fabs(a + y1 * (b + c * y1))), most_p = 0;
    if (c != 0) {
      const double y = -b / (2 * c);
      if (y > 0 && y < y1) most_f = fmax(most_f, fabs(a + y * (b + c * y)));
    }
    if (!(most_f < 3.99)) return false;
    auto take = [&](double y) {
      if (y >= 0 && y <= y1) most_p = fmax(most_p, fabs(sqrt(y) * (a + y * (b + c * y))));
    };
    take(y1);
    if (c != 0) {
      const double d = 9 * b * b - 20 * a * c;
      if (d >= 0) {
        take((-3 * b + sqrt(d)) / (10 * c));
        take((-3 * b - sqrt(d)) / (10 * c));
      }
    } else if (b != 0) {
      take(-a / (3 * b));
    }
    top = most_p;
  }
  return true;
}

bool finite(float v) { return v - v == 0.0f; }

int check_newton(const mq_newton& p) {
  if (p.steps < 1 || p.steps > MQ_NEWTON_STEPS_MAX) return MQ_ERR_UNSUPPORTED;
  if (!finite(p.a) || !finite(p.b) || !finite(p.c) || !finite(p.eps) || !(p.eps >= 0.0f)) return MQ_ERR_UNSUPPORTED;
  return newton_in_range(p) ? MQ_OK : MQ_ERR_UNSUPPORTED;
}

bool matrices_ok(int32_t count, const int32_t* rows, const int32_t* cols) {
  if (count < 1 || count > MQ_UPDATE_GROUP_MAX) return false;
  for (int i = 0; i < count; i++)
    if (rows[i] < 1 || cols[i] < 1 || rows[i] >= 1 << 30 || cols[i] >= 1 << 30 || !newton_shape_ok(rows[i], cols[i]))
      return false;
  return true;
}

int check_matrices(int32_t count, const int32_t* rows, const int32_t* cols, const float* const* in, float* const* mom,
                   bool update, float* const* out, const void* ws, size_t ws_bytes) {
  if (!rows || !cols || !in || !out || (update && !mom)) return MQ_ERR_NULL;
  if (!matrices_ok(count, rows, cols)) return MQ_ERR_SHAPE;
  for (int i = 0; i < count; i++) {
    if (!in[i] || !out[i] || (update && !mom[i])) return MQ_ERR_NULL;
    if (!aligned4(in[i]) || !aligned4(out[i]) || (update && !aligned4(mom[i]))) return MQ_ERR_ALIGN;
  }
  if (!ws || ws_bytes < newton_workspace_bytes(count, rows, cols)) return MQ_ERR_WORKSPACE;
  return aligned16(ws) ? MQ_OK : MQ_ERR_ALIGN;
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

size_t mqconv_nvfp_gemm_workspace_bytes(const mq_conv* cv, int op, mq_elem fa, mq_elem fb) {
  if (!conv_ok(cv) || op < 0 || op > 2 || !fmt_ok(fa) || !fmt_ok(fb) || !nvfp_gemm_ok(to_conv(cv), op)) return 0;
  return nvfp_gemm_workspace_bytes(to_conv(cv), op, fa);
}

int mqconv_nvfp_forward(const mq_conv* cv, mq_nvfp xq, mq_nvfp wq, float* y, void* ws, size_t ws_bytes, void* stream) {
  if (!cv) return MQ_ERR_NULL;
  if (!conv_ok(cv)) return MQ_ERR_SHAPE;
  NvfpView x, w;
  int e = check_nvfp(xq, MQ_ROLE_ACT, cv->h, cv->w, cv->n, cv->cin, &x);
  if (e != MQ_OK) return e;
  if ((e = check_nvfp(wq, MQ_ROLE_WEIGHT, cv->cout, cv->kh, cv->kw, cv->cin, &w)) != MQ_OK) return e;
  if ((e = check_product(cv, 0, x.fmt, y, ws, ws_bytes)) != MQ_OK) return e;
  return hip_status(launch_nvfp_forward(to_conv(cv), x, w, y, ws, (hipStream_t)stream));
}

int mqconv_nvfp_backward_data(const mq_conv* cv, mq_nvfp dyq, mq_nvfp wq, float* dx, void* ws, size_t ws_bytes,
                              void* stream) {
  if (!cv) return MQ_ERR_NULL;
  if (!conv_ok(cv)) return MQ_ERR_SHAPE;
  const Conv c = to_conv(cv);
  NvfpView dy, w;
  int e = check_nvfp(dyq, MQ_ROLE_GRAD, c.ho(), c.wo(), c.n, c.cout, &dy);
  if (e != MQ_OK) return e;
  if ((e = check_nvfp(wq, MQ_ROLE_WEIGHT, c.cout, c.kh, c.kw, c.cin, &w)) != MQ_OK) return e;
  if ((e = check_product(cv, 1, dy.fmt, dx, ws, ws_bytes)) != MQ_OK) return e;
  return hip_status(launch_nvfp_backward_data(c, dy, w, dx, ws, (hipStream_t)stream));
}

int mqconv_nvfp_backward_weight(const mq_conv* cv, mq_nvfp dyq, mq_nvfp xq, float* dw, void* ws, size_t ws_bytes,
                                void* stream) {
  if (!cv) return MQ_ERR_NULL;
  if (!conv_ok(cv)) return MQ_ERR_SHAPE;
  const Conv c = to_conv(cv);
  NvfpView dy, x;
  int e = check_nvfp(dyq, MQ_ROLE_GRAD, c.ho(), c.wo(), c.n, c.cout, &dy);
  if (e != MQ_OK) return e;
  if ((e = check_nvfp(xq, MQ_ROLE_ACT, c.h, c.w, c.n, c.cin, &x)) != MQ_OK) return e;
  if ((e = check_product(cv, 2, dy.fmt, dw, ws, ws_bytes)) != MQ_OK) return e;
  return hip_status(launch_nvfp_backward_weight(c, dy, x, dw, ws, (hipStream_t)stream));
}

size_t mqconv_orthogonalize_workspace_bytes(int32_t count, const int32_t* rows, const int32_t* cols) {
  if (!rows || !cols || !matrices_ok(count, rows, cols)) return 0;
  return newton_workspace_bytes(count, rows, cols);
}

int mqconv_orthogonalize(const mq_newton* newton, int32_t count, const int32_t* rows, const int32_t* cols,
                         const float* const* u, float* const* x, void* ws, size_t ws_bytes, void* stream) {
  if (!newton) return MQ_ERR_NULL;
  int e = check_newton(*newton);
  if (e != MQ_OK) return e;
  if ((e = check_matrices(count, rows, cols, u, nullptr, false, x, ws, ws_bytes)) != MQ_OK) return e;
  UpdateSpec s{};
  s.steps = newton->steps; s.a = newton->a; s.b = newton->b; s.c = newton->c; s.eps = newton->eps;
  return hip_status(launch_newton(s, count, rows, cols, u, nullptr, x, ws, (hipStream_t)stream));
}

int mqconv_muon_update(const mq_muon* opt, int32_t count, const int32_t* rows, const int32_t* cols,
                       const float* const* g, float* const* m, float* const* w, void* ws, size_t ws_bytes,
                       void* stream) {
  if (!opt) return MQ_ERR_NULL;
  int e = check_newton(opt->newton);
  if (e != MQ_OK) return e;
  if (!finite(opt->lr) || !finite(opt->momentum) || !finite(opt->decay) || (opt->nesterov & ~1)) return MQ_ERR_UNSUPPORTED;
  if (opt->scale < MQ_SCALE_NONE || opt->scale > MQ_SCALE_RMS) return MQ_ERR_FORMAT;
  if (!aligned4(opt->rate)) return MQ_ERR_ALIGN;
  if ((e = check_matrices(count, rows, cols, g, m, true, w, ws, ws_bytes)) != MQ_OK) return e;
  const mq_newton& n = opt->newton;
  const UpdateSpec s{n.steps, n.a, n.b, n.c, n.eps, opt->momentum, opt->decay, opt->lr, opt->nesterov != 0, opt->scale,
                     opt->rate};
  return hip_status(launch_newton(s, count, rows, cols, g, m, w, ws, (hipStream_t)stream));
}

}  // extern "C"
