// block_api.hip -- the C ABI declared in include/mqconv_block.h: argument
// checks (all before any HIP call) and hand-off to the launchers.
#include "mqconv_block.h"

#include <math.h>

#include "api_checks.h"
#include "block.h"

using namespace mq;

namespace {

int check_drop(const mq_drop* d, DropSpec* out) {
  *out = DropSpec{0.0f, 0, nullptr};
  if (!d) return MQ_OK;
  if (!(d->p >= 0.0f && d->p <= 1.0f)) return MQ_ERR_UNSUPPORTED;
  if ((uintptr_t)d->step & 7u) return MQ_ERR_ALIGN;
  *out = DropSpec{d->p, d->seed, d->step};
  return MQ_OK;
}

int check_norm(const mq_norm* gn, NormShape* s) {
  if (!gn) return MQ_ERR_NULL;
  if (!dims_ok(gn->h, gn->w, gn->n, gn->c)) return MQ_ERR_SHAPE;
  if (gn->groups < 1 || gn->c % gn->groups != 0) return MQ_ERR_SHAPE;
  if (gn->act < MQ_ACT_NONE || gn->act > MQ_ACT_GELU) return MQ_ERR_FORMAT;
  if (!(gn->eps >= 0.0f) || isinf(gn->eps)) return MQ_ERR_UNSUPPORTED;
  *s = NormShape{gn->h * gn->w, gn->n, gn->c, gn->groups, gn->act, gn->eps};
  return MQ_OK;
}

int check_ws(const NormShape& s, int op, const void* ws, size_t ws_bytes) {
  if (!ws || ws_bytes < norm_workspace_bytes(s, op)) return MQ_ERR_WORKSPACE;
  return aligned16(ws) ? MQ_OK : MQ_ERR_ALIGN;
}

const MxOutView kNoMx{nullptr, nullptr, 0, 0};

int group_norm(const mq_norm* gn, const float* x, const float* gamma, const float* beta, const mq_drop* drop,
               float* y, const mq_mx* yq, float* mean, float* rstd, void* ws, size_t ws_bytes, void* stream) {
  NormShape s;
  DropSpec d;
  int e = check_norm(gn, &s);
  if (e != MQ_OK) return e;
  if ((e = check_drop(drop, &d)) != MQ_OK) return e;
  if (!x || (!yq && !y)) return MQ_ERR_NULL;
  if (yq && (e = check_mx(*yq, MQ_ROLE_ACT, gn->h, gn->w, gn->n, gn->c)) != MQ_OK) return e;
  if (!aligned4(x) || !aligned4(gamma) || !aligned4(beta) || !aligned4(y) || !aligned4(mean) || !aligned4(rstd))
    return MQ_ERR_ALIGN;
  if ((e = check_ws(s, 0, ws, ws_bytes)) != MQ_OK) return e;
  return hip_status(launch_group_norm(s, x, gamma, beta, d, y, yq ? out_view(*yq) : kNoMx, mean, rstd, ws,
                                      (hipStream_t)stream));
}

int group_norm_backward(const mq_norm* gn, const float* dy, const float* x, const float* gamma, const float* beta,
                        const float* mean, const float* rstd, const mq_drop* drop, float* dx, const mq_mx* dxq,
                        float* dgamma, float* dbeta, void* ws, size_t ws_bytes, void* stream) {
  NormShape s;
  DropSpec d;
  int e = check_norm(gn, &s);
  if (e != MQ_OK) return e;
  if ((e = check_drop(drop, &d)) != MQ_OK) return e;
  if (!dy || !x || !mean || !rstd || (!dxq && !dx)) return MQ_ERR_NULL;
  if (dxq && (e = check_mx(*dxq, MQ_ROLE_GRAD, gn->h, gn->w, gn->n, gn->c)) != MQ_OK) return e;
  if (!aligned4(dy) || !aligned4(x) || !aligned4(gamma) || !aligned4(beta) || !aligned4(mean) || !aligned4(rstd) ||
      !aligned4(dx) || !aligned4(dgamma) || !aligned4(dbeta))
    return MQ_ERR_ALIGN;
  if ((e = check_ws(s, 1, ws, ws_bytes)) != MQ_OK) return e;
  return hip_status(launch_group_norm_backward(s, dy, x, gamma, beta, mean, rstd, d, dx,
                                               dxq ? out_view(*dxq) : kNoMx, dgamma, dbeta, ws,
                                               (hipStream_t)stream));
}

bool cache_dims_ok(int32_t slots, int32_t h, int32_t w, int32_t c) { return slots >= 1 && dims_ok(h, w, 1, c); }

int check_cache(const mq_cache& c, const int32_t* slot, CacheView* v) {
  if (!c.codes || !c.scales || !slot) return MQ_ERR_NULL;
  if (!fmt_ok(c.fmt)) return MQ_ERR_FORMAT;
  if (!cache_dims_ok(c.slots, c.h, c.w, c.c)) return MQ_ERR_SHAPE;
  if (!aligned16(c.codes) || !aligned16(c.scales) || !aligned4(slot)) return MQ_ERR_ALIGN;
  *v = CacheView{static_cast<uint8_t*>(c.codes), c.scales, c.fmt, c.slots, c.h * c.w, c.c};
  return MQ_OK;
}

// samples n0 .. n0 + count - 1 of a batch of n
bool range_ok(const mq_cache& c, int32_t n, int32_t n0, int32_t count) {
  return dims_ok(c.h, c.w, n, c.c) && n0 >= 0 && count >= 1 && count <= n && n0 <= n - count;
}

}  // namespace

extern "C" {

int mqconv_dropout(const float* x, const float* residual, int32_t h, int32_t w, int32_t n, int32_t c,
                   const mq_drop* drop, float* y, void* stream) {
  DropSpec d;
  if (!x || !drop || !y) return MQ_ERR_NULL;
  if (!dims_ok(h, w, n, c)) return MQ_ERR_SHAPE;
  const int e = check_drop(drop, &d);
  if (e != MQ_OK) return e;
  if (!aligned4(x) || !aligned4(residual) || !aligned4(y)) return MQ_ERR_ALIGN;
  return hip_status(launch_dropout(x, residual, h * w * n, c, d, y, (hipStream_t)stream));
}

int mqconv_dropout_mx(const float* x, const mq_drop* drop, mq_mx dst, void* stream) {
  DropSpec d;
  if (!x || !drop) return MQ_ERR_NULL;
  if (dst.role != MQ_ROLE_ACT && dst.role != MQ_ROLE_GRAD) return MQ_ERR_FORMAT;
  int e = check_mx(dst, dst.role, dst.d0, dst.d1, dst.d2, dst.d3);
  if (e != MQ_OK) return e;
  if (!dims_ok(dst.d0, dst.d1, dst.d2, dst.d3)) return MQ_ERR_SHAPE;
  if ((e = check_drop(drop, &d)) != MQ_OK) return e;
  if (!aligned4(x)) return MQ_ERR_ALIGN;
  return hip_status(
      launch_dropout_mx(x, dst.d0 * dst.d1, dst.d2, dst.d3, d, out_view(dst), (hipStream_t)stream));
}

size_t mqconv_group_norm_workspace_bytes(const mq_norm* gn, int op) {
  NormShape s;
  if (check_norm(gn, &s) != MQ_OK || op < 0 || op > 1) return 0;
  return norm_workspace_bytes(s, op);
}

int mqconv_group_norm(const mq_norm* gn, const float* x, const float* gamma, const float* beta, const mq_drop* drop,
                      float* y, float* mean, float* rstd, void* ws, size_t ws_bytes, void* stream) {
  return group_norm(gn, x, gamma, beta, drop, y, nullptr, mean, rstd, ws, ws_bytes, stream);
}

int mqconv_group_norm_mx(const mq_norm* gn, const float* x, const float* gamma, const float* beta,
                         const mq_drop* drop, mq_mx yq, float* mean, float* rstd, void* ws, size_t ws_bytes,
                         void* stream) {
  return group_norm(gn, x, gamma, beta, drop, nullptr, &yq, mean, rstd, ws, ws_bytes, stream);
}

int mqconv_group_norm_backward(const mq_norm* gn, const float* dy, const float* x, const float* gamma,
                               const float* beta, const float* mean, const float* rstd, const mq_drop* drop,
                               float* dx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes, void* stream) {
  return group_norm_backward(gn, dy, x, gamma, beta, mean, rstd, drop, dx, nullptr, dgamma, dbeta, ws, ws_bytes,
                             stream);
}

int mqconv_group_norm_backward_mx(const mq_norm* gn, const float* dy, const float* x, const float* gamma,
                                  const float* beta, const float* mean, const float* rstd, const mq_drop* drop,
                                  mq_mx dxq, float* dgamma, float* dbeta, void* ws, size_t ws_bytes, void* stream) {
  return group_norm_backward(gn, dy, x, gamma, beta, mean, rstd, drop, nullptr, &dxq, dgamma, dbeta, ws, ws_bytes,
                             stream);
}

size_t mqconv_cache_codes_bytes(mq_elem fmt, int32_t slots, int32_t h, int32_t w, int32_t c) {
  if (!fmt_ok(fmt) || !cache_dims_ok(slots, h, w, c)) return 0;
  return (size_t)slots * (size_t)((long long)h * w * row_bytes(fmt, c));
}

size_t mqconv_cache_scales_bytes(int32_t slots, int32_t h, int32_t w, int32_t c) {
  if (!cache_dims_ok(slots, h, w, c)) return 0;
  return (size_t)slots * (size_t)((long long)h * w * ((c + 31LL) / 32));
}

int mqconv_cache_write(mq_cache cache, const float* x, int32_t n, int32_t n0, int32_t count, const int32_t* slot,
                       void* stream) {
  CacheView v;
  if (!x) return MQ_ERR_NULL;
  const int e = check_cache(cache, slot, &v);
  if (e != MQ_OK) return e;
  if (!range_ok(cache, n, n0, count) || count > MQ_CACHE_COUNT_MAX) return MQ_ERR_SHAPE;
  if (!aligned4(x)) return MQ_ERR_ALIGN;
  return hip_status(launch_cache_write(v, x, n, n0, count, slot, (hipStream_t)stream));
}

int mqconv_cache_read(mq_cache cache, const int32_t* slot, int32_t count, float* x, int32_t n, int32_t n0,
                      void* stream) {
  CacheView v;
  if (!x) return MQ_ERR_NULL;
  const int e = check_cache(cache, slot, &v);
  if (e != MQ_OK) return e;
  if (!range_ok(cache, n, n0, count)) return MQ_ERR_SHAPE;
  if (!aligned4(x)) return MQ_ERR_ALIGN;
  return hip_status(launch_cache_read(v, slot, count, x, n, n0, (hipStream_t)stream));
}

int mqconv_cache_read_mx(mq_cache cache, const int32_t* slot, mq_mx xq, void* stream) {
  CacheView v;
  int e = check_cache(cache, slot, &v);
  if (e != MQ_OK) return e;
  if ((e = check_mx(xq, MQ_ROLE_ACT, cache.h, cache.w, xq.d2, cache.c)) != MQ_OK) return e;
  if (!dims_ok(xq.d0, xq.d1, xq.d2, xq.d3)) return MQ_ERR_SHAPE;
  return hip_status(launch_cache_read_mx(v, slot, xq.d2, out_view(xq), (hipStream_t)stream));
}

}  // extern "C"
