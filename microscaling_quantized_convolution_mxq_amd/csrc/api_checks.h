// api_checks.h -- argument checks shared by the C ABI's translation units
// (host only; nothing here makes a HIP call).
#pragma once
#include "mqconv.h"
#include "mqconv_internal.h"

namespace mq {

// Kernels address packed tensors with 32-bit byte offsets (buffer loads), so
// every tensor is limited to 2^30 elements (channel padding included).
const long long kMaxElems = 1LL << 30;

inline bool fmt_ok(int f) { return f >= MQ_E4M3 && f <= MQ_E2M1; }
inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool dims_ok(int32_t d0, int32_t d1, int32_t d2, int32_t d3) {
  if (d0 < 1 || d1 < 1 || d2 < 1 || d3 < 1) return false;
  long long n = (long long)d0 * d1;
  if (n > kMaxElems) return false;
  n *= d2;
  if (n > kMaxElems) return false;
  long long cpad = ((long long)d3 + 31) / 32 * 32;
  return n * cpad <= kMaxElems;
}

// Checks a packed tensor view against a role and expected dims.
inline int check_mx(const mq_mx& t, mq_role role, int32_t d0, int32_t d1, int32_t d2, int32_t d3) {
  if (!t.codes || !t.scales) return MQ_ERR_NULL;
  if (!fmt_ok(t.fmt)) return MQ_ERR_FORMAT;
  if (t.role != role) return MQ_ERR_FORMAT;
  if (t.block_partner != 1 && t.block_partner != 32) return MQ_ERR_UNSUPPORTED;
  if (t.d0 != d0 || t.d1 != d1 || t.d2 != d2 || t.d3 != d3) return MQ_ERR_SHAPE;
  if (!aligned16(t.codes) || !aligned16(t.scales)) return MQ_ERR_ALIGN;
  return MQ_OK;
}

// Element counts of the conv's tensors (0 if the geometry is invalid).
inline bool conv_ok(const mq_conv* c) {
  if (!c) return false;
  if (c->n < 1 || c->cin < 1 || c->h < 1 || c->w < 1 || c->cout < 1) return false;
  if (c->kh < 1 || c->kw < 1 || c->kh > 15 || c->kw > 15) return false;
  if (c->stride_h < 1 || c->stride_w < 1 || c->stride_h > 8 || c->stride_w > 8) return false;
  if (c->pad_h < 0 || c->pad_w < 0 || c->pad_h >= c->kh || c->pad_w >= c->kw) return false;
  long long ho = ((long long)c->h + 2LL * c->pad_h - c->kh) / c->stride_h + 1;
  long long wo = ((long long)c->w + 2LL * c->pad_w - c->kw) / c->stride_w + 1;
  if (c->h + 2LL * c->pad_h < c->kh || c->w + 2LL * c->pad_w < c->kw) return false;
  if (ho < 1 || wo < 1) return false;
  long long cpi = ((long long)c->cin + 31) / 32 * 32, cpo = ((long long)c->cout + 31) / 32 * 32;
  long long npad = ((long long)c->n + 31) / 32 * 32;
  if ((long long)c->h * c->w * npad * cpi > kMaxElems) return false;
  if (ho * wo * npad * cpo > kMaxElems) return false;
  if (ho * wo * c->n * (long long)c->kh * c->kw * cpi > kMaxElems) return false;
  if ((long long)c->cout * c->kh * c->kw * cpi > kMaxElems) return false;
  return true;
}

inline Conv to_conv(const mq_conv* c) {
  Conv v;
  v.n = c->n; v.cin = c->cin; v.h = c->h; v.w = c->w; v.cout = c->cout; v.kh = c->kh; v.kw = c->kw;
  v.sh = c->stride_h; v.sw = c->stride_w; v.ph = c->pad_h; v.pw = c->pad_w;
  return v;
}

inline MxOutView out_view(const mq_mx& t) {
  return MxOutView{static_cast<uint8_t*>(t.codes), t.scales, t.fmt, t.block_partner};
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? MQ_OK : MQ_ERR_HIP; }

}  // namespace mq
