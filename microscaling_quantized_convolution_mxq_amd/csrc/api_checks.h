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

inline int hip_status(hipError_t e) { return e == hipSuccess ? MQ_OK : MQ_ERR_HIP; }

}  // namespace mq
