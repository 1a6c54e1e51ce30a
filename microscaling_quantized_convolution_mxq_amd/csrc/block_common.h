// block_common.h -- device-side pieces of the group norm, dropout and replay
// cache kernels: channel octets of fp32 rows, activations and their slopes,
// and the dropout factor of an element.
//
// Values that two kernels must agree on to the bit (an fp32 result and the MX
// codes of the same result) are written with explicit fused multiply-adds and
// contraction off, so that no kernel rounds them in its own way.
#pragma once
#include "mx_common.h"
#include "mqconv_internal.h"
#include "philox.h"

namespace mq {

// Kernels are built for each activation: GELU's integral costs registers that
// the others need for values in flight.
enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };
template <int A>
struct ActTag {
  static constexpr int value = A;
};
// f(an ActTag of the activation)
template <class F>
auto with_act(int act, F&& f) {
  switch (act) {
    case kActNone: return f(ActTag<kActNone>{});
    case kActRelu: return f(ActTag<kActRelu>{});
    case kActSilu: return f(ActTag<kActSilu>{});
    default: return f(ActTag<kActGelu>{});
  }
}

// Four floats at any 4-byte aligned address (one 16-byte access: global
// memory accesses need no more than dword alignment).
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));

// cnt (of 8, or of 16) consecutive values at p; zeros past cnt. FULL: all K
// whatever cnt is, so p must be readable. Channel counts that are multiples
// of K take such kernels, whose loads stand under no condition (their callers
// move an address out of range to one in range and leave its values out): the
// compiler can then count which loads are under way, and waits for a pixel's
// values only, not for those it has just requested.
// Partial runs go by quads, so only a run whose end is no multiple of four
// takes single loads.
template <int K, bool FULL = false>
__device__ __forceinline__ void load_run(const float* p, int cnt, float (&v)[K]) {
#pragma unroll
  for (int i = 0; i < K; i += 4) {
    if (FULL || cnt >= i + 4) {
      const f4u t = *reinterpret_cast<const f4u*>(p + i);
#pragma unroll
      for (int j = 0; j < 4; j++) v[i + j] = t[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; j++) v[i + j] = 0.0f;
      if (cnt > i) {
#pragma unroll
        for (int j = 0; j < 3; j++)
          if (i + j < cnt) v[i + j] = p[i + j];
      }
    }
  }
}
// FULL: cnt is 0 or K.
template <int K, bool FULL = false>
__device__ __forceinline__ void store_run(float* p, int cnt, const float (&v)[K]) {
  if (FULL && cnt <= 0) return;
#pragma unroll
  for (int i = 0; i < K; i += 4) {
    if (FULL || cnt >= i + 4) {
      f4u t;
#pragma unroll
      for (int j = 0; j < 4; j++) t[j] = v[i + j];
      *reinterpret_cast<f4u*>(p + i) = t;
    } else if (cnt > i) {
#pragma unroll
      for (int j = 0; j < 3; j++)
        if (i + j < cnt) p[i + j] = v[i + j];
    }
  }
}

// exp(-u) as 2^(-u log2(e)): the rounding of the product is |u| 2^-24 of the
// result, which a sigmoid s passes on times s (1 - s); a correction for it took
// as long as the rest. Overflow to infinity makes a sigmoid 0, as it should.
__device__ __forceinline__ float exp_neg(float u) { return __builtin_amdgcn_exp2f(u * -1.4426950408889634f); }
__device__ __forceinline__ float sigmoid(float u) { return __builtin_amdgcn_rcpf(1.0f + exp_neg(u)); }
// The normal distribution: e = exp(-u^2 / 2) and the integral cdf up to u. The
// tail is e t P(t) with t = 1 / (1 + 0.38 |u|) and P of degree 9, fitted to the
// smallest largest relative error over |u| <= 14 (9e-9; 4.5 2^-24 as evaluated
// here), so below 0 cdf keeps its digits, which 1 + erf loses, but for the
// rounding of e's argument: u^2 2^-24 times 1.3 of the result. One exponential
// for both. Group norm of 160 x 160 x 32 x 128 245 us, 299 by a call of erfc.
struct Normal {
  float e, cdf;
};
__device__ __forceinline__ Normal normal(float u) {
#pragma clang fp contract(off)
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.38f, fabsf(u), 1.0f));
  float p = 0.0242854198f;
  p = __builtin_fmaf(p, t, -0.149213825f);
  p = __builtin_fmaf(p, t, 0.368569631f);
  p = __builtin_fmaf(p, t, -0.434484348f);
  p = __builtin_fmaf(p, t, 0.210207231f);
  p = __builtin_fmaf(p, t, -0.0559188846f);
  p = __builtin_fmaf(p, t, 0.106472857f);
  p = __builtin_fmaf(p, t, 0.126635639f);
  p = __builtin_fmaf(p, t, 0.151857647f);
  p = __builtin_fmaf(p, t, 0.151588629f);
  const float e = __builtin_amdgcn_exp2f(u * u * -0.72134752f);
  const float tail = e * (t * p);
  return Normal{e, u > 0.0f ? 1.0f - tail : tail};
}

// The activation of every value of u, in place.
template <int ACT, int K>
__device__ __forceinline__ void act_values(float (&u)[K]) {
#pragma clang fp contract(off)
  if constexpr (ACT == kActSilu) {
#pragma unroll
    for (int i = 0; i < K; i++) u[i] = u[i] * sigmoid(u[i]);
  } else if constexpr (ACT == kActRelu) {
#pragma unroll
    for (int i = 0; i < K; i++) u[i] = u[i] < 0.0f ? 0.0f : u[i];
  } else if constexpr (ACT == kActGelu) {
#pragma unroll
    for (int i = 0; i < K; i++) u[i] = u[i] * normal(u[i]).cdf;
  }
}
// g *= act'(u).
template <int ACT, int K>
__device__ __forceinline__ void act_slopes(const float (&u)[K], float (&g)[K]) {
#pragma clang fp contract(off)
  if constexpr (ACT == kActSilu) {
#pragma unroll
    for (int i = 0; i < K; i++) {
      const float s = sigmoid(u[i]);
      g[i] = g[i] * (s * __builtin_fmaf(u[i], 1.0f - s, 1.0f));
    }
  } else if constexpr (ACT == kActRelu) {
    // (a product, not a select: a NaN in u or g stays one)
#pragma unroll
    for (int i = 0; i < K; i++) g[i] = u[i] != u[i] ? u[i] : g[i] * (u[i] > 0.0f ? 1.0f : 0.0f);
  } else if constexpr (ACT == kActGelu) {
#pragma unroll
    for (int i = 0; i < K; i++) {
      const Normal d = normal(u[i]);
      g[i] = g[i] * __builtin_fmaf(u[i] * 0.39894228f, d.e, d.cdf);
    }
  }
}

// Dropout of one call: elements whose 16-bit number is below q are dropped
// (q = 0: none are), the others multiplied by scale.
struct DropArgs {
  uint64_t seed;
  const uint64_t* step;
  uint32_t q;
  float scale;
};
struct DropKey {
  uint32_t k0, k1;
};
__device__ __forceinline__ DropKey drop_key(const DropArgs& d) {
  if (d.q == 0) return DropKey{0, 0};
  const uint64_t s = d.seed + (d.step ? *d.step : 0);
  return DropKey{(uint32_t)s, (uint32_t)(s >> 32)};
}
// Dropout of channels c0 .. c0 + K - 1 (c0 a multiple of 8) of a row: one
// Philox block, eight 16-bit numbers, for each octet of channels. 32 bits an
// element would double the generator's work (20 64-bit products a block, about
// as long as the memory takes to bring the eight values) for a probability
// that is finer than 1.5e-5.
template <int K>
__device__ __forceinline__ void drop_values(const DropArgs& d, const DropKey& k, uint32_t row, uint32_t c0,
                                            float (&v)[K]) {
  if (d.q == 0) return;
#pragma unroll
  for (int b = 0; b < K / 8; b++) {
    uint32_t o[4];
    philox4x32_10(row, (c0 >> 3) + b, 1u, 0u, k.k0, k.k1, o);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t r = (i & 1) ? o[i >> 1] >> 16 : o[i >> 1] & 0xffffu;
      v[8 * b + i] = r < d.q ? 0.0f : v[8 * b + i] * d.scale;
    }
  }
}

}  // namespace mq
