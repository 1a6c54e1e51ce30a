// layer_norm_mx.hip -- the second pass of layer norm and of its gradient with
// MX output: every value again from x (and dy) and its row's parameters,
// quantized in place (mx_rows.h).
#include "layer_norm.h"
#include "mx_rows.h"

namespace mq {

namespace {

template <bool FULL>
__device__ __forceinline__ void load_or(const float* p, int c0, int cnt, float other, float (&v)[16]) {
  if (p) load_run<16, FULL>(p + c0, cnt, v);
  else {
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = other;
  }
}

template <bool FULL>
struct LnSrc {
  LnArgs a;
  int N;
  struct State {
    float gamma[16], beta[16];
  };
  struct Raw {
    float x[16], mean, rstd;
  };
  __device__ void rows(State&, int, int) const {}
  __device__ void params(State& s, int, int c0, int cnt) const {
    load_or<FULL>(a.gamma, c0, cnt, 1.0f, s.gamma);
    load_or<FULL>(a.beta, c0, cnt, 0.0f, s.beta);
  }
  __device__ void load(const State&, Raw& r, int p, int n, int c0, int cnt) const {
    const int row = p * N + n;
    load_run<16, FULL>(a.x + (long long)row * a.C + c0, cnt, r.x);
    r.mean = a.mean_in[row];
    r.rstd = a.rstd_in[row];
  }
  __device__ void values(const State& s, const Raw& r, int, int, int c0, float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = FULL || c0 + i < a.C ? ln_value(r.x[i], r.mean, r.rstd, s.gamma[i], s.beta[i]) : 0.0f;
  }
  __device__ void extra(int, int) const {}
};

template <bool FULL, bool ADD>
struct LnGradSrc {
  LnArgs a;
  int N;
  struct State {
    float gamma[16];
  };
  struct Raw {
    float x[16], dy[16], add[ADD ? 16 : 1], mean, rstd;
    LnRow k;
  };
  __device__ void rows(State&, int, int) const {}
  __device__ void params(State& s, int, int c0, int cnt) const { load_or<FULL>(a.gamma, c0, cnt, 1.0f, s.gamma); }
  __device__ void load(const State&, Raw& r, int p, int n, int c0, int cnt) const {
    const int row = p * N + n;
    const long long at = (long long)row * a.C + c0;
    load_run<16, FULL>(a.x + at, cnt, r.x);
    load_run<16, FULL>(a.dy + at, cnt, r.dy);
    if constexpr (ADD) load_run<16, FULL>(a.add + at, cnt, r.add);
    r.mean = a.mean_in[row];
    r.rstd = a.rstd_in[row];
    r.k = a.row[row];
  }
  __device__ void values(const State& s, const Raw& r, int, int, int c0, float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const float g = r.dy[i] * s.gamma[i], xh = ln_hat(r.x[i], r.mean, r.rstd);
      float d;
      if constexpr (ADD) d = ln_grad(g, xh, r.k.k1, r.k.k2, r.rstd, r.add[i]);
      else d = ln_grad(g, xh, r.k.k1, r.k.k2, r.rstd);
      v[i] = FULL || c0 + i < a.C ? d : 0.0f;
    }
  }
  __device__ void extra(int, int) const {}
};

}  // namespace

hipError_t launch_layer_norm_mx_rows(const LnArgs& a, int N, const MxOutView& out, hipStream_t st) {
  const MxRows g = mx_rows(out, a.R / N, N, a.C);
  return a.C % 16 == 0 ? launch_mx_rows(out.fmt, LnSrc<true>{a, N}, g, 0, st)
                       : launch_mx_rows(out.fmt, LnSrc<false>{a, N}, g, 0, st);
}

hipError_t launch_layer_norm_grad_mx_rows(const LnArgs& a, int N, const MxOutView& out, hipStream_t st) {
  const MxRows g = mx_rows(out, a.R / N, N, a.C);
  const bool full = a.C % 16 == 0;
  if (a.add)
    return full ? launch_mx_rows(out.fmt, LnGradSrc<true, true>{a, N}, g, 0, st)
                : launch_mx_rows(out.fmt, LnGradSrc<false, true>{a, N}, g, 0, st);
  return full ? launch_mx_rows(out.fmt, LnGradSrc<true, false>{a, N}, g, 0, st)
              : launch_mx_rows(out.fmt, LnGradSrc<false, false>{a, N}, g, 0, st);
}

}  // namespace mq
