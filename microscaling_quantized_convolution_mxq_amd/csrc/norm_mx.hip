// norm_mx.hip -- the elementwise pass of group norm and of its gradient with
// MX output: every value is made again from x (and dy) and the columns'
// parameters, and quantized in place (mx_rows.h).
#include "mx_rows.h"
#include "norm.h"

namespace mq {

struct NormSrc {
  NormArgs a;
  struct State {
    float mean[16], a[16], be[16];
    DropKey key;
  };
  struct Raw {
    float x[16];
  };
  __device__ void init(State& s, int n, int c0, int cnt) const {
    const long long col = (long long)n * a.g.C + c0;
    load_run<16>(a.col.mean + col, cnt, s.mean);
    load_run<16>(a.col.a + col, cnt, s.a);
    load_run<16>(a.beta + c0, a.beta ? cnt : 0, s.be);
    s.key = drop_key(a.drop);
  }
  __device__ void load(const State&, Raw& r, int p, int n, int c0, int cnt) const {
    load_run<16>(a.x + ((long long)p * a.g.N + n) * a.g.C + c0, cnt, r.x);
  }
  __device__ void values(const State& s, const Raw& r, int p, int n, int c0, float (&v)[16]) const {
    float d[16];
#pragma unroll
    for (int i = 0; i < 16; i++) d[i] = r.x[i];
    norm_values<16>(s.mean, s.a, s.be, d, v);
    act_values<16>(a.act, v);
    drop_values<16>(a.drop, s.key, (uint32_t)p * a.g.N + n, c0, v);
  }
  __device__ void extra(int) const {}
};

hipError_t launch_norm_mx(const NormArgs& a, const MxOutView& out, hipStream_t st) {
  return launch_mx_rows(out.fmt, NormSrc{a}, mx_rows(out, a.g.P, a.g.N, a.g.C), 0, st);
}

struct NormGradSrc {
  NormArgs a;
  struct State {
    float mean[16], a[16], be[16], k1[16], k2[16];
    DropKey key;
  };
  struct Raw {
    float x[16], dy[16];
  };
  __device__ void init(State& s, int n, int c0, int cnt) const {
    const long long col = (long long)n * a.g.C + c0;
    load_run<16>(a.col.mean + col, cnt, s.mean);
    load_run<16>(a.col.a + col, cnt, s.a);
    load_run<16>(a.col.k1 + col, cnt, s.k1);
    load_run<16>(a.col.k2 + col, cnt, s.k2);
    load_run<16>(a.beta + c0, a.beta ? cnt : 0, s.be);
    s.key = drop_key(a.drop);
  }
  __device__ void load(const State&, Raw& r, int p, int n, int c0, int cnt) const {
    const long long at = ((long long)p * a.g.N + n) * a.g.C + c0;
    load_run<16>(a.x + at, cnt, r.x);
    load_run<16>(a.dy + at, cnt, r.dy);
  }
  __device__ void values(const State& s, const Raw& r, int p, int n, int c0, float (&v)[16]) const {
    float d[16], u[16], g[16];
#pragma unroll
    for (int i = 0; i < 16; i++) {
      d[i] = r.x[i];
      g[i] = r.dy[i];
    }
    norm_values<16>(s.mean, s.a, s.be, d, u);
    drop_values<16>(a.drop, s.key, (uint32_t)p * a.g.N + n, c0, g);
    act_slopes<16>(a.act, u, g);
    norm_grad_values<16>(s.a, s.k1, s.k2, d, g, v);
  }
  __device__ void extra(int b) const { norm_channel_sums(a, b); }
};

hipError_t launch_norm_backward_mx(const NormArgs& a, const MxOutView& out, int extra, hipStream_t st) {
  return launch_mx_rows(out.fmt, NormGradSrc{a}, mx_rows(out, a.g.P, a.g.N, a.g.C), extra, st);
}

}  // namespace mq
