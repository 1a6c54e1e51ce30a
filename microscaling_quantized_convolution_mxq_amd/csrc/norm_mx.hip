// norm_mx.hip -- the elementwise pass of group norm and of its gradient with
// MX output: every value is made again from x (and dy) and the columns'
// parameters, and quantized in place (mx_rows.h). A read of x (and dy) and a
// quarter of that or less written: 80 x 80 x 16 x 64 with SiLU and dropout
// takes 12.2 us (33 MB; sigmoid, Philox and packing beside the loads: vector
// instructions issue in 58% of the busy cycles), the gradient of 20 x 20 x 128 x
// 256 26.3 us (118 MB, 4.5 TB/s, 55%; its five parameters a channel leave
// registers for eight waves a compute unit, and four for sixteen made it spill
// and take 35 us).
#include "mx_rows.h"
#include "norm.h"

namespace mq {

template <bool FULL, int ACT>
struct NormSrc {
  NormArgs a;
  struct State {
    float mean[16], a[16], be[16];
    DropKey key;
  };
  struct Raw {
    float x[16];
  };
  __device__ void rows(State&, int, int) const {}
  __device__ void params(State& s, int n, int c0, int cnt) const {
    const long long col = (long long)n * a.g.C + c0;
    load_run<16, FULL>(a.col.mean + col, cnt, s.mean);
    load_run<16, FULL>(a.col.a + col, cnt, s.a);
    if (a.beta) load_run<16, FULL>(a.beta + c0, cnt, s.be);
    else {
#pragma unroll
      for (int i = 0; i < 16; i++) s.be[i] = 0.0f;
    }
    s.key = drop_key(a.drop);
  }
  __device__ void load(const State&, Raw& r, int p, int n, int c0, int cnt) const {
    load_run<16, FULL>(a.x + ((long long)p * a.g.N + n) * a.g.C + c0, cnt, r.x);
  }
  __device__ void values(const State& s, const Raw& r, int p, int n, int c0, float (&v)[16]) const {
    float d[16];
#pragma unroll
    for (int i = 0; i < 16; i++) d[i] = r.x[i];
    norm_values<16>(s.mean, s.a, s.be, d, v);
    act_values<ACT, 16>(v);
    drop_values<16>(a.drop, s.key, (uint32_t)p * a.g.N + n, c0, v);
  }
  __device__ void extra(int, int) const {}
};

template <bool FULL, int ACT>
struct NormGradSrc {
  NormArgs a;
  struct State {
    float mean[16], a[16], be[16], k1[16], k2[16];
    DropKey key;
  };
  struct Raw {
    float x[16], dy[16];
  };
  __device__ void rows(State&, int, int) const {}
  __device__ void params(State& s, int n, int c0, int cnt) const {
    const long long col = (long long)n * a.g.C + c0;
    load_run<16, FULL>(a.col.mean + col, cnt, s.mean);
    load_run<16, FULL>(a.col.a + col, cnt, s.a);
    load_run<16, FULL>(a.col.k1 + col, cnt, s.k1);
    load_run<16, FULL>(a.col.k2 + col, cnt, s.k2);
    if (a.beta) load_run<16, FULL>(a.beta + c0, cnt, s.be);
    else {
#pragma unroll
      for (int i = 0; i < 16; i++) s.be[i] = 0.0f;
    }
    s.key = drop_key(a.drop);
  }
  __device__ void load(const State&, Raw& r, int p, int n, int c0, int cnt) const {
    const long long at = ((long long)p * a.g.N + n) * a.g.C + c0;
    load_run<16, FULL>(a.x + at, cnt, r.x);
    load_run<16, FULL>(a.dy + at, cnt, r.dy);
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
    act_slopes<ACT, 16>(u, g);
    norm_grad_values<16>(s.a, s.k1, s.k2, d, g, v);
  }
  __device__ void extra(int b, int n) const { norm_channel_sums(a, b, n); }
};

namespace {
template <template <bool, int> class Src>
hipError_t launch(const NormArgs& a, const MxOutView& out, int extra, hipStream_t st) {
  const MxRows g = mx_rows(out, a.g.P, a.g.N, a.g.C);
  return with_act(a.act, [&](auto act) {
    constexpr int A = decltype(act)::value;
    return a.g.C % 16 == 0 ? launch_mx_rows(out.fmt, Src<true, A>{a}, g, extra, st)
                           : launch_mx_rows(out.fmt, Src<false, A>{a}, g, extra, st);
  });
}
}  // namespace

hipError_t launch_norm_mx(const NormArgs& a, const MxOutView& out, hipStream_t st) {
  return launch<NormSrc>(a, out, 0, st);
}
hipError_t launch_norm_backward_mx(const NormArgs& a, const MxOutView& out, int extra, hipStream_t st) {
  return launch<NormGradSrc>(a, out, extra, st);
}

}  // namespace mq
