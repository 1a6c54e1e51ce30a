// dropout.hip -- dropout from a counter-based generator: y = drop(x) +
// residual. The mask is a function of an element's place and the seed, so
// nothing is stored and the backward pass is the same kernel on the gradient.
// Memory bound: x (and residual) read once, y written once; the Philox block
// that decides eight neighbouring channels is computed while the loads are
// in flight. 80 x 80 x 32 x 256 with a residual: 629 MB in 116.7 us, 5.4 TB/s,
// what a copy reaches.
#include <math.h>

#include "block.h"
#include "mx_rows.h"

namespace mq {

DropArgs drop_args(const DropSpec& d) {
  DropArgs a{};
  a.seed = d.seed;
  a.step = d.step;
  a.q = (uint32_t)floor((double)d.p * 65536.0 + 0.5);
  a.scale = a.q < 65536u ? (float)(65536.0 / (65536.0 - (double)a.q)) : 0.0f;
  return a;
}

// A thread takes octets of channels i, i + gridDim.x * 256, ... of the
// [rows][octets] grid, kDropUnroll of them in flight.
constexpr int kDropUnroll = 2;
template <bool RES, bool FULL>
__global__ __launch_bounds__(256) void dropout_kernel(const float* x, const float* res, float* y, int C, int NO,
                                                      FastDiv dNO, int total, DropArgs d) {
  const DropKey key = drop_key(d);
  const int stride = gridDim.x * 256;
  for (int i0 = blockIdx.x * 256 + threadIdx.x; i0 < total; i0 += kDropUnroll * stride) {
    float v[kDropUnroll][8], r[RES ? kDropUnroll : 1][8];
    uint32_t row[kDropUnroll], oct[kDropUnroll];
    int cnt[kDropUnroll];
    long long at[kDropUnroll];
#pragma unroll
    for (int u = 0; u < kDropUnroll; u++) {
      const int i = i0 + u * stride, j = i < total ? i : 0;  // (i is below 2^30 + 2^20)
      row[u] = fdiv((unsigned)j, dNO);
      oct[u] = (uint32_t)j - row[u] * NO;
      cnt[u] = i < total ? min(8, C - (int)oct[u] * 8) : 0;
      at[u] = (long long)row[u] * C + oct[u] * 8;
      load_run<8, FULL>(x + at[u], cnt[u], v[u]);
      if constexpr (RES) load_run<8, FULL>(res + at[u], cnt[u], r[u]);
    }
#pragma unroll
    for (int u = 0; u < kDropUnroll; u++) {
      drop_values<8>(d, key, row[u], oct[u] * 8, v[u]);
      if constexpr (RES) {
#pragma clang fp contract(off)
#pragma unroll
        for (int j = 0; j < 8; j++) v[u][j] = v[u][j] + r[u][j];
      }
      store_run<8, FULL>(y + at[u], cnt[u], v[u]);
    }
  }
}

hipError_t launch_dropout(const float* x, const float* residual, int rows, int C, const DropSpec& drop, float* y,
                          hipStream_t st) {
  const int NO = ceil_div(C, 8);
  const int total = rows * NO;
  const int need = ceil_div(total, 256 * kDropUnroll);
  const dim3 grid((unsigned)(need < 2048 ? need : 2048));
  const FastDiv dNO = make_fastdiv((unsigned)NO);
  const DropArgs d = drop_args(drop);
  const bool full = C % 8 == 0;
  const auto kern = residual ? (full ? dropout_kernel<true, true> : dropout_kernel<true, false>)
                             : (full ? dropout_kernel<false, true> : dropout_kernel<false, false>);
  hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, x, residual, y, C, NO, dNO, total, d);
  return launch_check();
}

// The same values as MX codes.
template <bool FULL>
struct DropSrc {
  const float* x;
  int N, C;
  DropArgs d;
  struct State {
    DropKey key;
  };
  struct Raw {
    float x[16];
  };
  __device__ void rows(State&, int, int) const {}
  __device__ void params(State& s, int, int, int) const { s.key = drop_key(d); }
  __device__ void load(const State&, Raw& r, int p, int n, int c0, int cnt) const {
    load_run<16, FULL>(x + ((long long)p * N + n) * C + c0, cnt, r.x);
  }
  __device__ void values(const State& s, const Raw& r, int p, int n, int c0, float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = r.x[i];
    drop_values<16>(d, s.key, (uint32_t)p * N + n, c0, v);
  }
  __device__ void extra(int, int) const {}
};

hipError_t launch_dropout_mx(const float* x, int P, int N, int C, const DropSpec& drop, const MxOutView& out,
                             hipStream_t st) {
  const MxRows g = mx_rows(out, P, N, C);
  const DropArgs d = drop_args(drop);
  return C % 16 == 0 ? launch_mx_rows(out.fmt, DropSrc<true>{x, N, C, d}, g, 0, st)
                     : launch_mx_rows(out.fmt, DropSrc<false>{x, N, C, d}, g, 0, st);
}

}  // namespace mq
