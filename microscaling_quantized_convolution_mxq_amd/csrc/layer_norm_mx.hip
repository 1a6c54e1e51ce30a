// layer_norm_mx.hip -- layer norm and its gradient with MX output.
//
// Rows of 33 to 256 channels (a multiple of four) take one pass: a workgroup
// takes the 32 rows at most of one tile of blocks, whole pixels where a pixel
// has fewer samples, computes them as the fp32 form does, leaves their values
// in LDS and quantizes them from there, so x (and dy) are read once and nothing
// but codes and scales is written. All rows' loads of a tile are under way at
// once, and a compute unit holds several workgroups (the next tile's requested
// before this one's codes: the gradient of 20 x 20 x 128 x 256 61 us instead of
// 41). Measured: 80 x 80
// x 16 x 64 to E4M3 12.6 us (33 MB, 2.6 TB/s: a third of it is the rows' fp64
// sums), 19 in two passes; the gradient of 20 x 20 x 128 x 256 with a skip
// path to E5M2 39.5 us (170 MB, 4.3 TB/s), 61 in two.
// Other rows take two: the fp32 form's pass leaves each row's parameters, and the
// second computes every value again from them, quantized in place (mx_rows.h).
#include <algorithm>

#include "layer_norm_rows.h"
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

// ---- one pass -----------------------------------------------------------------------------------
constexpr int kThreads = 256;

struct Tiles {
  MxRows g;
  int fmt, across, tiles;  // across: tiles of a pixel's samples
};
struct TileAt {
  int p0, n0, rows;
  long long row0;
};
__device__ __forceinline__ TileAt tile_at(const Tiles& u, int id) {
  const int tp = id / u.across, nt = id - tp * u.across;
  TileAt t;
  t.p0 = tp * u.g.ppt;
  t.n0 = nt * 32;
  t.rows = min(u.g.ppt, u.g.P - t.p0) * min(32, u.g.N - t.n0);
  t.row0 = (long long)t.p0 * u.g.N + t.n0;
  return t;
}

template <int T>
struct TileLds {
  static constexpr int PITCH = 4 * T + 4;
  float y[32 * PITCH];  // (a row's pitch moves the next row to other banks)
  uint8_t codes[32 * (4 * T)];
};

// A tile's values from LDS to codes and scales, by the quantizer's functions in its arrangement: a wave takes 32 rows of a block
// of 32 channels, two lanes a row.
template <int T>
__device__ __forceinline__ void quantize_tile(const Tiles& u, const TileAt& t, TileLds<T>& lds) {
  const MxRows& g = u.g;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane >> 1, half = lane & 1;
  const int psub = r / g.grp, in = r - psub * g.grp, n = t.n0 + in, p = t.p0 + psub, srow = psub * g.N + in;
  const bool row_ok = n < g.N && psub < g.ppt && p < g.P;
  const auto blocks = [&](auto f) {
    constexpr int F = decltype(f)::value, RB = run_bytes_of(F);
    for (int cb = wave; cb < g.nCB; cb += kThreads / 64) {
      const float* const from = lds.y + (row_ok ? srow : 0) * TileLds<T>::PITCH + cb * 32 + half * 16;
      float x[16], v[16];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 16; i++) {
        x[i] = row_ok ? from[i] : 0.0f;
        m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
      }
      const uint32_t S = scale_byte_from_amax<F>(group_max(m, g.glanes));
      scale_clamp16<F>(x, S, v);
      if (!row_ok) continue;
      convert_store_half_run<F>(lds.codes + (srow * g.nCB + cb) * RB + half * (RB / 2), v, code_keep(S));
      if (half != 0) continue;
      if (g.bp == 1) g.scales[((long long)p * g.N + n) * g.nCB + cb] = (uint8_t)S;
      else if ((n & 31) == 0) g.scales[((long long)p * g.nPB + (n >> 5)) * g.nCB + cb] = (uint8_t)S;
    }
  };
  switch (u.fmt) {
    case 0: blocks(std::integral_constant<int, 0>{}); break;
    case 1: blocks(std::integral_constant<int, 1>{}); break;
    case 2: blocks(std::integral_constant<int, 2>{}); break;
    case 3: blocks(std::integral_constant<int, 3>{}); break;
    default: blocks(std::integral_constant<int, 4>{}); break;
  }
  __syncthreads();
  // whole rows: one stretch
  const int rb = g.nCB * run_bytes_of(u.fmt), pieces = t.rows * rb / 8;
  uint2* const to = reinterpret_cast<uint2*>(g.codes + t.row0 * rb);
  for (int i = threadIdx.x; i < pieces; i += kThreads) to[i] = reinterpret_cast<const uint2*>(lds.codes)[i];
}

// A row's values to LDS, zeros up to a whole block.
template <int T>
__device__ __forceinline__ void leave_row(const Tiles& u, TileLds<T>& lds, int i, int t, const quad_t (&v)[1], int C) {
  const int c = 4 * t;
  if (c < 32 * u.g.nCB)
    *reinterpret_cast<float4*>(lds.y + i * TileLds<T>::PITCH + c) =
        c < C ? make_float4(v[0][0], v[0][1], v[0][2], v[0][3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}

template <int T, bool ADD>
__global__ __launch_bounds__(kThreads) void ln_mx_kernel(const LnArgs a, const Tiles u) {
  __shared__ __attribute__((aligned(16))) TileLds<T> lds;
  constexpr int G = kThreads / T, K = 32 / G;
  const int t = threadIdx.x % T, i0 = threadIdx.x / T;
  quad_t gamma[1], beta[1];
  load_param<T, 1, true>(a.gamma, a.C, t, 1.0f, gamma);
  load_param<T, 1, true>(a.beta, a.C, t, 0.0f, beta);
  for (int id = blockIdx.x; id < u.tiles; id += gridDim.x) {
    const TileAt at = tile_at(u, id);
    quad_t v[K][1], more[ADD ? K : 1][1];
#pragma unroll
    for (int k = 0; k < K; k++) {
      const int i = k * G + i0;
      const long long row = at.row0 + (i < at.rows ? i : 0);
      load_row<T, 1, true>(a.x + row * a.C, a.C, t, v[k]);
      if constexpr (ADD) load_row<T, 1, true>(a.add + row * a.C, a.C, t, more[k]);
    }
#pragma unroll
    for (int k = 0; k < K; k++) {
      const int i = k * G + i0;
      const bool row_ok = i < at.rows;
      const long long row = at.row0 + i;
      double s[1] = {0};
#pragma unroll
      for (int e = 0; e < 4; e++) {
        if constexpr (ADD) v[k][0][e] += more[k][0][e];
        s[0] += has<T, true>(0, e, t, a.C) ? (double)v[k][0][e] : 0.0;
      }
      if (ADD && row_ok) store_row<T, 1, true>(a.sum + row * a.C, a.C, t, v[k]);
      row_sums<T, 1>(s, 0);
      const double mean = s[0] * a.inv;
      s[0] = 0;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const double d = has<T, true>(0, e, t, a.C) ? (double)v[k][0][e] - mean : 0.0;
        s[0] = __builtin_fma(d, d, s[0]);
      }
      row_sums<T, 1>(s, 1);
      const float m = (float)mean, rs = rstd_of(s[0], a);
      if (t == 0 && row_ok) {
        if (a.mean) a.mean[row] = m;
        if (a.rstd) a.rstd[row] = rs;
      }
#pragma unroll
      for (int e = 0; e < 4; e++) v[k][0][e] = ln_value(v[k][0][e], m, rs, gamma[0][e], beta[0][e]);
      leave_row<T>(u, lds, i, t, v[k], a.C);
    }
    __syncthreads();
    quantize_tile<T>(u, at, lds);
  }
}

template <int T, bool ADD>
__global__ __launch_bounds__(kThreads) void ln_grad_mx_kernel(const LnArgs a, const Tiles u) {
  __shared__ __attribute__((aligned(16))) TileLds<T> lds;
  constexpr int G = kThreads / T, K = 32 / G;
  static_assert(sizeof(lds) >= (kThreads / 64 - 1) * T * 4 * sizeof(double2), "column sums");
  const int t = threadIdx.x % T, i0 = threadIdx.x / T;
  quad_t gamma[1];
  load_param<T, 1, true>(a.gamma, a.C, t, 1.0f, gamma);
  double sb[1][4] = {}, sg[1][4] = {};
  for (int id = blockIdx.x; id < u.tiles; id += gridDim.x) {
    const TileAt at = tile_at(u, id);
    quad_t x[K][1], dy[K][1], add[ADD ? K : 1][1];
    float mean[K], rstd[K];
#pragma unroll
    for (int k = 0; k < K; k++) {
      const int i = k * G + i0;
      const long long row = at.row0 + (i < at.rows ? i : 0);
      load_row<T, 1, true>(a.x + row * a.C, a.C, t, x[k]);
      load_row<T, 1, true>(a.dy + row * a.C, a.C, t, dy[k]);
      if constexpr (ADD) load_row<T, 1, true>(a.add + row * a.C, a.C, t, add[k]);
      mean[k] = a.mean_in[row];
      rstd[k] = a.rstd_in[row];
    }
#pragma unroll
    for (int k = 0; k < K; k++) {
      const int i = k * G + i0;
      quad_t g[1], xh[1];
      double s[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const bool in = has<T, true>(0, e, t, a.C), ours = in && i < at.rows;
        const float d = in ? dy[k][0][e] : 0.0f;
        xh[0][e] = in ? ln_hat(x[k][0][e], mean[k], rstd[k]) : 0.0f;
        g[0][e] = d * gamma[0][e];
        s[0] += in ? (double)g[0][e] : 0.0;
        s[1] += in ? (double)g[0][e] * (double)xh[0][e] : 0.0;
        sb[0][e] += ours ? (double)d : 0.0;
        sg[0][e] = ours ? __builtin_fma((double)d, (double)xh[0][e], sg[0][e]) : sg[0][e];
      }
      row_sums<T, 2>(s, 0);
      const float k1 = (float)(s[0] * a.inv), k2 = (float)(s[1] * a.inv);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        if constexpr (ADD) g[0][e] = ln_grad(g[0][e], xh[0][e], k1, k2, rstd[k], add[k][0][e]);
        else g[0][e] = ln_grad(g[0][e], xh[0][e], k1, k2, rstd[k]);
      }
      leave_row<T>(u, lds, i, t, g, a.C);
    }
    __syncthreads();
    quantize_tile<T>(u, at, lds);
  }
  if (!a.part) return;
  __syncthreads();  // (the last tile's codes are read)
  leave_columns<T, 1, kThreads>(a, reinterpret_cast<double2*>(&lds), t, sb, sg);
}

Tiles tiles_of(const LnArgs& a, int N, const MxOutView& out) {
  Tiles u{};
  u.g = mx_rows(out, a.R / N, N, a.C);
  u.fmt = out.fmt;
  u.across = ceil_div(N, 32);
  u.tiles = u.g.npt * u.across;
  return u;
}
template <class F>
hipError_t with_threads(int C, F&& f) {
  if (C <= 64) return f(std::integral_constant<int, 16>{});
  if (C <= 128) return f(std::integral_constant<int, 32>{});
  return f(std::integral_constant<int, 64>{});
}

}  // namespace

bool layer_norm_mx_one_pass(int C) { return C > 32 && C <= 256 && C % 4 == 0; }

hipError_t launch_layer_norm_mx(const LnArgs& a, int N, const MxOutView& out, hipStream_t st) {
  const Tiles u = tiles_of(a, N, out);
  return with_threads(a.C, [&](auto t) {
    constexpr int T = decltype(t)::value;
    const auto kern = a.add ? ln_mx_kernel<T, true> : ln_mx_kernel<T, false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)std::min(u.tiles, 2048)), dim3(kThreads), 0, st, a, u);
    return launch_check();
  });
}

hipError_t launch_layer_norm_grad_mx(LnArgs& a, int N, const MxOutView& out, hipStream_t st) {
  const Tiles u = tiles_of(a, N, out);
  a.parts = std::min(u.tiles, a.parts);
  return with_threads(a.C, [&](auto t) {
    constexpr int T = decltype(t)::value;
    const auto kern = a.add ? ln_grad_mx_kernel<T, true> : ln_grad_mx_kernel<T, false>;
    hipLaunchKernelGGL(kern, dim3((unsigned)a.parts), dim3(kThreads), 0, st, a, u);
    return launch_check();
  });
}

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
