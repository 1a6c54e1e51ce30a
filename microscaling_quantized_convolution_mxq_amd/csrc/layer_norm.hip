// layer_norm.hip -- layer normalization over the channels of every pixel's
// sample, and its gradient.
//
// A row is the C channels of one pixel and sample, contiguous in memory:
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   y = gamma (x - mean) rstd + beta
//   g = gamma dy,  xh = (x - mean) rstd,  dx = rstd (g - k1 - xh k2)
//   with k1 = sum g / C, k2 = sum g xh / C over the row;
//   dgamma = sum dy xh, dbeta = sum dy over the rows.
// All of it is bound by memory: 10 to 20 operations for each value of 8 to 16
// bytes. T threads hold a row in registers (four neighbouring channels a load),
// so every tensor is read once and the squares are summed around the mean
// itself. Groups of T threads walk over the rows with the next row's loads
// under way. Sums are fp64, in an order that depends on C alone, so the fp32
// and the MX form of one call have the same statistics to the bit.
// dgamma and dbeta stay in a thread's registers over all of its rows, as its
// columns never change; a workgroup leaves one row of sums, and a second
// kernel adds those of all workgroups in a fixed order.
// The gradient of 512 x 16 x 4096: 78 us for 403 MB (5.1 TB/s, a copy's rate); 7 x 9
// x 3 x 45 with a residual: 3.3 us, latency.
// Rows of more channels than a workgroup's registers hold are read once for
// every sum, from the caches after the first time (one row a workgroup); their
// gradient's column sums are a pass of its own over dy and x.
#include <algorithm>

#include "layer_norm_rows.h"
#include "mx_rows.h"
#include "norm.h"

namespace mq {

namespace {

// Most channels of a row held in registers: forward, 512 threads of 16 values;
// backward, which holds two tensors and the columns' sums (32 registers of eight
// values), 512 of 8. Whole calls with rows held and with rows read again: forward of
// 256 x 16 x 8192 50.7 and 105.6 us; gradient of 512 x 16 x 4096 78.7 and 269, of
// 512 x 16 x 2048 43.3 and 170. Above these: forward of 512 x 16 x 12288 330 us
// (805 MB), gradient of 256 x 16 x 8192 239 (403 MB).
constexpr int kWide = 8192;
constexpr int kWideGrad = 4096;
// Most workgroups of the gradient's pass, each of which leaves a row of column
// sums: two a compute unit, one for rows of more than 1024 channels, whose
// workgroups have more threads and more loads under way. Each more costs its row.
// Whole calls: 512 x 16 x 4096 with 128, 256, 512 and 1024 workgroups 99.7, 79.0,
// 83.8 and 93.3 us; with 256, 512 and 1024, 512 x 16 x 1024 32.5, 26.7 and 28.8,
// 20 x 20 x 128 x 256 with a skip path 54.9, 43.8 and 48.5, to E5M2 63.0, 44.4 and 46.7.
constexpr int kParts = 512, kPartsWide = 256;

template <int T>
constexpr int threads_of() {
  return T < 256 ? 256 : T;
}

// ---- forward ------------------------------------------------------------------------------------
// ADD: a residual is added first (and the sum stored).
template <int T, int Q, bool FULL, bool ADD>
__global__ __launch_bounds__(threads_of<T>()) void ln_kernel(const LnArgs a) {
  constexpr int G = threads_of<T>() / T;
  const int t = threadIdx.x % T;
  const int step = gridDim.x * G;
  int r = blockIdx.x * G + threadIdx.x / T;
  if (r >= a.R) return;  // whole groups; a workgroup of one group always has a row
  quad_t gamma[Q], beta[Q], next[Q], more[Q];
  load_row<T, Q, FULL>(a.x + (long long)r * a.C, a.C, t, next);
  if (ADD) load_row<T, Q, FULL>(a.add + (long long)r * a.C, a.C, t, more);
  if (T <= 64) {
    load_param<T, Q, FULL>(a.gamma, a.C, t, 1.0f, gamma);
    load_param<T, Q, FULL>(a.beta, a.C, t, 0.0f, beta);
  }
  while (true) {
    const long long at = (long long)r * a.C;
    const int rn = r + step < a.R ? r + step : r;
    quad_t v[Q];
    double s[1] = {0};
#pragma unroll
    for (int q = 0; q < Q; q++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[q][i] = ADD ? next[q][i] + more[q][i] : next[q][i];
        s[0] += has<T, FULL>(q, i, t, a.C) ? (double)v[q][i] : 0.0;
      }
    if (ADD) store_row<T, Q, FULL>(a.sum + at, a.C, t, v);
    if (rn != r) {
      load_row<T, Q, FULL>(a.x + (long long)rn * a.C, a.C, t, next);
      if (ADD) load_row<T, Q, FULL>(a.add + (long long)rn * a.C, a.C, t, more);
    }
    row_sums<T, 1>(s, 0);
    const double mean = s[0] * a.inv;
    s[0] = 0;
#pragma unroll
    for (int q = 0; q < Q; q++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const double d = has<T, FULL>(q, i, t, a.C) ? (double)v[q][i] - mean : 0.0;
        s[0] = __builtin_fma(d, d, s[0]);
      }
    row_sums<T, 1>(s, 1);
    const float m = (float)mean, rs = rstd_of(s[0], a);
    if (t == 0) {
      if (a.mean) a.mean[r] = m;
      if (a.rstd) a.rstd[r] = rs;
    }
    if (a.out) {
      if (T > 64) {  // (kept over the rows they would cost a wide row's threads 32 registers)
        load_param<T, Q, FULL>(a.gamma, a.C, t, 1.0f, gamma);
        load_param<T, Q, FULL>(a.beta, a.C, t, 0.0f, beta);
      }
#pragma unroll
      for (int q = 0; q < Q; q++)
#pragma unroll
        for (int i = 0; i < 4; i++) v[q][i] = ln_value(v[q][i], m, rs, gamma[q][i], beta[q][i]);
      store_row<T, Q, FULL>(a.out + at, a.C, t, v);
    }
    if (rn == r) break;
    r = rn;
  }
}

// Rows too long for registers: a workgroup reads its row three times.
template <bool ADD>
__global__ __launch_bounds__(1024) void ln_long_kernel(const LnArgs a) {
  for (int r = blockIdx.x; r < a.R; r += gridDim.x) {
    const long long at = (long long)r * a.C;
    const float* x = a.x + at;
    double s[1] = {0};
    for (int c = threadIdx.x; c < a.C; c += 1024) {
      const float v = ADD ? x[c] + a.add[at + c] : x[c];
      if (ADD) a.sum[at + c] = v;
      s[0] += v;
    }
    row_sums<1024, 1>(s, 0);
    const double mean = s[0] * a.inv;
    const float* from = ADD ? a.sum + at : x;  // (a thread reads back what it wrote itself)
    s[0] = 0;
    for (int c = threadIdx.x; c < a.C; c += 1024) {
      const double d = (double)from[c] - mean;
      s[0] = __builtin_fma(d, d, s[0]);
    }
    row_sums<1024, 1>(s, 1);
    const float m = (float)mean, rs = rstd_of(s[0], a);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = m;
      if (a.rstd) a.rstd[r] = rs;
    }
    if (a.out)
      for (int c = threadIdx.x; c < a.C; c += 1024)
        a.out[at + c] = ln_value(from[c], m, rs, a.gamma ? a.gamma[c] : 1.0f, a.beta ? a.beta[c] : 0.0f);
  }
}

// ---- backward -----------------------------------------------------------------------------------
template <int T, int Q, bool FULL, bool ADD>
__global__ __launch_bounds__(threads_of<T>()) void ln_grad_kernel(const LnArgs a) {
  constexpr int B = threads_of<T>(), G = B / T;
  const int t = threadIdx.x % T;
  const int step = gridDim.x * G;
  int r = blockIdx.x * G + threadIdx.x / T;
  quad_t gamma[Q], x[Q], dy[Q], add[Q];
  float mean = 0, rstd = 0;
  double sb[Q][4], sg[Q][4];  // this thread's columns: sums of dy and dy xh
#pragma unroll
  for (int q = 0; q < Q; q++)
#pragma unroll
    for (int i = 0; i < 4; i++) sb[q][i] = sg[q][i] = 0;
  auto load = [&](int row) {
    const long long at = (long long)row * a.C;
    load_row<T, Q, FULL>(a.x + at, a.C, t, x);
    load_row<T, Q, FULL>(a.dy + at, a.C, t, dy);
    if (ADD) load_row<T, Q, FULL>(a.add + at, a.C, t, add);
    mean = a.mean_in[row];
    rstd = a.rstd_in[row];
  };
  if (r < a.R) load(r);
  load_param<T, Q, FULL>(a.gamma, a.C, t, 1.0f, gamma);
  for (int phase = 0; r < a.R; r += step, phase ^= 1) {
    const long long at = (long long)r * a.C;
    quad_t xh[Q], g[Q], sk[Q];
    const float rs = rstd;
    double s[2] = {0, 0};
#pragma unroll
    for (int q = 0; q < Q; q++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const bool in = has<T, FULL>(q, i, t, a.C);
        const float d = in ? dy[q][i] : 0.0f;
        xh[q][i] = in ? ln_hat(x[q][i], mean, rs) : 0.0f;
        g[q][i] = d * gamma[q][i];
        if (ADD) sk[q][i] = add[q][i];
        s[0] += in ? (double)g[q][i] : 0.0;
        s[1] += in ? (double)g[q][i] * (double)xh[q][i] : 0.0;
        sb[q][i] += (double)d;
        sg[q][i] = __builtin_fma((double)d, (double)xh[q][i], sg[q][i]);
      }
    if (r + step < a.R) load(r + step);
    row_sums<T, 2>(s, phase);
    const float k1 = (float)(s[0] * a.inv), k2 = (float)(s[1] * a.inv);
    if (a.out) {
#pragma unroll
      for (int q = 0; q < Q; q++)
#pragma unroll
        for (int i = 0; i < 4; i++)
          g[q][i] = ADD ? ln_grad(g[q][i], xh[q][i], k1, k2, rs, sk[q][i]) : ln_grad(g[q][i], xh[q][i], k1, k2, rs);
      store_row<T, Q, FULL>(a.out + at, a.C, t, g);
    } else if (t == 0) {
      a.row[r] = LnRow{k1, k2};
    }
  }
  if (!a.part) return;
  if constexpr (T <= 64) {
    __shared__ double2 cols[(B / 64 - 1) * T * Q * 4];
    leave_columns<T, Q, B>(a, cols, t, sb, sg);
  } else {
    leave_columns<T, Q, B>(a, nullptr, t, sb, sg);
  }
}

template <bool ADD>
__global__ __launch_bounds__(1024) void ln_grad_long_kernel(const LnArgs a) {
  for (int r = blockIdx.x, phase = 0; r < a.R; r += gridDim.x, phase ^= 1) {
    const long long at = (long long)r * a.C;
    const float mean = a.mean_in[r], rs = a.rstd_in[r];
    double s[2] = {0, 0};
    for (int c = threadIdx.x; c < a.C; c += 1024) {
      const float g = a.gamma ? a.dy[at + c] * a.gamma[c] : a.dy[at + c];
      s[0] += g;
      s[1] += (double)g * (double)ln_hat(a.x[at + c], mean, rs);
    }
    row_sums<1024, 2>(s, phase);
    const float k1 = (float)(s[0] * a.inv), k2 = (float)(s[1] * a.inv);
    if (a.out) {
      for (int c = threadIdx.x; c < a.C; c += 1024) {
        const float g = a.gamma ? a.dy[at + c] * a.gamma[c] : a.dy[at + c];
        const float xh = ln_hat(a.x[at + c], mean, rs);
        a.out[at + c] = ADD ? ln_grad(g, xh, k1, k2, rs, a.add[at + c]) : ln_grad(g, xh, k1, k2, rs);
      }
    } else if (threadIdx.x == 0) {
      a.row[r] = LnRow{k1, k2};
    }
  }
}

// Column sums of long rows: a thread takes a column of the rows blockIdx.y, blockIdx.y + parts, ....
__global__ __launch_bounds__(256) void ln_long_columns_kernel(const LnArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.C) return;
  double sb = 0, sg = 0;
  for (int r = blockIdx.y; r < a.R; r += a.parts) {
    const double d = a.dy[(long long)r * a.C + c];
    sb += d;
    sg = __builtin_fma(d, (double)ln_hat(a.x[(long long)r * a.C + c], a.mean_in[r], a.rstd_in[r]), sg);
  }
  a.part[(long long)blockIdx.y * a.C + c] = make_float2((float)sb, (float)sg);
}

// dgamma and dbeta from the workgroups' rows of sums, eight channels a workgroup
__global__ __launch_bounds__(512) void ln_columns_kernel(const LnArgs a) {
  for (int c0 = blockIdx.x * 8; c0 < a.C; c0 += gridDim.x * 8) {
    if (c0 != (int)blockIdx.x * 8) __syncthreads();  // (the sums before are read)
    double s1, s2;
    sum_rows<8>(a.part, a.C, c0, 0, a.parts, s1, s2);
    const int c = c0 + (int)threadIdx.x;
    if (threadIdx.x < 8 && c < a.C) {
      if (a.dbeta) a.dbeta[c] = (float)s1;
      if (a.dgamma) a.dgamma[c] = (float)s2;
    }
  }
}

// f(threads of a row, quads of a thread): the fewest threads that hold a row in
// one quad each, up to a wave; then more quads, then more waves.
template <int T_, int Q_>
struct Tile {
  static constexpr int T = T_, Q = Q_;
};
template <bool GRAD, class F>
auto with_tile(int C, F&& f) {
  if (C <= 4) return f(Tile<1, 1>{});
  if (C <= 8) return f(Tile<2, 1>{});
  if (C <= 16) return f(Tile<4, 1>{});
  if (C <= 32) return f(Tile<8, 1>{});
  if (C <= 64) return f(Tile<16, 1>{});
  if (C <= 128) return f(Tile<32, 1>{});
  if (C <= 256) return f(Tile<64, 1>{});
  if (C <= 512) return f(Tile<64, 2>{});
  if constexpr (GRAD) {  // at most two quads: their column sums alone are 32 registers
    if (C <= 1024) return f(Tile<256, 1>{});
    return C <= 2048 ? f(Tile<256, 2>{}) : f(Tile<512, 2>{});
  } else {
    if (C <= 1024) return f(Tile<64, 4>{});
    if (C <= 2048) return f(Tile<256, 2>{});
    return C <= 4096 ? f(Tile<256, 4>{}) : f(Tile<512, 4>{});
  }
}
int rows_of_group(int C) {
  return with_tile<true>(C, [](auto t) { return threads_of<decltype(t)::T>() / decltype(t)::T; });
}

template <bool FULL, bool ADD>
hipError_t launch_forward_rows(const LnArgs& a, hipStream_t st) {
  return with_tile<false>(a.C, [&](auto tile) {
    constexpr int T = decltype(tile)::T, Q = decltype(tile)::Q, B = threads_of<T>();
    const auto kern = ln_kernel<T, Q, FULL, ADD>;
    static const int resident = resident_groups(reinterpret_cast<const void*>(kern), B);
    const int grid = std::min(ceil_div(a.R, B / T), resident);
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(B), 0, st, a);
    return launch_check();
  });
}
template <bool FULL, bool ADD>
hipError_t launch_backward_rows(const LnArgs& a, hipStream_t st) {
  return with_tile<true>(a.C, [&](auto tile) {
    constexpr int T = decltype(tile)::T, Q = decltype(tile)::Q, B = threads_of<T>();
    hipLaunchKernelGGL((ln_grad_kernel<T, Q, FULL, ADD>), dim3((unsigned)a.parts), dim3(B), 0, st, a);
    return launch_check();
  });
}

}  // namespace

// Workgroups of the gradient's pass over the rows, each of which leaves a row
// of column sums.
static int grad_parts(int R, int C) {
  if (C > kWideGrad) return std::min(R, 64);
  return std::min(ceil_div(R, rows_of_group(C)), C > 1024 ? kPartsWide : kParts);
}

size_t layer_norm_workspace_bytes(const LnShape& s, int op) {
  const long long R = (long long)s.P * s.N;
  const size_t rows = ((size_t)R * 8 + 15) / 16 * 16;  // the rows' parameters, for MX results
  return op == 0 ? rows : rows + (size_t)grad_parts((int)R, s.C) * s.C * sizeof(float2);
}

hipError_t launch_layer_norm_rows(const LnArgs& a, hipStream_t st) {
  if (a.C > kWide) {
    const dim3 grid((unsigned)std::min(a.R, 2048));
    if (a.add) hipLaunchKernelGGL(ln_long_kernel<true>, grid, dim3(1024), 0, st, a);
    else hipLaunchKernelGGL(ln_long_kernel<false>, grid, dim3(1024), 0, st, a);
    return launch_check();
  }
  const bool full = a.C % 4 == 0;
  if (a.add) return full ? launch_forward_rows<true, true>(a, st) : launch_forward_rows<false, true>(a, st);
  return full ? launch_forward_rows<true, false>(a, st) : launch_forward_rows<false, false>(a, st);
}

hipError_t launch_layer_norm_grad_rows(const LnArgs& a, hipStream_t st) {
  if (a.C > kWideGrad) {
    if (a.part) {  // first: dx may take the place of x or dy
      hipLaunchKernelGGL(ln_long_columns_kernel, dim3((unsigned)ceil_div(a.C, 256), (unsigned)a.parts), dim3(256), 0, st, a);
      const hipError_t e = launch_check();
      if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)std::min(a.R, 2048));
    if (a.add) hipLaunchKernelGGL(ln_grad_long_kernel<true>, grid, dim3(1024), 0, st, a);
    else hipLaunchKernelGGL(ln_grad_long_kernel<false>, grid, dim3(1024), 0, st, a);
    return launch_check();
  }
  const bool full = a.C % 4 == 0;
  if (a.add) return full ? launch_backward_rows<true, true>(a, st) : launch_backward_rows<false, true>(a, st);
  return full ? launch_backward_rows<true, false>(a, st) : launch_backward_rows<false, false>(a, st);
}

hipError_t launch_layer_norm_columns(const LnArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(ln_columns_kernel, dim3((unsigned)std::min(ceil_div(a.C, 8), 1 << 16)), dim3(512), 0, st, a);
  return launch_check();
}

hipError_t launch_layer_norm(const LnShape& s, const float* x, const float* residual, const float* gamma,
                             const float* beta, float* sum, float* y, const MxOutView& yq, float* mean, float* rstd,
                             void* ws, hipStream_t st) {
  LnArgs a{};
  a.x = x; a.add = residual; a.gamma = gamma; a.beta = beta;
  a.sum = sum; a.out = y; a.mean = mean; a.rstd = rstd;
  a.R = s.P * s.N; a.C = s.C; a.eps = s.eps; a.inv = 1.0 / s.C;
  if (!yq.codes) return launch_layer_norm_rows(a, st);
  if (layer_norm_mx_one_pass(s.C)) return launch_layer_norm_mx(a, s.N, yq, st);
  // the second pass reads the statistics that the first one leaves
  float* const kept = static_cast<float*>(ws);
  if (!a.mean) a.mean = kept;
  if (!a.rstd) a.rstd = kept + a.R;
  hipError_t e = launch_layer_norm_rows(a, st);
  if (e != hipSuccess) return e;
  a.mean_in = a.mean; a.rstd_in = a.rstd;
  if (residual) { a.x = sum; a.add = nullptr; }
  return launch_layer_norm_mx_rows(a, s.N, yq, st);
}

hipError_t launch_layer_norm_backward(const LnShape& s, const float* dy, const float* x, const float* gamma,
                                      const float* mean, const float* rstd, const float* dskip, float* dx,
                                      const MxOutView& dxq, float* dgamma, float* dbeta, void* ws, hipStream_t st) {
  LnArgs a{};
  a.x = x; a.dy = dy; a.add = dskip; a.gamma = gamma;
  a.mean_in = mean; a.rstd_in = rstd; a.out = dx; a.dgamma = dgamma; a.dbeta = dbeta;
  a.R = s.P * s.N; a.C = s.C; a.eps = s.eps; a.inv = 1.0 / s.C;
  a.parts = grad_parts(a.R, a.C);
  a.row = static_cast<LnRow*>(ws);
  if (dgamma || dbeta)
    a.part = reinterpret_cast<float2*>(static_cast<char*>(ws) + ((size_t)a.R * 8 + 15) / 16 * 16);
  hipError_t e;
  if (dxq.codes && layer_norm_mx_one_pass(s.C)) {
    e = launch_layer_norm_grad_mx(a, s.N, dxq, st);
    if (e == hipSuccess && a.part) e = launch_layer_norm_columns(a, st);
    return e;
  }
  e = launch_layer_norm_grad_rows(a, st);
  if (e == hipSuccess && dxq.codes) e = launch_layer_norm_grad_mx_rows(a, s.N, dxq, st);
  if (e == hipSuccess && a.part) e = launch_layer_norm_columns(a, st);
  return e;
}

}  // namespace mq
