// norm.hip -- group normalization with an activation, channels last, and its
// gradient: statistics, sums, and the elementwise passes with fp32 output.
//
// All of it is memory bound (10-30 operations for each value of 4 to 12
// bytes). A pixel's row holds every sample and channel side by side, so a
// thread takes an octet of neighbouring channels of one sample and walks over
// the pixels: loads are whole lines, and what belongs to its columns stays in
// registers.
//   One pass: where a slab of whole groups over all pixels fits the registers
//     of a workgroup, that workgroup reads it once, joins the statistics in
//     LDS and writes the result from its registers: one launch, no workspace.
//   Streaming: partial statistics (a mean and the mean square around it) or
//     sums of chunks of pixels, and an elementwise pass that reads x (and dy)
//     again. The fp32 pass joins the chunks of its own columns' groups first,
//     in a fixed order (narrow tiles have few chunks, so that is one round of
//     loads); for MX results, whose tiles span 32 samples, and for groups of
//     very many columns a kernel in between joins them once.
// Sums of values, and of the gradient's terms, are fp64 (two operations a
// value, hidden behind the loads), so a mean is its fp32 rounding, whatever
// cancels in it, and no sum loses digits with its length. Squares are summed in
// fp32 around the mean of the few values that a thread has at one time, and
// joined in fp64 around one of those means, so a mean far from zero costs no
// digits. Partial results are kept in fp32.
#include <algorithm>

#include "norm.h"

namespace mq {

namespace {

constexpr int kOneR = 8;         // most pixels a thread of the one-pass kernels holds
// Values that a thread of the streaming kernels has in flight: two pixels of
// one tensor or one pixel of two, beside as many being computed. Few registers
// and many waves read faster than many loads a wave (two, four and eight
// pixels: 160 x 160 x 32 x 128 236, 239, 244 us; gradient of 80 x 80 x 16 x 64
// 31.2, 32.5, 40.7 us).
constexpr int kBatch = 2;
constexpr int kStreamGroups = 512;  // workgroups of the streaming kernels, about
constexpr int kMinPixels = 4;       // pixels of a thread, before there are fewer workgroups

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

}  // namespace

NormGeo norm_geo(const NormShape& s, bool backward) {
  NormGeo g{};
  g.P = s.P; g.N = s.N; g.C = s.C; g.G = s.G;
  g.D = s.C / s.G;
  g.NO = ceil_div(s.C, 8);
  g.TO = s.N * g.NO;
  g.UW = backward ? 1 : gcd(g.D, 8);  // the backward sums columns (dgamma, dbeta)
  g.e = g.D / g.UW;
  g.de = make_fastdiv((unsigned)g.e);
  g.dNO = make_fastdiv((unsigned)g.NO);
  g.dD = make_fastdiv((unsigned)g.D);

  // a slab is a run of octets that ends where a group does: multiples of
  // lcm(D, 8) channels where they divide C, else whole samples
  const long long L = (long long)g.D / gcd(g.D, 8) * 8;
  const bool within = s.C % L == 0;
  const int unit = within ? (int)(L / 8) : g.NO;
  const int tmax = backward || g.UW == 1 ? 512 : 1024;
  // The backward holds two tensors, too few workgroups of them: up to 2^22
  // values, where a launch less counts (20 x 20 x 16 x 256: 16.7 against 17.4
  // us streaming; with 128 samples 52 against 58 us with fp32 results, but 66
  // against 57 us with MX results, whose sums must be the same ones)
  const bool small = !backward || (long long)s.P * s.N * s.C <= 1 << 22;
  if (unit <= tmax && small) {
    // at least a cache line's 32 channels, and enough octets that a
    // workgroup of few pixels has 256 threads
    long long so = unit * (long long)ceil_div(4, unit);
    so = std::max(so, unit * (long long)ceil_div(256, (long long)std::min(s.P, 256) * unit));
    so = std::min(so, (long long)tmax / unit * unit);
    so = std::min(so, (long long)ceil_div(g.TO, unit) * unit);
    // few slabs take more threads of fewer pixels, many the smallest
    // workgroups that hold them (backward, 1,024 slabs of 400 pixels: 256
    // threads 66, 512 threads 80 us)
    int t = backward && ceil_div(g.TO, so) >= 256 ? 256 : 512;
    for (; t <= tmax && !g.one; t *= 2) {
      if (so > t) continue;
      const int ty = std::min(s.P, t / (int)so);
      // (1,024 threads have 128 registers each, room for half as many pixels)
      if (ceil_div(s.P, ty) > (t > 512 ? kOneR / 2 : kOneR)) continue;
      // a small tensor's few slabs need workgroups more than whole lines
      // (124 x 4 x 32 x 8, gradient of GELU: 15 us with four octets, 11 with one)
      if (ceil_div(g.TO, so) < 64) so = unit;
      g.one = true;
      g.so = (int)so;
      g.ty1 = std::min(s.P, t / (int)so);
      g.T1 = ceil_div((long long)so * g.ty1, 64) * 64;
      g.nslab = ceil_div(g.TO, so);
      g.nseg = within ? (int)(so * 8 / g.D) : (int)(so / g.NO) * g.G;
    }
  }

  // streaming tiles: 16 octets (512 bytes of a pixel's row) wide, 8 where a
  // row has few: the narrower, the fewer chunks there are of a column, which
  // the elementwise pass joins; below 512 bytes large tensors read more slowly
  // (160 x 160 x 32 x 128, both passes: 32 octets 246, 16 233, 8 271, 4 303
  // us); of such widths the one that leaves the fewest of 256 threads idle
  double best = 0;
  const int n0 = ceil_div(g.TO, g.TO >= 256 ? 16 : 8);
  for (int nt = n0; nt < n0 + 4; nt++) {
    const int tx = ceil_div(g.TO, nt), ty = 256 / tx;
    const double use = (double)g.TO / nt * ty / 256;
    if (use > best * 1.02) {
      best = use;
      g.ntile = nt; g.tx = tx; g.ty = std::min(ty, s.P);
    }
  }
  // up to 512 workgroups (two per compute unit) of at least four pixels a
  // thread (MX gradient of 20 x 20 x 128 x 256: 52.4 us, 55.5 with 1,024)
  g.ngroup = ceil_div(s.P, g.ty);
  g.nchunk = std::max(1, std::min(kStreamGroups / std::min(kStreamGroups, g.ntile), std::max(ceil_div(g.ngroup, kMinPixels), std::min(g.ngroup, 256 / std::min(256, g.ntile)))));
  // and no more chunks than a workgroup of the elementwise pass joins at once
  g.nchunk = std::min(g.nchunk, 256 / g.tx);
  // eight loads a lane
  const long long entries = (long long)g.e * g.nchunk;
  g.wide = entries > 2048;
  g.lanes = 1;
  while (g.lanes < 64 && g.lanes * 8 < entries) g.lanes *= 2;
  return g;
}

namespace {

// ---------------------------------------------------------------------------
// shared pieces
// ---------------------------------------------------------------------------
// Workgroups go to the eight XCDs in turn; this order gives each XCD a
// contiguous range of the n pieces of work. Neighbouring slabs share DRAM
// pages, and slabs eight apart would use an eighth of an XCD's L2 channels.
__device__ __forceinline__ int xcd_order(int b, int n) {
  const int x = b & 7, i = b >> 3, q = n >> 3, r = n & 7;
  return x * q + min(x, r) + i;
}

// a thread's octet
struct Oct {
  int n, c0, cnt;
  long long col;  // n * C + c0
};
__device__ __forceinline__ Oct octet(const NormGeo& g, int o, bool active) {
  Oct t;
  t.n = (int)fdiv((unsigned)(active ? o : 0), g.dNO);
  t.c0 = ((active ? o : 0) - t.n * g.NO) * 8;
  t.cnt = active ? min(8, g.C - t.c0) : 0;
  t.col = (long long)t.n * g.C + t.c0;
  return t;
}

// cnt values at p + c0, or `none` where there is no p
template <bool FULL>
__device__ __forceinline__ void load_optional(const float* p, int c0, int cnt, float none, float (&v)[8]) {
  if (p) {
    load_run<8, FULL>(p + c0, cnt, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = i < cnt ? none : 0.0f;
  }
}

// gamma (1 where there is none) and beta of an octet
template <bool FULL>
__device__ __forceinline__ void affine(const NormArgs& a, const Oct& t, float (&ga)[8], float (&be)[8]) {
  load_optional<FULL>(a.beta, t.c0, t.cnt, 0.0f, be);
  load_optional<FULL>(a.gamma, t.c0, t.cnt, 1.0f, ga);
}

// Statistics of some values: their mean m + lo (m is its fp32 rounding) and the
// mean q of squared deviations from m (a mean, which stays in fp32's range
// however many values there are).
using Part = NormPart;
// Sums of c values' deviations from a reference p, and of the squares of
// these, in fp64. p is a mean of some of the values, so what is summed is as
// small as their spread whatever their mean is, and nothing cancels in
// sq - s^2 / c; no step multiplies by 0 or divides.
struct Sums {
  float p = 0;
  double s = 0, sq = 0;
  // n values of sum `sum`, rounded mean m and squared deviations q from m
  __device__ void add(double sum, float m, float q, double n) {
    const double e = (double)m - p, t = __builtin_fma(-n, (double)p, sum);
    s += t;
    sq += __builtin_fma(e, __builtin_fma(-n, e, 2.0 * t), (double)q);
  }
  __device__ void add(const Part& a, double n) {
    const double d = (double)a.m - p;
    s += n * (d + a.lo);
    sq += n * ((double)a.q + d * (d + 2.0 * a.lo));
  }
  __device__ Part part(double n) const {
    const double inv = 1.0 / n, d = s * inv, mean = p + d;
    const float m = (float)mean;
    const double e = (double)m - p;
    return Part{m, (float)(mean - m), (float)(sq * inv - e * (2.0 * d - e))};
  }
};

// sum, mean (rounded) and sum of squared deviations of the UW values of every
// unit of an octet over the first `rows` of R rows
template <int R, int UW>
__device__ __forceinline__ void unit_stats(const float (&v)[R][8], int rows, double (&sum)[8 / UW],
                                           float (&mean)[8 / UW], float (&m2)[8 / UW]) {
  // fp64: the sum of finite values may pass fp32's range, their mean does not
  // (1 / n by one Newton step from fp32's, so that the mean of equal values is
  // that value)
  const double n = (double)(rows * UW), r = (double)(1.0f / (float)(rows * UW));
  const double inv = r * __builtin_fma(-n, r, 2.0);
#pragma unroll
  for (int u = 0; u < 8 / UW; u++) {
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < R; k++)
#pragma unroll
      for (int i = 0; i < UW; i++) s += k < rows ? (double)v[k][u * UW + i] : 0.0;
    sum[u] = s;
    const float m = (float)(s * inv);
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < R; k++)
#pragma unroll
      for (int i = 0; i < UW; i++) {
        const float d = v[k][u * UW + i] - m;
        q += k < rows ? d * d : 0.0f;
      }
    mean[u] = m;
    m2[u] = q;
  }
}

// mean and rstd of M values
__device__ __forceinline__ float2 finish_stats(const Sums& t, double M, float eps) {
  const double d = t.s / M;
  double var = t.sq / M - d * d;
  if (var < 0.0) var = 0.0;
  return make_float2((float)(t.p + d), (float)(1.0 / sqrt(var + (double)eps)));
}

__device__ __forceinline__ double group_sum(double v, int lanes) {  // aligned groups of lanes (a power of two)
  for (int o = 1; o < lanes; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// Sums of columns 0 .. W - 1 over rows 0 .. n - 1 by T threads: get(row,
// column, s1, s2) adds a row's values, done(column, s1, s2) takes the sums.
// Thread t adds rows t / W, t / W + T / W, ... of column t % W; then a tree
// over x1, x2 [T]. W is at most T.
template <class Get, class Done>
__device__ __forceinline__ void reduce_rows(int T, int W, int n, double* x1, double* x2, Get get, Done done) {
  const int t = (int)threadIdx.x, r = t / W, u = t - r * W, R = T / W;
  double s1 = 0, s2 = 0;
  if (r < R)
    for (int row = r; row < n; row += R) get(row, u, s1, s2);
  x1[t] = s1;
  x2[t] = s2;
  int have = min(R, n), h = 1;
  while (h < have) h <<= 1;
  for (h >>= 1; h > 0; h >>= 1) {
    __syncthreads();
    if (r < h && r + h < have) {
      x1[t] += x1[t + h * W];
      x2[t] += x2[t + h * W];
    }
    have = min(have, h);
  }
  if (t < W) done(u, x1[t], x2[t]);
}

// lanes that reduce one segment together: a power of two up to 64
__device__ __forceinline__ int seg_lanes(int threads, int nseg) {
  int t = 1;
  while (t < 64 && 2 * t * nseg <= threads) t <<= 1;
  return t;
}

// ---------------------------------------------------------------------------
// forward, one pass
// ---------------------------------------------------------------------------
// A slab of whole groups over all pixels, R pixels of an octet a thread in
// registers. Bound by latency (one round of loads, two barriers, one of
// stores): 16 x 16 x 2 x 32 in 8 groups takes 6.1 us.
template <int R, int UW, bool FULL, int ACT>
__global__ __launch_bounds__(UW == 1 || R == kOneR ? 512 : 1024) void norm_one_kernel(const NormArgs a) {
  constexpr int UN = 8 / UW;
  extern __shared__ float2 sh[];
  const NormGeo& g = a.g;
  const int W = g.so * UN;           // units of the slab
  float2* const sseg = sh;           // [nseg]
  Part* const su = reinterpret_cast<Part*>(sh + g.nseg);  // [ty1][W]
  const int ox = (int)threadIdx.x % g.so, py = (int)threadIdx.x / g.so;
  const int o0 = xcd_order((int)blockIdx.x, (int)gridDim.x) * g.so;
  const bool active = py < g.ty1 && o0 + ox < g.TO;
  const Oct t = octet(g, o0 + ox, active);
  const long long stride = (long long)g.N * g.C;
  const int rows = active ? (g.P - py + g.ty1 - 1) / g.ty1 : 0;  // pixels py, py + ty1, ...
  float v[R][8];
#pragma unroll
  for (int k = 0; k < R; k++)
    load_run<8, FULL>(a.x + (k < rows ? py + k * g.ty1 : 0) * stride + t.col, k < rows ? t.cnt : 0, v[k]);
  if (active) {
    double sum[UN];
    float mean[UN], m2[UN];
    unit_stats<R, UW>(v, rows, sum, mean, m2);
#pragma unroll
    for (int u = 0; u < UN; u++) {
      Sums one;
      one.p = mean[u];
      one.add(sum[u], mean[u], m2[u], (double)(rows * UW));
      su[py * W + ox * UN + u] = one.part((double)(rows * UW));
    }
  }
  __syncthreads();
  // segments (sample, group) of the slab: e units each, over ty1 rows
  const int n0 = (int)fdiv((unsigned)o0, g.dNO);
  const int S0 = n0 * g.G + (o0 - n0 * g.NO) * 8 / g.D;
  {
    const int lanes = seg_lanes((int)blockDim.x, g.nseg);
    const int j = (int)threadIdx.x & (lanes - 1);
    const double M = (double)g.P * g.D;
    for (int s = (int)threadIdx.x / lanes; s < g.nseg && S0 + s < g.N * g.G; s += (int)blockDim.x / lanes) {
      const int S = S0 + s, n = S / g.G, gr = S - n * g.G;
      const int pos = (n * g.NO - o0) * UN + gr * g.e;
      Sums sum;
      sum.p = su[pos].m;
      for (int i = j; i < g.ty1 * g.e; i += lanes) {
        const int row = i / g.e;
        sum.add(su[row * W + pos + (i - row * g.e)], (double)(((g.P - row + g.ty1 - 1) / g.ty1) * UW));
      }
      sum.s = group_sum(sum.s, lanes);
      sum.sq = group_sum(sum.sq, lanes);
      if (j == 0) {
        const float2 st = finish_stats(sum, M, a.eps);
        sseg[s] = st;
        if (a.mean) a.mean[S] = st.x;
        if (a.rstd) a.rstd[S] = st.y;
      }
    }
  }
  __syncthreads();
  if (!active) return;
  float mean[8], ga[8], be[8];
  affine<FULL>(a, t, ga, be);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int s = t.n * g.G + (int)fdiv((unsigned)(t.c0 + (i < t.cnt ? i : 0)), g.dD) - S0;
    const float2 st = sseg[s];
    mean[i] = i < t.cnt ? st.x : 0.0f;
    ga[i] = i < t.cnt ? st.y * ga[i] : 0.0f;
  }
  if (a.out) {
    const DropKey key = drop_key(a.drop);
#pragma unroll
    for (int k = 0; k < R; k++)
      if (k < rows) {
        const int p = py + k * g.ty1;
        float u[8];
        norm_values<8>(mean, ga, be, v[k], u);
        act_values<ACT, 8>(u);
        drop_values<8>(a.drop, key, (uint32_t)p * g.N + t.n, t.c0, u);
        store_run<8, FULL>(a.out + p * stride + t.col, t.cnt, u);
      }
  } else if (py == 0) {
    store_run<8, FULL>(a.col.mean + t.col, t.cnt, mean);
    store_run<8, FULL>(a.col.a + t.col, t.cnt, ga);
  }
}

// ---------------------------------------------------------------------------
// forward, streaming
// ---------------------------------------------------------------------------
// Partial statistics: one read of x. A thread carries batches of pixels of its
// octet in fp64 sums, then a tree in LDS joins the threads of a column, so a
// chunk leaves one entry a unit. Bound by reading x: 160 x 160 x 32 x 128 92 us
// (4.6 TB/s; vector instructions issue in 43% of the busy cycles);
// 80 x 80 x 16 x 64 8.3 us, mostly the first loads' latency.
template <int UW, bool FULL>
__global__ __launch_bounds__(256) void norm_stats_kernel(const NormArgs a) {
  constexpr int UN = 8 / UW;
  __shared__ Part su[256 * UN];
  const NormGeo& g = a.g;
  const int chunk = (int)blockIdx.x / g.ntile, tile = (int)blockIdx.x - chunk * g.ntile;
  const int ox = (int)threadIdx.x % g.tx, py = (int)threadIdx.x / g.tx;
  const int o = tile * g.tx + ox;
  const bool active = py < g.ty && o < g.TO;
  const Oct t = octet(g, o, active);
  const long long stride = (long long)g.N * g.C;
  const int p0 = chunk * g.ty + py, dp = g.nchunk * g.ty;  // pixels p0, p0 + dp, ...
  Sums sum[UN];
  double have = 0;
  if (active) {
    const float* src = a.x + t.col;
    // (the next pixels are requested before the current ones are summed)
    float next[kBatch][8];
    auto load = [&](int p) {
#pragma unroll
      for (int k = 0; k < kBatch; k++) {
        const int q = p + k * dp;
        load_run<8, FULL>(src + (q < g.P ? q : 0) * stride, q < g.P ? t.cnt : 0, next[k]);
      }
    };
    load(p0);
    for (int p = p0; p < g.P; p += kBatch * dp) {
      const int rows = min(kBatch, (g.P - p + dp - 1) / dp);
      float v[kBatch][8], bm[UN], bq[UN];
      double bs[UN];
#pragma unroll
      for (int k = 0; k < kBatch; k++)
#pragma unroll
        for (int i = 0; i < 8; i++) v[k][i] = next[k][i];
      load(p + kBatch * dp);
      unit_stats<kBatch, UW>(v, rows, bs, bm, bq);
      const double n = (double)(rows * UW);
#pragma unroll
      for (int u = 0; u < UN; u++) {
        if (p == p0) sum[u].p = bm[u];
        sum[u].add(bs[u], bm[u], bq[u], n);
      }
      have += n;
    }
  }
  const int W = g.tx * UN;
  if (py < g.ty)
#pragma unroll
    for (int u = 0; u < UN; u++) su[py * W + ox * UN + u] = sum[u].part(have);
  __syncthreads();
  // units of the tile, joined over the rows of pixels
  const int NU = g.N * g.C / UW;
  const double c = (double)chunk_pixels(g, chunk) * UW;
  // pixels of row r of the chunk: a group less where the last group is short
  const int groups = (g.ngroup - chunk + g.nchunk - 1) / g.nchunk, last = g.ngroup - 1;
  const bool owns_last = last % g.nchunk == chunk;
  __shared__ double x1[256], x2[256];
  reduce_rows(
      256, W, g.ty, x1, x2,
      [&](int r, int i, double& s1, double& s2) {
        const int rows = groups - (owns_last && last * g.ty + r >= g.P ? 1 : 0);
        if (rows == 0) return;
        Sums q;
        q.p = su[i].m;  // (row 0 has pixels in every chunk)
        q.add(su[r * W + i], (double)rows * UW);
        s1 += q.s;
        s2 += q.sq;
      },
      [&](int i, double s1, double s2) {
        const int oo = tile * g.tx + i / UN, u = i % UN;
        if (oo >= g.TO) return;
        const Oct q = octet(g, oo, true);
        if (u * UW >= q.cnt) return;
        Sums all;
        all.p = su[i].m;
        all.s = s1;
        all.sq = s2;
        a.part[(long long)chunk * NU + (q.col / UW + u)] = all.part(c);
      });
}

// ---------------------------------------------------------------------------
// joining the chunks
// ---------------------------------------------------------------------------
// Threads of a workgroup that joins segments. The backward's few segments have
// four parameters a column to write, so they are spread over more workgroups
// (128 samples of 256 channels in 32 groups, two chunks: 64 threads 4.8, 256
// 5.8 us); the forward's two are not (16 of 64 channels, 32 chunks: 64 threads
// half a microsecond more than 256, 4.4 us).
constexpr int join_threads(bool bwd) { return bwd ? 64 : 256; }
constexpr int kWideT = 1024;

// Statistics of segment (sample, group) S from its units of all chunks: lane
// j of `lanes` takes every lanes-th. Every caller's lanes sum in the same
// order.
__device__ __forceinline__ Sums segment_stats(const NormArgs& a, int S, int j, int lanes) {
  const NormGeo& g = a.g;
  const int n = g.e * g.nchunk;
  const long long NU = (long long)g.N * g.C / g.UW;
  const Part* part = a.part + (long long)S * g.e;
  constexpr int B = 8;
  Sums s;
  s.p = part->m;  // of the segment's first unit and chunk, for every lane
  for (int i = j; i < n; i += B * lanes) {
    Part q[B];
    int k[B];
#pragma unroll
    for (int b = 0; b < B; b++) {
      const int at = min(i + b * lanes, n - 1);
      k[b] = (int)fdiv((unsigned)at, g.de);
      q[b] = part[k[b] * NU + (at - k[b] * g.e)];
    }
#pragma unroll
    for (int b = 0; b < B; b++)
      if (i + b * lanes < n) s.add(q[b], (double)chunk_pixels(g, k[b]) * g.UW);
  }
  return s;
}

// The same for the backward: sums of gamma g and gamma g xh.
__device__ __forceinline__ void segment_sums(const NormArgs& a, int S, int j, int lanes, double& s1, double& s2) {
  const NormGeo& g = a.g;
  const int n = g.D * g.nchunk, c0 = (S - S / g.G * g.G) * g.D;
  const long long NC = (long long)g.N * g.C;
  const float2* part = a.psum + (long long)S * g.D;
  constexpr int B = 8;
  s1 = s2 = 0;
  for (int i = j; i < n; i += B * lanes) {
    float2 w[B];
    float gm[B];
#pragma unroll
    for (int b = 0; b < B; b++) {
      const int at = min(i + b * lanes, n - 1);
      const int k = (int)fdiv((unsigned)at, g.dD), u = at - k * g.D;
      w[b] = part[k * NC + u];
      gm[b] = a.gamma ? a.gamma[c0 + u] : 1.0f;
    }
#pragma unroll
    for (int b = 0; b < B; b++)
      if (i + b * lanes < n) {
        s1 += (double)gm[b] * w[b].x;
        s2 += (double)gm[b] * w[b].y;
      }
  }
}

// k1 = rstd * mean_M(gamma g) and k2 = rstd^2 * mean_M(gamma g xh) of a group
// from the sums of gamma g and gamma g xh
__device__ __forceinline__ float2 grad_means(double s1, double s2, double M, float rstd) {
  return make_float2((float)((double)rstd * s1 / M), (float)((double)rstd * rstd * s2 / M));
}

// Segments S0 .. S0 + ns - 1 by a workgroup: (mean, rstd), or (k1, k2), into
// sseg.
template <bool BWD>
__device__ __forceinline__ void join_segments(const NormArgs& a, int S0, int ns, float2* sseg) {
  const NormGeo& g = a.g;
  const int L = g.lanes, j = (int)threadIdx.x & (L - 1), step = (int)blockDim.x / L;
  const double M = (double)g.P * g.D;
  for (int s = (int)threadIdx.x / L; s < ns; s += step) {
    if constexpr (BWD) {
      const float rstd = a.rstd_in[S0 + s];
      double s1, s2;
      segment_sums(a, S0 + s, j, L, s1, s2);
      s1 = group_sum(s1, L);
      s2 = group_sum(s2, L);
      if (j == 0) sseg[s] = grad_means(s1, s2, M, rstd);
    } else {
      Sums t = segment_stats(a, S0 + s, j, L);
      t.s = group_sum(t.s, L);
      t.sq = group_sum(t.sq, L);
      if (j == 0) sseg[s] = finish_stats(t, M, a.eps);
    }
  }
  __syncthreads();
}

// What spreading reads for column i of the segments from S0 on.
struct ColIn {
  float ga, mean, rstd;
};
template <bool BWD>
__device__ __forceinline__ ColIn column_in(const NormArgs& a, int S0, int ns, int i) {
  const NormGeo& g = a.g;
  i = min(i, ns * g.D - 1);
  const int S = S0 + (int)fdiv((unsigned)i, g.dD), c = i - (S - S0) * g.D + (S - S / g.G * g.G) * g.D;
  return ColIn{a.gamma ? a.gamma[c] : 1.0f, BWD ? a.mean_in[S] : 0.0f, BWD ? a.rstd_in[S] : 0.0f};
}
// The columns' parameters of segments S0 .. S0 + ns - 1; `in` is what the
// thread's first column reads, requested before the segments were joined.
template <bool BWD>
__device__ __forceinline__ void spread_segments(const NormArgs& a, int S0, int ns, const float2* sseg, ColIn in) {
  const NormGeo& g = a.g;
  const long long col0 = (long long)S0 * g.D;
  for (int i = (int)threadIdx.x; i < ns * g.D; i += (int)blockDim.x) {
    if (i != (int)threadIdx.x) in = column_in<BWD>(a, S0, ns, i);
    const float2 st = sseg[fdiv((unsigned)i, g.dD)];
    a.col.mean[col0 + i] = BWD ? in.mean : st.x;
    a.col.a[col0 + i] = (BWD ? in.rstd : st.y) * in.ga;
    if constexpr (BWD) {
      a.col.k1[col0 + i] = st.x;
      a.col.k2[col0 + i] = st.y;
    }
  }
}
__device__ __forceinline__ void keep_stats(const NormArgs& a, int S0, int ns, const float2* sseg) {
  for (int s = (int)threadIdx.x; s < ns; s += (int)blockDim.x) {
    if (a.mean) a.mean[S0 + s] = sseg[s].x;
    if (a.rstd) a.rstd[S0 + s] = sseg[s].y;
  }
}

// join_threads / lanes segments a workgroup, a latency of three dependent
// loads: what it costs is mostly its launch.
template <bool BWD>
__global__ __launch_bounds__(join_threads(BWD)) void norm_join_kernel(const NormArgs a) {
  __shared__ float2 sseg[join_threads(BWD)];
  const int per = join_threads(BWD) / a.g.lanes, S0 = (int)blockIdx.x * per, ns = min(per, a.g.N * a.g.G - S0);
  const ColIn in = column_in<BWD>(a, S0, ns, (int)threadIdx.x);
  join_segments<BWD>(a, S0, ns, sseg);
  if constexpr (!BWD) keep_stats(a, S0, ns, sseg);
  spread_segments<BWD>(a, S0, ns, sseg, in);
}

// A workgroup for every segment.
template <bool BWD>
__global__ __launch_bounds__(kWideT) void norm_join_wide_kernel(const NormArgs a) {
  __shared__ double r1[kWideT / 64], r2[kWideT / 64];
  __shared__ float2 sseg[1];
  const int S = (int)blockIdx.x, t = (int)threadIdx.x;
  const ColIn in = column_in<BWD>(a, S, 1, t);
  double s1, s2;
  Sums stats;
  if constexpr (BWD) {
    segment_sums(a, S, t, kWideT, s1, s2);
  } else {
    stats = segment_stats(a, S, t, kWideT);
    s1 = stats.s;
    s2 = stats.sq;
  }
  s1 = group_sum(s1, 64);
  s2 = group_sum(s2, 64);
  if ((t & 63) == 0) {
    r1[t >> 6] = s1;
    r2[t >> 6] = s2;
  }
  __syncthreads();
  if (t == 0) {
    for (int k = 1; k < kWideT / 64; k++) {
      s1 += r1[k];
      s2 += r2[k];
    }
    const double M = (double)a.g.P * a.g.D;
    if constexpr (BWD) {
      sseg[0] = grad_means(s1, s2, M, a.rstd_in[S]);
    } else {
      stats.s = s1;
      stats.sq = s2;
      sseg[0] = finish_stats(stats, M, a.eps);
    }
  }
  __syncthreads();
  if constexpr (!BWD) keep_stats(a, S, 1, sseg);
  spread_segments<BWD>(a, S, 1, sseg, in);
}

// Segments of the columns of a tile: the first one, and how many.
__device__ __forceinline__ int tile_segments(const NormGeo& g, int tile, int& ns) {
  const Oct first = octet(g, tile * g.tx, true), last = octet(g, min(g.TO, (tile + 1) * g.tx) - 1, true);
  const int S0 = first.n * g.G + (int)fdiv((unsigned)first.c0, g.dD);
  ns = last.n * g.G + (int)fdiv((unsigned)(last.c0 + last.cnt - 1), g.dD) - S0 + 1;
  return S0;
}
constexpr int kTileOcts = 16;  // widest tile, so at most 8 * kTileOcts segments of it

// y, on the tiles and chunks of the statistics. Every workgroup joins the few
// chunks of its own columns while its first pixels are on their way, which
// saves a launch. Bound by memory: 160 x 160 x 32 x 128 146 us, 839 MB at
// 5.8 TB/s.
template <bool FULL, int ACT>
__global__ __launch_bounds__(256) void norm_apply_kernel(const NormArgs a) {
  const NormGeo& g = a.g;
  const int chunk = (int)blockIdx.x / g.ntile, tile = (int)blockIdx.x - chunk * g.ntile;
  const int ox = (int)threadIdx.x % g.tx, py = (int)threadIdx.x / g.tx;
  const int o = tile * g.tx + ox;
  const bool active = py < g.ty && o < g.TO;
  const Oct t = octet(g, o, active);
  const long long stride = (long long)g.N * g.C;
  const int p0 = chunk * g.ty + py, dp = g.nchunk * g.ty;
  // (the first pixels are requested before the parameters)
  float next[kBatch][8], mean[8], ga[8], be[8];
  auto load = [&](int p) {
#pragma unroll
    for (int k = 0; k < kBatch; k++) {
      const int q = p + k * dp;
      load_run<8, FULL>(a.x + (q < g.P ? q : 0) * stride + t.col, q < g.P ? t.cnt : 0, next[k]);
    }
  };
  load(p0);
  if (g.wide) {
    load_run<8, FULL>(a.col.mean + t.col, t.cnt, mean);
    load_run<8, FULL>(a.col.a + t.col, t.cnt, ga);
    load_optional<FULL>(a.beta, t.c0, t.cnt, 0.0f, be);
  } else {
    __shared__ float2 sseg[8 * kTileOcts];
    int ns;
    const int S0 = tile_segments(g, tile, ns);
    affine<FULL>(a, t, ga, be);
    join_segments<false>(a, S0, ns, sseg);
    if (chunk == 0) keep_stats(a, S0, ns, sseg);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const bool ok = i < t.cnt;
      const float2 st = sseg[ok ? t.n * g.G + (int)fdiv((unsigned)(t.c0 + i), g.dD) - S0 : 0];
      mean[i] = ok ? st.x : 0.0f;
      ga[i] = ok ? st.y * ga[i] : 0.0f;
    }
  }
  if (!active) return;
  const DropKey key = drop_key(a.drop);
  for (int p = p0; p < g.P; p += kBatch * dp) {
    float v[kBatch][8];
#pragma unroll
    for (int k = 0; k < kBatch; k++)
#pragma unroll
      for (int i = 0; i < 8; i++) v[k][i] = next[k][i];
    load(p + kBatch * dp);
#pragma unroll
    for (int k = 0; k < kBatch; k++) {
      const int q = p + k * dp;
      if (q >= g.P) break;
      float u[8];
      norm_values<8>(mean, ga, be, v[k], u);
      act_values<ACT, 8>(u);
      drop_values<8>(a.drop, key, (uint32_t)q * g.N + t.n, t.c0, u);
      store_run<8, FULL>(a.out + q * stride + t.col, t.cnt, u);
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// mean, rstd, gamma * rstd and beta of an octet from the forward's statistics
template <bool FULL>
__device__ __forceinline__ void grad_params(const NormArgs& a, const Oct& t, float (&mean)[8], float (&rstd)[8],
                                            float (&ga)[8], float (&be)[8]) {
  const NormGeo& g = a.g;
  affine<FULL>(a, t, ga, be);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const bool ok = i < t.cnt;
    const int s = t.n * g.G + (int)fdiv((unsigned)(t.c0 + (ok ? i : 0)), g.dD);
    mean[i] = ok ? a.mean_in[s] : 0.0f;
    rstd[i] = ok ? a.rstd_in[s] : 0.0f;
    ga[i] = rstd[i] * ga[i];
  }
}

// turns x (in d) into x - mean, and dy (in gr) into g = drop(dy) act'(u), for one
// pixel of the octet
template <int ACT>
__device__ __forceinline__ void grad_terms(const NormArgs& a, const DropKey& key, const Oct& t, int p,
                                           const float (&mean)[8], const float (&ga)[8], const float (&be)[8],
                                           float (&d)[8], float (&gr)[8]) {
  float u[8];
  norm_values<8>(mean, ga, be, d, u);
  drop_values<8>(a.drop, key, (uint32_t)p * a.g.N + t.n, t.c0, gr);
  act_slopes<ACT, 8>(u, gr);
}

// The gradient of a slab of whole groups whose x and dy stay in registers: the
// columns' sums of g and g (x - mean) through LDS, the groups' means of them,
// then dx. Bound by latency (124 x 4 x 32 x 8, GELU: 10.1 us, and 3.8 of the
// channels' sums behind it).
template <int R, bool FULL, int ACT>
__global__ __launch_bounds__(512) void norm_one_backward_kernel(const NormArgs a) {
  extern __shared__ float2 sh[];
  const NormGeo& g = a.g;
  const int W = g.so * 8;             // columns of the slab (some past a sample's last channel)
  float2* const su = sh;              // [ty1][W], then the columns' sums in its first row
  float2* const sseg = sh + g.ty1 * W;
  const int ox = (int)threadIdx.x % g.so, py = (int)threadIdx.x / g.so;
  const int o0 = xcd_order((int)blockIdx.x, (int)gridDim.x) * g.so;
  const bool active = py < g.ty1 && o0 + ox < g.TO;
  const Oct t = octet(g, o0 + ox, active);
  const long long stride = (long long)g.N * g.C;
  const int rows = active ? (g.P - py + g.ty1 - 1) / g.ty1 : 0;
  float d[R][8], gr[R][8];
#pragma unroll
  for (int k = 0; k < R; k++) {
    const int cnt = k < rows ? t.cnt : 0;
    const long long at = (k < rows ? py + k * g.ty1 : 0) * stride + t.col;
    load_run<8, FULL>(a.x + at, cnt, d[k]);
    load_run<8, FULL>(a.dy + at, cnt, gr[k]);
  }
  float mean[8], rstd[8], ga[8], be[8];
  const DropKey key = drop_key(a.drop);
  if (active) {
    grad_params<FULL>(a, t, mean, rstd, ga, be);
    float s1[8], s2[8];
#pragma unroll
    for (int i = 0; i < 8; i++) s1[i] = s2[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < R; k++)
      if (k < rows) {
        grad_terms<ACT>(a, key, t, py + k * g.ty1, mean, ga, be, d[k], gr[k]);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          s1[i] += gr[k][i];
          s2[i] = __builtin_fmaf(gr[k][i], d[k][i], s2[i]);
        }
      }
#pragma unroll
    for (int i = 0; i < 8; i++) su[py * W + ox * 8 + i] = make_float2(s1[i], s2[i] * rstd[i]);
  }
  __syncthreads();
  // the columns' sums over the rows, T at a time
  const int T = (int)blockDim.x;
  double* const x1 = reinterpret_cast<double*>(sseg);  // [T], x2 behind it: before the segments' values
  for (int w0 = 0; w0 < W; w0 += T) {
    const int w = min(T, W - w0);
    if (w0 > 0) __syncthreads();
    reduce_rows(
        T, w, g.ty1, x1, x1 + T,
        [&](int r, int i, double& s1, double& s2) {
          s1 += su[r * W + w0 + i].x;
          s2 += su[r * W + w0 + i].y;
        },
        [&](int i, double s1, double s2) {
          i += w0;
          const int oo = o0 + (i >> 3);
          if (oo >= g.TO) return;
          const Oct q = octet(g, oo, true);
          if ((i & 7) >= q.cnt) return;
          const float2 tot = make_float2((float)s1, (float)s2);
          a.psum[q.col + (i & 7)] = tot;
          su[i] = tot;  // (row 0 of this column, which only this thread still reads)
        });
  }
  __syncthreads();
  const int n0 = (int)fdiv((unsigned)o0, g.dNO);
  const int S0 = n0 * g.G + (o0 - n0 * g.NO) * 8 / g.D;
  {
    const int lanes = seg_lanes((int)blockDim.x, g.nseg);
    const int j = (int)threadIdx.x & (lanes - 1);
    const double M = (double)g.P * g.D;
    for (int s = (int)threadIdx.x / lanes; s < g.nseg && S0 + s < g.N * g.G; s += (int)blockDim.x / lanes) {
      const int S = S0 + s, n = S / g.G, grp = S - n * g.G;
      const int pos = (n * g.NO - o0) * 8 + grp * g.D;
      double s1 = 0, s2 = 0;
      for (int i = j; i < g.D; i += lanes) {
        const float2 w = su[pos + i];
        const double gm = a.gamma ? (double)a.gamma[grp * g.D + i] : 1.0;
        s1 += gm * w.x;
        s2 += gm * w.y;
      }
      s1 = group_sum(s1, lanes);
      s2 = group_sum(s2, lanes);
      if (j == 0) sseg[s] = grad_means(s1, s2, M, a.rstd_in[S]);
    }
  }
  __syncthreads();
  if (!active) return;
  float k1[8], k2[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const bool ok = i < t.cnt;
    const float2 k = sseg[t.n * g.G + (int)fdiv((unsigned)(t.c0 + (ok ? i : 0)), g.dD) - S0];
    k1[i] = ok ? k.x : 0.0f;
    k2[i] = ok ? k.y : 0.0f;
  }
  if (a.out) {
#pragma unroll
    for (int k = 0; k < R; k++)
      if (k < rows) {
        float dx[8];
        norm_grad_values<8>(ga, k1, k2, d[k], gr[k], dx);
        store_run<8, FULL>(a.out + (py + k * g.ty1) * stride + t.col, t.cnt, dx);
      }
  } else if (py == 0) {
    store_run<8, FULL>(a.col.mean + t.col, t.cnt, mean);
    store_run<8, FULL>(a.col.a + t.col, t.cnt, ga);
    store_run<8, FULL>(a.col.k1 + t.col, t.cnt, k1);
    store_run<8, FULL>(a.col.k2 + t.col, t.cnt, k2);
  }
}

// Sums of very many rows of sums (samples and chunks) to kFoldRows.
constexpr int kFoldC = 32;
__global__ __launch_bounds__(256) void norm_fold_kernel(const NormArgs a) {
  const int cb = (int)blockIdx.x / kFoldRows, k = (int)blockIdx.x - cb * kFoldRows;
  const int per = (a.sum_rows + kFoldRows - 1) / kFoldRows, r0 = min(a.sum_rows, k * per);
  double s1, s2;
  sum_rows<kFoldC>(a.sum_src, a.g.C, cb * kFoldC, r0, min(a.sum_rows, r0 + per), s1, s2);
  const int c = cb * kFoldC + (int)threadIdx.x;
  if (threadIdx.x < kFoldC && c < a.g.C) a.fold[(long long)k * a.g.C + c] = make_float2((float)s1, (float)s2);
}

// dgamma and dbeta behind the one-pass kernel
__global__ __launch_bounds__(256) void norm_channel_kernel(const NormArgs a) {
  norm_channel_sums(a, (int)blockIdx.x, (int)gridDim.x);
}

// Every column's sums of g and g xh over a chunk of pixels: one read of x and
// dy. Columns, not groups, because dgamma and dbeta need them. Bound by
// reading: 20 x 20 x 128 x 256 20.8 us (5.0 TB/s; vector instructions in 56% of
// the busy cycles), 80 x 80 x 16 x 64 12.0 us.
template <bool FULL, int ACT>
__global__ __launch_bounds__(256) void norm_sums_kernel(const NormArgs a) {
  __shared__ float2 su[256 * 8];
  const NormGeo& g = a.g;
  const int chunk = (int)blockIdx.x / g.ntile, tile = (int)blockIdx.x - chunk * g.ntile;
  const int ox = (int)threadIdx.x % g.tx, py = (int)threadIdx.x / g.tx;
  const int o = tile * g.tx + ox;
  const bool active = py < g.ty && o < g.TO;
  const Oct t = octet(g, o, active);
  const long long stride = (long long)g.N * g.C;
  const int p0 = chunk * g.ty + py, dp = g.nchunk * g.ty;
  double s1[8], s2[8];  // (a thread's pixels are thousands where there are many columns)
#pragma unroll
  for (int i = 0; i < 8; i++) s1[i] = s2[i] = 0;
  if (active) {
    constexpr int B = kBatch / 2;  // two tensors
    float nd[B][8], ng[B][8];
    auto load = [&](int p) {
#pragma unroll
      for (int k = 0; k < B; k++) {
        const int q = p + k * dp, cnt = q < g.P ? t.cnt : 0;
        const long long at = (q < g.P ? q : 0) * stride + t.col;
        load_run<8, FULL>(a.x + at, cnt, nd[k]);
        load_run<8, FULL>(a.dy + at, cnt, ng[k]);
      }
    };
    load(p0);
    float mean[8], rstd[8], ga[8], be[8];
    grad_params<FULL>(a, t, mean, rstd, ga, be);
    const DropKey key = drop_key(a.drop);
    for (int p = p0; p < g.P; p += B * dp) {
      float d[B][8], gr[B][8];
#pragma unroll
      for (int k = 0; k < B; k++)
#pragma unroll
        for (int i = 0; i < 8; i++) {
          d[k][i] = nd[k][i];
          gr[k][i] = ng[k][i];
        }
      load(p + B * dp);
#pragma unroll
      for (int k = 0; k < B; k++) {
        const int q = p + k * dp;
        if (q >= g.P) break;
        grad_terms<ACT>(a, key, t, q, mean, ga, be, d[k], gr[k]);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          s1[i] += gr[k][i];
          s2[i] = __builtin_fma((double)gr[k][i], (double)d[k][i], s2[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) s2[i] *= rstd[i];
  }
  const int W = g.tx * 8;
  if (py < g.ty)
#pragma unroll
    for (int i = 0; i < 8; i++) su[py * W + ox * 8 + i] = make_float2((float)s1[i], (float)s2[i]);
  __syncthreads();
  const long long NC = stride;
  __shared__ double x1[256], x2[256];
  reduce_rows(
      256, W, g.ty, x1, x2,
      [&](int r, int i, double& s1, double& s2) {
        s1 += su[r * W + i].x;
        s2 += su[r * W + i].y;
      },
      [&](int i, double s1, double s2) {
        const int oo = tile * g.tx + (i >> 3);
        if (oo >= g.TO) return;
        const Oct q = octet(g, oo, true);
        if ((i & 7) >= q.cnt) return;
        a.psum[chunk * NC + q.col + (i & 7)] = make_float2((float)s1, (float)s2);
      });
}

// dx, on the tiles and chunks of the sums, whose chunks it joins for its own
// columns; the first `extra` workgroups sum dgamma and dbeta. Bound by memory
// and, at small sizes, by the chain of loads before the first result: 80 x 80 x
// 16 x 64 18.7 us (79 MB), 80 x 80 x 64 x 64 56 us (315 MB, 5.6 TB/s).
template <bool FULL, int ACT>
__global__ __launch_bounds__(256) void norm_apply_backward_kernel(const NormArgs a, int extra) {
  const NormGeo& g = a.g;
  if ((int)blockIdx.x < extra) {
    norm_channel_sums(a, (int)blockIdx.x, extra);
    return;
  }
  const int id = (int)blockIdx.x - extra;
  const int chunk = id / g.ntile, tile = id - chunk * g.ntile;
  const int ox = (int)threadIdx.x % g.tx, py = (int)threadIdx.x / g.tx;
  const int o = tile * g.tx + ox;
  const bool active = py < g.ty && o < g.TO;
  const Oct t = octet(g, o, active);
  const long long stride = (long long)g.N * g.C;
  const int p0 = chunk * g.ty + py, dp = g.nchunk * g.ty;
  constexpr int B = kBatch / 2;
  float nd[B][8], ng[B][8];
  auto load = [&](int p) {
#pragma unroll
    for (int k = 0; k < B; k++) {
      const int q = p + k * dp, cnt = q < g.P ? t.cnt : 0;
      const long long at = (q < g.P ? q : 0) * stride + t.col;
      load_run<8, FULL>(a.x + at, cnt, nd[k]);
      load_run<8, FULL>(a.dy + at, cnt, ng[k]);
    }
  };
  load(p0);
  float mean[8], ga[8], be[8], k1[8], k2[8];
  if (g.wide) {
    load_run<8, FULL>(a.col.mean + t.col, t.cnt, mean);
    load_run<8, FULL>(a.col.a + t.col, t.cnt, ga);
    load_run<8, FULL>(a.col.k1 + t.col, t.cnt, k1);
    load_run<8, FULL>(a.col.k2 + t.col, t.cnt, k2);
    load_optional<FULL>(a.beta, t.c0, t.cnt, 0.0f, be);
  } else {
    __shared__ float2 sseg[8 * kTileOcts];
    int ns;
    const int S0 = tile_segments(g, tile, ns);
    float rstd[8];
    grad_params<FULL>(a, t, mean, rstd, ga, be);
    join_segments<true>(a, S0, ns, sseg);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const bool ok = i < t.cnt;
      const float2 k = sseg[ok ? t.n * g.G + (int)fdiv((unsigned)(t.c0 + i), g.dD) - S0 : 0];
      k1[i] = ok ? k.x : 0.0f;
      k2[i] = ok ? k.y : 0.0f;
    }
  }
  if (!active) return;
  const DropKey key = drop_key(a.drop);
  for (int p = p0; p < g.P; p += B * dp) {
    float d[B][8], gr[B][8];
#pragma unroll
    for (int k = 0; k < B; k++)
#pragma unroll
      for (int i = 0; i < 8; i++) {
        d[k][i] = nd[k][i];
        gr[k][i] = ng[k][i];
      }
    load(p + B * dp);
#pragma unroll
    for (int k = 0; k < B; k++) {
      const int q = p + k * dp;
      if (q >= g.P) break;
      grad_terms<ACT>(a, key, t, q, mean, ga, be, d[k], gr[k]);
      float dx[8];
      norm_grad_values<8>(ga, k1, k2, d[k], gr[k], dx);
      store_run<8, FULL>(a.out + q * stride + t.col, t.cnt, dx);
    }
  }
}

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

// The workspace's parts: the columns' parameters, the rows of sums of many
// samples and chunks, and the chunks' partial statistics or sums.
struct NormWs {
  size_t cols, fold, part, bytes;
  int rows;  // backward: rows of sums
};
NormWs norm_ws(const NormGeo& g, bool backward) {
  NormWs w{};
  const size_t nc = (size_t)g.N * g.C, chunks = g.one ? 1 : (size_t)g.nchunk;
  w.cols = align256(nc * sizeof(float));
  w.fold = w.cols * (backward ? 4 : 2);
  w.part = w.fold;
  if (backward) {
    w.rows = (int)(g.N * chunks);
    if (w.rows > kFoldFrom) w.part += align256((size_t)kFoldRows * g.C * sizeof(float2));
    w.bytes = w.part + chunks * nc * sizeof(float2);
  } else {
    w.bytes = w.part + (g.one ? 0 : chunks * (nc / g.UW) * sizeof(Part));
  }
  return w;
}

void bind_ws(NormArgs& a, void* ws, bool backward) {
  const NormWs w = norm_ws(a.g, backward);
  uint8_t* b = static_cast<uint8_t*>(ws);
  a.col.mean = reinterpret_cast<float*>(b);
  a.col.a = reinterpret_cast<float*>(b + w.cols);
  if (backward) {
    a.col.k1 = reinterpret_cast<float*>(b + 2 * w.cols);
    a.col.k2 = reinterpret_cast<float*>(b + 3 * w.cols);
    a.fold = reinterpret_cast<float2*>(b + w.fold);
    a.psum = reinterpret_cast<float2*>(b + w.part);
    a.sum_src = a.psum;
    a.sum_rows = w.rows;
  } else {
    a.part = reinterpret_cast<Part*>(b + w.part);
  }
}

template <int UW, bool FULL>
void launch_stats(const NormArgs& a, hipStream_t st) {
  const NormGeo& g = a.g;
  if (!g.one) {
    hipLaunchKernelGGL((norm_stats_kernel<UW, FULL>), dim3((unsigned)(g.ntile * g.nchunk)), dim3(256), 0, st, a);
    return;
  }
  const int R = ceil_div(g.P, g.ty1);
  const size_t lds = (size_t)(g.ty1 * g.so * (8 / UW)) * sizeof(Part) + (size_t)g.nseg * sizeof(float2);
  with_act(a.act, [&](auto act) {
    constexpr int A = decltype(act)::value;
    const auto kern = R <= 1   ? norm_one_kernel<1, UW, FULL, A>
                      : R <= 2 ? norm_one_kernel<2, UW, FULL, A>
                      : R <= 4 ? norm_one_kernel<4, UW, FULL, A>
                               : norm_one_kernel<kOneR, UW, FULL, A>;
    hipLaunchKernelGGL(kern, dim3((unsigned)g.nslab), dim3((unsigned)g.T1), lds, st, a);
  });
}
template <bool FULL>
void launch_stats(const NormArgs& a, hipStream_t st) {
  switch (a.g.UW) {
    case 1: launch_stats<1, FULL>(a, st); break;
    case 2: launch_stats<2, FULL>(a, st); break;
    case 4: launch_stats<4, FULL>(a, st); break;
    default: launch_stats<8, FULL>(a, st); break;
  }
}

// Joins the chunks of every group into the columns' parameters.
template <bool BWD>
void launch_join(const NormArgs& a, hipStream_t st) {
  const NormGeo& g = a.g;
  const int NS = g.N * g.G;
  if (g.wide) hipLaunchKernelGGL(norm_join_wide_kernel<BWD>, dim3((unsigned)NS), dim3(kWideT), 0, st, a);
  else {
    constexpr int T = join_threads(BWD);
    hipLaunchKernelGGL(norm_join_kernel<BWD>, dim3((unsigned)ceil_div(NS, T / g.lanes)), dim3(T), 0, st, a);
  }
}

template <bool FULL>
void launch_sums(const NormArgs& a, hipStream_t st) {
  const NormGeo& g = a.g;
  if (!g.one) {
    with_act(a.act, [&](auto act) {
      hipLaunchKernelGGL((norm_sums_kernel<FULL, decltype(act)::value>), dim3((unsigned)(g.ntile * g.nchunk)),
                         dim3(256), 0, st, a);
    });
    return;
  }
  const int R = ceil_div(g.P, g.ty1);
  const size_t lds = (size_t)g.ty1 * g.so * 8 * sizeof(float2) +
                     std::max((size_t)g.nseg * sizeof(float2), (size_t)g.T1 * 2 * sizeof(double));
  with_act(a.act, [&](auto act) {
    constexpr int A = decltype(act)::value;
    const auto kern = R <= 1   ? norm_one_backward_kernel<1, FULL, A>
                      : R <= 2 ? norm_one_backward_kernel<2, FULL, A>
                      : R <= 4 ? norm_one_backward_kernel<4, FULL, A>
                               : norm_one_backward_kernel<kOneR, FULL, A>;
    hipLaunchKernelGGL(kern, dim3((unsigned)g.nslab), dim3((unsigned)g.T1), lds, st, a);
  });
}

template <bool FULL>
void launch_apply(const NormArgs& a, hipStream_t st) {
  with_act(a.act, [&](auto act) {
    hipLaunchKernelGGL((norm_apply_kernel<FULL, decltype(act)::value>), dim3((unsigned)(a.g.ntile * a.g.nchunk)),
                       dim3(256), 0, st, a);
  });
}
template <bool FULL>
void launch_apply_backward(const NormArgs& a, int extra, hipStream_t st) {
  with_act(a.act, [&](auto act) {
    hipLaunchKernelGGL((norm_apply_backward_kernel<FULL, decltype(act)::value>),
                       dim3((unsigned)(a.g.ntile * a.g.nchunk + extra)), dim3(256), 0, st, a, extra);
  });
}

}  // namespace

size_t norm_workspace_bytes(const NormShape& s, int op) { return norm_ws(norm_geo(s, op == 1), op == 1).bytes; }

hipError_t launch_group_norm(const NormShape& s, const float* x, const float* gamma, const float* beta,
                             const DropSpec& drop, float* y, const MxOutView& yq, float* mean, float* rstd, void* ws,
                             hipStream_t st) {
  NormArgs a{};
  a.g = norm_geo(s, false);
  a.x = x; a.gamma = gamma; a.beta = beta; a.mean = mean; a.rstd = rstd; a.out = y;
  a.act = s.act; a.eps = s.eps; a.drop = drop_args(drop);
  bind_ws(a, ws, false);
  const NormGeo& g = a.g;
  const bool full = g.C % 8 == 0;
  if (full) launch_stats<true>(a, st);
  else launch_stats<false>(a, st);
  hipError_t e = launch_check();
  if (e != hipSuccess || (g.one && y)) return e;
  if (!g.one) {
    if (!y || g.wide) {
      launch_join<false>(a, st);
      e = launch_check();
      if (e != hipSuccess) return e;
    }
    if (y) {
      if (full) launch_apply<true>(a, st);
      else launch_apply<false>(a, st);
      return launch_check();
    }
  }
  return launch_norm_mx(a, yq, st);
}

hipError_t launch_group_norm_backward(const NormShape& s, const float* dy, const float* x, const float* gamma,
                                      const float* beta, const float* mean, const float* rstd, const DropSpec& drop,
                                      float* dx, const MxOutView& dxq, float* dgamma, float* dbeta, void* ws,
                                      hipStream_t st) {
  NormArgs a{};
  a.g = norm_geo(s, true);
  a.x = x; a.dy = dy; a.gamma = gamma; a.beta = beta; a.mean_in = mean; a.rstd_in = rstd; a.out = dx;
  a.dgamma = dgamma; a.dbeta = dbeta;
  a.act = s.act; a.eps = s.eps; a.drop = drop_args(drop);
  bind_ws(a, ws, true);
  const NormGeo& g = a.g;
  const bool full = g.C % 8 == 0;
  const int extra = dgamma || dbeta ? std::min(ceil_div(g.C, kSumC), kSumGroups) : 0;
  if (full) launch_sums<true>(a, st);
  else launch_sums<false>(a, st);
  hipError_t e = launch_check();
  if (e != hipSuccess) return e;
  if (extra && a.sum_rows > kFoldFrom) {
    hipLaunchKernelGGL(norm_fold_kernel, dim3((unsigned)(ceil_div(g.C, kFoldC) * kFoldRows)), dim3(256), 0, st, a);
    e = launch_check();
    if (e != hipSuccess) return e;
    a.sum_src = a.fold;
    a.sum_rows = kFoldRows;
  }
  if (!g.one) {
    if (!dx || g.wide) {
      launch_join<true>(a, st);
      e = launch_check();
      if (e != hipSuccess) return e;
    }
    if (dx) {
      if (full) launch_apply_backward<true>(a, extra, st);
      else launch_apply_backward<false>(a, extra, st);
      return launch_check();
    }
  } else if (dx) {
    if (!extra) return e;
    hipLaunchKernelGGL(norm_channel_kernel, dim3((unsigned)extra), dim3(256), 0, st, a);
    return launch_check();
  }
  return launch_norm_backward_mx(a, dxq, extra, st);
}

}  // namespace mq
