// norm.h -- the group norm's plan (which kernels a shape takes, and their
// tiles) and the arguments its kernels share.
#pragma once
#include "block.h"
#include "block_common.h"

namespace mq {

DropArgs drop_args(const DropSpec& d);

// The row of N * C values of a pixel as octets of channels: octet o holds
// channels 8 (o % NO) .. of sample o / NO (fewer than 8 in a sample's last
// one). A unit is UW = gcd(D, 8) neighbouring channels, which one group
// holds.
struct NormGeo {
  int P, N, C, G, D, NO, TO;  // TO = N * NO octets a pixel
  int UW;
  FastDiv dNO, dD;
  // one workgroup holds a slab of `so` octets of all pixels in registers
  bool one;
  int so, ty1, T1, nslab, nseg;
  // streaming: tiles of tx octets; groups of ty neighbouring pixels, of which
  // chunk k takes groups k, k + nchunk, ... (what runs at one time is then
  // one stretch of memory, whose lines fall on all channels alike)
  int tx, ty, ntile, nchunk, ngroup;
  // joining the chunks of a group: its units (backward: columns) of all
  // chunks by `lanes` neighbouring lanes, or (wide) by a workgroup
  int e, lanes;
  bool wide;
  FastDiv de;
};
// pixels of chunk k
__device__ __forceinline__ int chunk_pixels(const NormGeo& g, int k) {
  const int n = (g.ngroup - k + g.nchunk - 1) / g.nchunk * g.ty;
  return n - ((g.ngroup - 1) % g.nchunk == k ? g.ngroup * g.ty - g.P : 0);
}
NormGeo norm_geo(const NormShape& s, bool backward);

// Per-column parameters of the elementwise pass, [N * C] floats each: mean
// and gamma * rstd, and for the backward k1 = rstd * mean_M(gamma g) and k2 =
// rstd^2 * mean_M(gamma g xh).
struct NormCols {
  float *mean, *a, *k1, *k2;
};

struct NormPart {
  float m, lo, q;
};

struct NormArgs {
  NormGeo g;
  const float *x, *dy, *gamma, *beta;
  const float *mean_in, *rstd_in;  // backward
  float *mean, *rstd;              // forward's statistics (may be null)
  float* out;                      // y or dx; null: the columns' parameters instead
  NormPart* part;                  // streaming: chunks' statistics [nchunk][N * C / UW]
  float2* psum;                    // backward: sums of g and g xh of the chunks [nchunk][N][C]
  const float2* sum_src;           // dgamma, dbeta: rows of sums [sum_rows][C]
  int sum_rows;
  float2* fold;                    // rows of sums [kFoldRows][C]
  NormCols col;
  float *dgamma, *dbeta;
  int act;
  float eps;
  DropArgs drop;
};

hipError_t launch_norm_mx(const NormArgs& a, const MxOutView& out, hipStream_t st);
hipError_t launch_norm_backward_mx(const NormArgs& a, const MxOutView& out, int extra, hipStream_t st);

// Sums of rows r0 .. r1 - 1 of `rows` [.][C] over channels c0 .. c0 + W - 1 by
// a workgroup of up to 512 threads: thread t takes channel t % W of rows r0 +
// t / W, .... Thread t < W gets its channel's sums.
template <int W>
__device__ __forceinline__ void sum_rows(const float2* rows, int C, int c0, int r0, int r1, double& s1, double& s2) {
  __shared__ double x1[512], x2[512];
  const int t = (int)threadIdx.x, n = (int)blockDim.x / W, r = t / W, c = c0 + t % W;
  s1 = s2 = 0;
  if (c < C) {
    constexpr int B = 8;
    for (int i = r0 + r; i < r1; i += B * n) {
      float2 w[B];
#pragma unroll
      for (int j = 0; j < B; j++)
        w[j] = i + j * n < r1 ? rows[(long long)(i + j * n) * C + c] : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < B; j++) {
        s1 += w[j].x;
        s2 += w[j].y;
      }
    }
  }
  x1[t] = s1;
  x2[t] = s2;
  __syncthreads();
  if (t < W)
    for (int k = 1; k < n; k++) {
      s1 += x1[k * W + t];
      s2 += x2[k * W + t];
    }
}

// dgamma and dbeta by workgroup b of n: eight channels at a time, so that its
// threads share the samples' and chunks' rows between them (a thread a channel
// had been the tail of the whole gradient). At most kSumGroups workgroups: one
// for every eight of 2^27 channels would be more threads than a launch takes.
constexpr int kSumC = 8, kSumGroups = 1 << 16;
constexpr int kFoldRows = 64, kFoldFrom = 1024;  // more rows than kFoldFrom are first summed to kFoldRows
__device__ __forceinline__ void norm_channel_sums(const NormArgs& a, int b, int n) {
  for (int c0 = b * kSumC; c0 < a.g.C; c0 += n * kSumC) {
    if (c0 != b * kSumC) __syncthreads();  // (the sums before are read)
    double s1, s2;
    sum_rows<kSumC>(a.sum_src, a.g.C, c0, 0, a.sum_rows, s1, s2);
    const int c = c0 + (int)threadIdx.x;
    if (threadIdx.x < kSumC && c < a.g.C) {
      if (a.dbeta) a.dbeta[c] = (float)s1;
      if (a.dgamma) a.dgamma[c] = (float)s2;
    }
  }
}

// u = (x - mean) * a + beta, and with x turned into x - mean.
template <int K>
__device__ __forceinline__ void norm_values(const float (&mean)[K], const float (&a)[K], const float (&be)[K],
                                            float (&x)[K], float (&u)[K]) {
#pragma clang fp contract(off)
#pragma unroll
  for (int i = 0; i < K; i++) {
    x[i] = x[i] - mean[i];
    u[i] = __builtin_fmaf(x[i], a[i], be[i]);
  }
}
// dx from d = x - mean and g.
template <int K>
__device__ __forceinline__ void norm_grad_values(const float (&a)[K], const float (&k1)[K], const float (&k2)[K],
                                                 const float (&d)[K], const float (&g)[K], float (&dx)[K]) {
#pragma unroll
  for (int i = 0; i < K; i++) dx[i] = __builtin_fmaf(-k2[i], d[i], __builtin_fmaf(a[i], g[i], -k1[i]));
}

}  // namespace mq
