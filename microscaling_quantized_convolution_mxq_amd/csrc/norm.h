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
// holds; a group is e = D / UW units.
struct NormGeo {
  int P, N, C, G, D, NO, TO;  // TO = N * NO octets a pixel
  int UW, e;
  FastDiv dNO, dD;
  // one workgroup holds a slab of `so` octets of all pixels in registers
  bool one;
  int so, ty1, T1, nslab, nseg;
  // streaming: tiles of tx octets; groups of ty neighbouring pixels, of which
  // chunk k takes groups k, k + nchunk, ... (what runs at one time is then
  // one stretch of memory, whose lines fall on all channels alike)
  int tx, ty, ntile, nchunk, ngroup;
};
// pixels of row py (of ty) in chunk k
__device__ __forceinline__ int chunk_rows(const NormGeo& g, int k, int py) {
  const int n = (g.ngroup - k + g.nchunk - 1) / g.nchunk;
  const int last = g.ngroup - 1;
  return n - (last % g.nchunk == k && last * g.ty + py >= g.P ? 1 : 0);
}
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
  float2* psum;                    // streaming backward: chunks' sums [nchunk][N * C]
  float2* tot;                     // backward: sums over the pixels [N * C]
  NormCols col;
  float *dgamma, *dbeta;
  int act;
  float eps;
  DropArgs drop;
};

hipError_t launch_norm_mx(const NormArgs& a, const MxOutView& out, hipStream_t st);
hipError_t launch_norm_backward_mx(const NormArgs& a, const MxOutView& out, int extra, hipStream_t st);

// dgamma and dbeta of channels kSumC b .. from the sums of every sample, by a
// workgroup of up to 512 threads: thread t takes channel t % kSumC of samples
// t / kSumC, ... (one thread a channel would wait for memory once a sample).
constexpr int kSumC = 32;
__device__ __forceinline__ void norm_channel_sums(const NormArgs& a, int b) {
  __shared__ double r1[512], r2[512];
  const int t = (int)threadIdx.x, rows = (int)blockDim.x / kSumC, r = t / kSumC;
  const int c = b * kSumC + t % kSumC, C = a.g.C, N = a.g.N;
  double s1 = 0, s2 = 0;
  if (c < C) {
    int n = r;
    for (; n + 3 * rows < N; n += 4 * rows) {
      float2 w[4];
#pragma unroll
      for (int j = 0; j < 4; j++) w[j] = a.tot[(long long)(n + j * rows) * C + c];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        s1 += w[j].x;
        s2 += w[j].y;
      }
    }
    for (; n < N; n += rows) {
      const float2 w = a.tot[(long long)n * C + c];
      s1 += w.x;
      s2 += w.y;
    }
  }
  r1[t] = s1;
  r2[t] = s2;
  __syncthreads();
  if (r == 0 && c < C) {
    for (int k = 1; k < rows; k++) {
      s1 += r1[k * kSumC + t];
      s2 += r2[k * kSumC + t];
    }
    if (a.dbeta) a.dbeta[c] = (float)s1;
    if (a.dgamma) a.dgamma[c] = (float)s2;
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
