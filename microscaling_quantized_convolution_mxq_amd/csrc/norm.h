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
  // streaming: tiles of tx octets x chunks of ppc pixels, ty pixels at once
  int tx, ty, ntile, nchunk, ppc;
};
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

// dgamma and dbeta of channels 256 b .. 256 b + 255 from the sums of every
// sample, in their order.
__device__ __forceinline__ void norm_channel_sums(const NormArgs& a, int b) {
  for (int c = b * 256 + (int)threadIdx.x; c < min(a.g.C, b * 256 + 256); c += blockDim.x) {
    double s1 = 0, s2 = 0;
    for (int n = 0; n < a.g.N; n++) {
      const float2 t = a.tot[(long long)n * a.g.C + c];
      s1 += t.x;
      s2 += t.y;
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
