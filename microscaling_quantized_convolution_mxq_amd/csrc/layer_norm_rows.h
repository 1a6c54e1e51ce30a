// layer_norm_rows.h -- how the layer norm's kernels hold rows in registers, and their sums.
#pragma once
#include "layer_norm.h"

namespace mq {

typedef float quad_t[4];

// Channel of quad q of thread t of the row's T threads.
template <int T>
__device__ __forceinline__ int chan(int q, int t) {
  return (q * T + t) * 4;
}

// FULL: C is a multiple of four, so a quad is in the row or outside; loads then stand under no condition.
template <int T, int Q, bool FULL>
__device__ __forceinline__ void load_row(const float* row, int C, int t, quad_t (&v)[Q]) {
#pragma unroll
  for (int q = 0; q < Q; q++) {
    const int c = chan<T>(q, t);
    if (FULL) load_run<4, true>(row + (c < C ? c : 0), 4, v[q]);
    else load_run<4, false>(row + c, C - c, v[q]);
  }
}
template <int T, int Q, bool FULL>
__device__ __forceinline__ void store_row(float* row, int C, int t, const quad_t (&v)[Q]) {
#pragma unroll
  for (int q = 0; q < Q; q++) {
    const int c = chan<T>(q, t);
    store_run<4, FULL>(row + c, C - c, v[q]);
  }
}
// whether value i of quad q exists
template <int T, bool FULL>
__device__ __forceinline__ bool has(int q, int i, int t, int C) {
  return FULL ? chan<T>(q, t) < C : chan<T>(q, t) + i < C;
}

template <int T, int Q, bool FULL>
__device__ __forceinline__ void load_param(const float* p, int C, int t, float other, quad_t (&v)[Q]) {
  if (p) {
    load_row<T, Q, FULL>(p, C, t, v);
  } else {
#pragma unroll
    for (int q = 0; q < Q; q++)
#pragma unroll
      for (int i = 0; i < 4; i++) v[q][i] = other;
  }
}

template <int CTRL>
__device__ __forceinline__ double add_dpp(double a) {
  const long long b = __double_as_longlong(a);
  const int lo = __builtin_amdgcn_update_dpp(0, (int)b, CTRL, 0xF, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xF, 0xF, false);
  return a + __longlong_as_double(((long long)hi << 32) | (unsigned)lo);
}
__device__ __forceinline__ double lane_of(double a, int lane) {
  const long long b = __double_as_longlong(a);
  return __longlong_as_double(((long long)__builtin_amdgcn_readlane((int)(b >> 32), lane) << 32) |
                              (unsigned)__builtin_amdgcn_readlane((int)b, lane));
}
// Sum over aligned groups of T lanes, on every lane of the group: at each step
// a lane adds the sum of the other half of its group (DPP within 16 lanes).
template <int T>
__device__ __forceinline__ double group_sum(double a) {
  if constexpr (T >= 2) a = add_dpp<0xB1>(a);   // lane ^ 1
  if constexpr (T >= 4) a = add_dpp<0x4E>(a);   // lane ^ 2
  if constexpr (T >= 8) a = add_dpp<0x141>(a);  // 7 - lane within 8
  if constexpr (T >= 16) a = add_dpp<0x140>(a); // 15 - lane within 16
  if constexpr (T >= 32) a += __shfl_xor(a, 16);
  if constexpr (T >= 64) a = lane_of(a, 0) + lane_of(a, 32);
  return a;
}

// Sums of K values over a row's T threads, on all of them. Where these are
// several waves (a whole workgroup) each leaves its part in LDS; `phase`
// alternates between calls, so one barrier a call is enough: a wave that
// writes a phase's slots again has passed the barrier of the other phase, which
// every wave reaches only after its reads of this one.
template <int T, int K>
__device__ __forceinline__ void row_sums(double (&s)[K], int phase) {
#pragma unroll
  for (int k = 0; k < K; k++) s[k] = group_sum<(T < 64 ? T : 64)>(s[k]);
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    __shared__ double red[2][W][K];
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; k++) red[phase][w][k] = s[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; k++) {
      s[k] = red[phase][0][k];
#pragma unroll
      for (int i = 1; i < W; i++) s[k] += red[phase][i][k];
    }
  }
}

// (a reciprocal of C and one function: divisions cost a row of 64 channels a sixth of its time)
__device__ __forceinline__ float rstd_of(double sq, const LnArgs& a) {
  return (float)rsqrt(__builtin_fma(sq, a.inv, (double)a.eps));
}

// The column sums of a workgroup of B threads, as its row of `part`: groups of a wave by lanes, waves in turn through LDS
// (cols: B / 64 - 1 rows of T Q 4).
template <int T, int Q, int B>
__device__ __forceinline__ void leave_columns(const LnArgs& a, double2* cols, int t, double (&sb)[Q][4], double (&sg)[Q][4]) {
  if constexpr (T < 64) {
#pragma unroll
    for (int off = T; off < 64; off *= 2)
#pragma unroll
      for (int q = 0; q < Q; q++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          sb[q][i] += __shfl_xor(sb[q][i], off);
          sg[q][i] += __shfl_xor(sg[q][i], off);
        }
  }
  if constexpr (T <= 64) {
    const int w = threadIdx.x >> 6;
    if (w > 0 && (threadIdx.x & 63) < T)
#pragma unroll
      for (int q = 0; q < Q; q++)
#pragma unroll
        for (int i = 0; i < 4; i++) cols[(w - 1) * (T * Q * 4) + chan<T>(q, t) + i] = make_double2(sb[q][i], sg[q][i]);
    __syncthreads();
    if (threadIdx.x >= T) return;
#pragma unroll
    for (int q = 0; q < Q; q++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        for (int k = 0; k < B / 64 - 1; k++) {
          const double2 o = cols[k * (T * Q * 4) + chan<T>(q, t) + i];
          sb[q][i] += o.x;
          sg[q][i] += o.y;
        }
  }
  float2* const to = a.part + (long long)blockIdx.x * a.C;
#pragma unroll
  for (int q = 0; q < Q; q++)
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (chan<T>(q, t) + i < a.C) to[chan<T>(q, t) + i] = make_float2((float)sb[q][i], (float)sg[q][i]);
}

}  // namespace mq
