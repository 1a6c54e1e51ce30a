// mx_rows.h -- writes an [pixel][N][C] tensor as MX codes and scales whose
// values a source computes on the fly (group norm, its gradient, dropout,
// samples of a replay cache), exactly as a quantization of the fp32 tensor
// would, without that tensor reaching memory.
//
// A wave takes a tile of 32 rows x one block of 32 channels: lane l has row
// l / 2 and the 16 channels (l % 2) * 16 .., the quantizer's own arrangement,
// so block maximum, scale, rounding and packing are its functions. Rows of a
// tile are consecutive in memory: 32 samples of one pixel, or, with fewer
// samples, all samples of 32 / N pixels. A wave keeps its samples and
// channels and walks over the pixels, so that a source's per-sample and
// per-channel parameters stay in registers; the next tile's values are
// requested before the current one is converted. The up to eight channel
// blocks of a tile are one workgroup's waves; they pack their codes in LDS
// and the tile leaves as one contiguous stretch (a row's 32-byte pieces
// stored one by one reach HBM far less efficiently). Eight waves: four were 2
// to 5% faster for single tensors of 26 MB and as much slower for larger ones
// (group norm of 160 x 160 x 32 x 128 as E4M3 182 against 187 us).
// Measured at dropout of 80 x 80 x 16 x 64 as E5M2, a source of few operations:
// 33 MB in 8.3 us with its launch.
#pragma once
#include <type_traits>

#include "block_common.h"

namespace mq {

struct MxRows {
  uint8_t *codes, *scales;
  int P, N, C, nCB, bp, nPB;
  int grp;          // lane pairs of a pixel, where a tile holds several (N < 32)
  int ppt, npt;     // pixels per tile, tiles along the pixels
  int cbw, pw;      // a workgroup's channel blocks and pixel tiles (waves)
  int nslice;       // groups of cbw channel blocks
  int glanes;       // lanes that share a block
  int ny, blocks;   // workgroups along samples and channels, and along the pixels
  int extra;        // workgroups of the source's own work, before these
};

constexpr int kRowsWaves = 8;

inline MxRows mx_rows(const MxOutView& out, int P, int N, int C) {
  MxRows g{};
  g.codes = out.codes; g.scales = out.scales;
  g.P = P; g.N = N; g.C = C; g.bp = out.bp;
  g.nCB = ceil_div(C, 32); g.nPB = ceil_div(N, out.bp);
  // with fewer than 32 samples a tile holds whole pixels; squares need each
  // pixel's rows in an aligned group of lanes, a power of two of them
  g.grp = N < 32 ? N : 32;
  if (out.bp != 1)
    for (g.grp = 1; g.grp < 32 && g.grp < N;) g.grp *= 2;
  g.ppt = 32 / g.grp;
  g.npt = ceil_div(P, g.ppt);
  g.glanes = out.bp == 1 ? 2 : 2 * g.grp;
  g.cbw = g.nCB < kRowsWaves ? g.nCB : kRowsWaves;
  g.pw = kRowsWaves / g.cbw;
  if (g.pw > g.npt) g.pw = g.npt;
  g.nslice = ceil_div(g.nCB, g.cbw);
  g.ny = ceil_div(N, 32) * g.nslice;
  g.blocks = 1;  // launch_mx_rows
  return g;
}

// Src: State, what a lane keeps: where its rows are, by rows(state, n, cnt),
// and its parameters, by params(state, n, c0, cnt), where cnt (0 to 16) of
// the channels c0 .. exist and the first tile is on its way; Raw (what a lane
// reads of a pixel) by load(state, raw, p, n, c0, cnt); the 16 values, zeros
// past cnt, by values(state, raw, p, n, c0, x); extra(b, n) runs in n
// workgroups of its own.
// p, n and c0 are in range on every lane (a lane without a row or channels
// gets those of another, with cnt 0, and its values are left out).
template <int F, class Src>
__global__ __launch_bounds__(64 * kRowsWaves) void mx_rows_kernel(const Src src, const MxRows g) {
  constexpr int RB = run_bytes_of(F);
  __shared__ __attribute__((aligned(16))) uint8_t stage[2][kRowsWaves * 32 * RB];
  if ((int)blockIdx.x < g.extra) {  // the source's own work
    src.extra((int)blockIdx.x, g.extra);
    return;
  }
  // neighbouring workgroups: neighbouring rows and channels of a pixel
  const int id = (int)blockIdx.x - g.extra;
  const int xb = id / g.ny, yb = id - xb * g.ny;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nt = yb / g.nslice, slice = yb - nt * g.nslice;
  const int cb0 = slice * g.cbw, cbe = min(g.cbw, g.nCB - cb0);  // this workgroup's channel blocks
  const int pi = wave / g.cbw, cbi = wave - pi * g.cbw;
  const int r = lane >> 1, half = lane & 1;
  const int cb = cb0 + cbi, c0 = cb * 32 + half * 16;
  const int psub = r / g.grp, n = nt * 32 + r - psub * g.grp;
  const int srow = psub * g.N + (n - nt * 32);  // the tile's rows in memory order
  const bool row_ok = n < g.N && psub < g.ppt, lane_ok = row_ok && c0 < g.C && cbi < cbe;
  const int cnt = lane_ok ? min(16, g.C - c0) : 0;  // this lane's channels
  const int na = row_ok ? n : 0, ca = c0 < g.C ? c0 : 0;
  typename Src::State s;
  src.rows(s, na, cnt);
  const int pitch = cbe * RB;
  typename Src::Raw raw;
  auto pixel_of = [&](int t) { return (t + pi) * g.ppt + psub; };
  auto load = [&](int t) {
    const int p = pixel_of(t);
    const bool ok = t + pi < g.npt && p < g.P;
    src.load(s, raw, ok ? p : 0, na, ca, ok ? cnt : 0);
  };
  const int step = g.blocks * g.pw;
  int t = xb * g.pw;
  load(t);
  src.params(s, na, ca, cnt);
  for (int buf = 0; t < g.npt; t += step, buf ^= 1) {
    const int p = pixel_of(t);
    const bool ok = lane_ok && t + pi < g.npt && p < g.P;
    const typename Src::Raw cur = raw;
    load(t + step);
    float x[16];
    src.values(s, cur, p, na, ca, x);
    if (__builtin_amdgcn_ballot_w64(!ok) != 0) {  // (uniform)
#pragma unroll
      for (int i = 0; i < 16; i++) x[i] = ok ? x[i] : 0.0f;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    m = group_max(m, g.glanes);
    const uint32_t S = scale_byte_from_amax<F>(m);
    float v[16];
    scale_clamp16<F>(x, S, v);
    uint8_t* const tile = &stage[buf][pi * 32 * pitch];
    if (row_ok && cbi < cbe)
      convert_store_half_run<F>(tile + srow * pitch + cbi * RB + half * (RB / 2), v, code_keep(S));
    if (row_ok && cbi < cbe && t + pi < g.npt && p < g.P && half == 0) {
      if (g.bp == 1) g.scales[((long long)p * g.N + n) * g.nCB + cb] = (uint8_t)S;
      else if ((n & 31) == 0) g.scales[((long long)p * g.nPB + (n >> 5)) * g.nCB + cb] = (uint8_t)S;
    }
    // the tile's waves have packed their blocks (LDS only: the next tile's
    // loads stay in flight); two buffers, so the copy below and the next
    // tile's packing need no second barrier
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (t + pi < g.npt) {
      const int p0 = (t + pi) * g.ppt;
      const int rows = min(g.ppt, g.P - p0) * min(32, g.N - nt * 32);
      const long long row0 = (long long)p0 * g.N + nt * 32;
      constexpr int VW = RB % 16 == 0 ? 16 : 8;
      typedef uint32_t vw_t __attribute__((ext_vector_type(VW / 4)));
      const int sw = pitch / VW;
      uint8_t* const to = g.codes + row0 * ((long long)g.nCB * RB) + cb0 * RB;
      const int me = cbi * 64 + lane, all = g.cbw * 64;
      if (g.nslice == 1) {  // whole rows: one stretch
        for (int i = me; i < rows * sw; i += all)
          *reinterpret_cast<vw_t*>(to + i * VW) = *reinterpret_cast<const vw_t*>(tile + i * VW);
      } else {
        for (int i = me; i < rows * sw; i += all) {
          const int row = i / sw, off = i - row * sw;
          *reinterpret_cast<vw_t*>(to + (long long)row * g.nCB * RB + off * VW) =
              *reinterpret_cast<const vw_t*>(tile + i * VW);
        }
      }
    }
  }
}

// Workgroups of a kernel that the current device holds at once (1,024 if the
// runtime cannot say).
inline int resident_groups(const void* kern, int threads) {
  int occ = 0, dev = 0, cus = 0;
  if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, threads, 0) != hipSuccess ||
      hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || occ < 1 || cus < 1) {
    (void)hipGetLastError();
    return 1024;
  }
  return occ * cus;
}

template <int F, class Src>
hipError_t launch_mx_rows_f(const Src& src, MxRows g, int extra, hipStream_t st) {
  const auto kern = mx_rows_kernel<F, Src>;
  const int threads = 64 * g.cbw * g.pw;
  // as many workgroups as the chip holds at once: a source's parameters are
  // then read once a wave, and all of a wave's tiles but the first are
  // requested ahead (a workgroup for every tile: samples of 20 x 20 x 256 read
  // back into squares 13.0 instead of 11.0 us, dropout of 80 x 80 x 16 x 64
  // 9.6 instead of 8.7 us)
  static const int waves = resident_groups(reinterpret_cast<const void*>(kern), 64 * kRowsWaves) * kRowsWaves;
  const int most = ceil_div(g.npt, g.pw), fit = waves * 64 / threads / g.ny;
  g.blocks = fit < 1 ? 1 : (fit < most ? fit : most);
  g.extra = extra;
  hipLaunchKernelGGL(kern, dim3((unsigned)(g.blocks * g.ny + extra)), dim3((unsigned)threads), 0, st, src, g);
  return launch_check();
}

// extra: workgroups of the source's own work
template <class Src>
hipError_t launch_mx_rows(int fmt, const Src& src, const MxRows& g, int extra, hipStream_t st) {
  switch (fmt) {
    case 0: return launch_mx_rows_f<0>(src, g, extra, st);
    case 1: return launch_mx_rows_f<1>(src, g, extra, st);
    case 2: return launch_mx_rows_f<2>(src, g, extra, st);
    case 3: return launch_mx_rows_f<3>(src, g, extra, st);
    default: return launch_mx_rows_f<4>(src, g, extra, st);
  }
}

}  // namespace mq
