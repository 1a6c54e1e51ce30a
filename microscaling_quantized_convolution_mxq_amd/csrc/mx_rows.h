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
// stored one by one reach HBM far less efficiently).
#pragma once
#include <type_traits>

#include "block_common.h"

namespace mq {

struct MxRows {
  uint8_t *codes, *scales;
  int P, N, C, nCB, bp, nPB;
  int ppt, npt;     // pixels per tile, tiles along the pixels
  int cbw, pw;      // a workgroup's channel blocks and pixel tiles (waves)
  int nslice;       // groups of cbw channel blocks
  int glanes;       // lanes that share a block
  int ny, blocks;   // workgroups along samples and channels, and along the pixels
};

constexpr int kRowsWaves = 8;

inline MxRows mx_rows(const MxOutView& out, int P, int N, int C) {
  MxRows g{};
  g.codes = out.codes; g.scales = out.scales;
  g.P = P; g.N = N; g.C = C; g.bp = out.bp;
  g.nCB = ceil_div(C, 32); g.nPB = ceil_div(N, out.bp);
  // with fewer than 32 samples a tile holds whole pixels; squares need their
  // rows in aligned groups of lanes, hence a power of two
  const bool pack = N < 32 && (out.bp == 1 || 32 % N == 0);
  g.ppt = pack ? 32 / N : 1;
  g.npt = ceil_div(P, g.ppt);
  g.glanes = out.bp == 1 ? 2 : (pack ? 2 * N : 64);
  g.cbw = g.nCB < kRowsWaves ? g.nCB : kRowsWaves;
  g.pw = kRowsWaves / g.cbw;
  if (g.pw > g.npt) g.pw = g.npt;
  g.nslice = ceil_div(g.nCB, g.cbw);
  g.ny = ceil_div(N, 32) * g.nslice;
  // about four workgroups per compute unit, each walking over the pixels
  int b = ceil_div(1024, g.ny);
  const int most = ceil_div(g.npt, g.pw);
  g.blocks = b < most ? b : most;
  return g;
}

template <int F, class Src>
__global__ __launch_bounds__(64 * kRowsWaves) void mx_rows_kernel(const Src src, const MxRows g) {
  constexpr int RB = run_bytes_of(F);
  __shared__ __attribute__((aligned(16))) uint8_t stage[2][kRowsWaves * 32 * RB];
  // neighbouring workgroups: neighbouring rows and channels of a pixel
  const int xb = (int)blockIdx.x / g.ny, yb = (int)blockIdx.x - xb * g.ny;
  if (xb >= g.blocks) {  // the source's own work
    src.extra((int)blockIdx.x - g.blocks * g.ny);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nt = yb / g.nslice, slice = yb - nt * g.nslice;
  const int cb0 = slice * g.cbw, cbe = min(g.cbw, g.nCB - cb0);  // this workgroup's channel blocks
  const int pi = wave / g.cbw, cbi = wave - pi * g.cbw;
  const int r = lane >> 1, half = lane & 1;
  const int cb = cb0 + cbi, c0 = cb * 32 + half * 16;
  int psub = 0, n = nt * 32 + r;
  if (g.N < 32) {
    psub = r / g.N;
    n = r - psub * g.N;
  }
  const bool lane_ok = n < g.N && psub < g.ppt && cbi < cbe;
  const int cnt = lane_ok ? min(16, g.C - c0) : 0;  // this lane's channels
  typename Src::State s;
  src.init(s, n, c0, cnt);
  const int pitch = cbe * RB;
  typename Src::Raw raw;
  auto pixel_of = [&](int t) { return (t + pi) * g.ppt + psub; };
  auto load = [&](int t) {
    const int p = pixel_of(t);
    const bool ok = t + pi < g.npt && p < g.P;
    src.load(s, raw, p, n, c0, ok ? cnt : 0);
  };
  const int step = g.blocks * g.pw;
  int t = xb * g.pw;
  if (t < g.npt) load(t);
  for (int buf = 0; t < g.npt; t += step, buf ^= 1) {
    const int p = pixel_of(t);
    const bool ok = lane_ok && t + pi < g.npt && p < g.P;
    float x[16];
    src.values(s, raw, p, n, c0, x);
    if (t + step < g.npt) load(t + step);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    m = group_max(m, g.glanes);
    const uint32_t S = scale_byte_from_amax<F>(m);
    float v[16];
    scale_clamp16<F>(x, S, v);
    uint8_t* const tile = &stage[buf][pi * 32 * pitch];
    if (cbi < cbe) convert_store_half_run<F>(tile + r * pitch + cbi * RB + half * (RB / 2), v, code_keep(S));
    if (ok && half == 0) {
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
      const int rows = g.N < 32 ? min(g.ppt, g.P - p0) * g.N : min(32, g.N - nt * 32);
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

// extra: workgroups of the source's own work behind the rows'
template <class Src>
hipError_t launch_mx_rows(int fmt, const Src& src, const MxRows& g, int extra, hipStream_t st) {
  const dim3 grid((unsigned)(g.blocks * g.ny + extra));
  const dim3 wg((unsigned)(64 * g.cbw * g.pw));
  switch (fmt) {
    case 0: hipLaunchKernelGGL((mx_rows_kernel<0, Src>), grid, wg, 0, st, src, g); break;
    case 1: hipLaunchKernelGGL((mx_rows_kernel<1, Src>), grid, wg, 0, st, src, g); break;
    case 2: hipLaunchKernelGGL((mx_rows_kernel<2, Src>), grid, wg, 0, st, src, g); break;
    case 3: hipLaunchKernelGGL((mx_rows_kernel<3, Src>), grid, wg, 0, st, src, g); break;
    default: hipLaunchKernelGGL((mx_rows_kernel<4, Src>), grid, wg, 0, st, src, g); break;
  }
  return launch_check();
}

}  // namespace mq
