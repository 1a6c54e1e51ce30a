// cache.hip -- the replay cache: samples quantized in lines as they are
// stored, and read back as values or as a packed activation.
//
// A slot's codes and scales are contiguous (slot-major), so a sample is
// written and read in long stretches wherever its slot is; a batch interleaves
// its samples at every pixel. Everything is memory bound: each side touches
// its bytes once.
#include "block.h"
#include "mx_rows.h"

namespace mq {

// 2^(S - 127) as fp32 (2^-127 is subnormal); NaN for S = 0xFF.
__device__ __forceinline__ float scale_value(uint32_t S) {
  return __uint_as_float(S == 0u ? 0x00400000u : S == 255u ? 0x7fc00000u : S << 23);
}

// The value of the 6-bit code at bit `at` of w: sign-extended from its bit 5
// and shifted to where its magnitude is fp32 exponent and mantissa bits, with
// the copies of the sign in between masked out, then multiplied by 2^(127 -
// bias), which makes subnormal codes right too.
template <int F>
__device__ __forceinline__ float value6(uint32_t w, int at) {
  using T = Fmt<F>;
  constexpr float up = F == 2 ? 0x1p126f : 0x1p124f;  // 2^(127 - bias)
  static_assert(T::bias == (F == 2 ? 1 : 3), "exponent bias");
  const uint32_t code = (uint32_t)((int)(w << (26 - at)) >> 26);
  return __uint_as_float(code << (23 - T::M) & (0x80000000u | 31u << (23 - T::M))) * up;
}

// Values of 4 codes packed in the low 4 * bits of w, times sc.
template <int F>
__device__ __forceinline__ void values4(uint32_t w, float sc, float (&v)[4]) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  if constexpr (F <= 1) {
    v2f a, b;
    if constexpr (F == 0) {
      a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
      b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    } else {
      a = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
      b = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
    }
    v[0] = a[0] * sc; v[1] = a[1] * sc; v[2] = b[0] * sc; v[3] = b[1] * sc;
  } else if constexpr (F <= 3) {
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = value6<F>(w, 6 * i) * sc;
  } else {
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    v[0] = a[0] * sc; v[1] = a[1] * sc; v[2] = b[0] * sc; v[3] = b[1] * sc;
  }
}

// ---------------------------------------------------------------------------
// write
// ---------------------------------------------------------------------------
// One workgroup: a sample, up to eight of its channel blocks (one wave each)
// and tiles of 32 consecutive pixels, whose rows are one stretch of the slot.
// The wave's arrangement is the quantizer's (lane l: row l / 2, 16 channels).
// Bound by reading pieces of a row as long as a sample's channels: 128 samples
// of 20 x 20 x 256 as E4M3 14 to 15 us (65.9 MB, 4.5 TB/s).
struct CacheWrite {
  CacheView c;
  const float* x;
  const int32_t* slot;
  int N, n0, count, nCB, cbw, pw, nslice, npt, blocks;
};

template <int F>
__global__ __launch_bounds__(64 * kRowsWaves) void cache_write_kernel(const CacheWrite a) {
  constexpr int RB = run_bytes_of(F);
  __shared__ __attribute__((aligned(16))) uint8_t stage[2][kRowsWaves * 32 * RB];
  int id = (int)blockIdx.x;
  const int xb = id % a.blocks;
  id /= a.blocks;
  const int slice = id % a.nslice, m = id / a.nslice;
  const int slot = a.slot[m];
  // of several samples with this slot the last one is stored
  int later = 0;
  for (int i = m + 1 + (int)threadIdx.x; i < a.count; i += (int)blockDim.x) later |= a.slot[i] == slot;
  later = __syncthreads_or(later);
  if (later || slot < 0 || slot >= a.c.slots) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cb0 = slice * a.cbw, cbe = min(a.cbw, a.nCB - cb0);
  const int pi = wave / a.cbw, cbi = wave - pi * a.cbw;
  const int r = lane >> 1, half = lane & 1;
  const int cb = cb0 + cbi, c0 = cb * 32 + half * 16, C = a.c.C, P = a.c.P;
  const int cnt = cbi < cbe ? min(16, C - c0) : 0;
  const long long row0 = (long long)slot * P;
  const long long row_bytes = (long long)a.nCB * RB;
  const int pitch = cbe * RB;
  const float* const src = a.x + (long long)(a.n0 + m) * C + c0;
  const long long pstride = (long long)a.N * C;
  auto load = [&](int t, float (&x)[16]) {
    const int p = (t + pi) * 32 + r;
    load_run<16>(src + p * pstride, t + pi < a.npt && p < P ? cnt : 0, x);
  };
  const int step = a.blocks * a.pw;
  int t = xb * a.pw;
  float xn[16];
  if (t < a.npt) load(t, xn);
  for (int buf = 0; t < a.npt; t += step, buf ^= 1) {
    float x[16], v[16];
#pragma unroll
    for (int i = 0; i < 16; i++) x[i] = xn[i];
    if (t + step < a.npt) load(t + step, xn);
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) mx = max(mx, __float_as_uint(x[i]) & 0x7fffffffu);
    mx = group_max(mx, 2);
    const uint32_t S = scale_byte_from_amax<F>(mx);
    scale_clamp16<F>(x, S, v);
    uint8_t* const tile = &stage[buf][pi * 32 * pitch];
    if (cbi < cbe) convert_store_half_run<F>(tile + r * pitch + cbi * RB + half * (RB / 2), v, code_keep(S));
    const int p0 = (t + pi) * 32;
    if (half == 0 && cbi < cbe && t + pi < a.npt && p0 + r < P)
      a.c.scales[(row0 + p0 + r) * a.nCB + cb] = (uint8_t)S;
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (t + pi < a.npt) {
      const int rows = min(32, P - p0);
      constexpr int VW = RB % 16 == 0 ? 16 : 8;
      typedef uint32_t vw_t __attribute__((ext_vector_type(VW / 4)));
      const int sw = pitch / VW;
      uint8_t* const to = a.c.codes + (row0 + p0) * row_bytes + cb0 * RB;
      const int me = cbi * 64 + lane, all = a.cbw * 64;
      if (a.nslice == 1) {
        for (int i = me; i < rows * sw; i += all)
          *reinterpret_cast<vw_t*>(to + i * VW) = *reinterpret_cast<const vw_t*>(tile + i * VW);
      } else {
        for (int i = me; i < rows * sw; i += all) {
          const int row = i / sw, off = i - row * sw;
          *reinterpret_cast<vw_t*>(to + row * row_bytes + off * VW) = *reinterpret_cast<const vw_t*>(tile + i * VW);
        }
      }
    }
  }
}

hipError_t launch_cache_write(const CacheView& c, const float* x, int N, int n0, int count, const int32_t* slot,
                              hipStream_t st) {
  CacheWrite a{};
  a.c = c; a.x = x; a.slot = slot; a.N = N; a.n0 = n0; a.count = count;
  a.nCB = ceil_div(c.C, 32);
  a.cbw = a.nCB < kRowsWaves ? a.nCB : kRowsWaves;
  a.npt = ceil_div(c.P, 32);
  a.pw = kRowsWaves / a.cbw;
  if (a.pw > a.npt) a.pw = a.npt;
  a.nslice = ceil_div(a.nCB, a.cbw);
  const int most = ceil_div(a.npt, a.pw);
  int b = ceil_div(1024, (long long)count * a.nslice);
  a.blocks = b < most ? b : most;
  const dim3 grid((unsigned)(a.blocks * a.nslice * count)), wg((unsigned)(64 * a.cbw * a.pw));
  switch (c.fmt) {
    case 0: hipLaunchKernelGGL(cache_write_kernel<0>, grid, wg, 0, st, a); break;
    case 1: hipLaunchKernelGGL(cache_write_kernel<1>, grid, wg, 0, st, a); break;
    case 2: hipLaunchKernelGGL(cache_write_kernel<2>, grid, wg, 0, st, a); break;
    case 3: hipLaunchKernelGGL(cache_write_kernel<3>, grid, wg, 0, st, a); break;
    default: hipLaunchKernelGGL(cache_write_kernel<4>, grid, wg, 0, st, a); break;
  }
  return launch_check();
}

// ---------------------------------------------------------------------------
// read, values
// ---------------------------------------------------------------------------
// A thread turns four codes into one 16-byte store, so a wave's stores are
// 1 KB of consecutive bytes. A workgroup's tile is kReadPix pixels x a few
// samples: the scale bytes of a slot's neighbouring pixels share cache lines,
// which one workgroup then uses up. Bound by instructions (addresses and
// decoding issue in 72% of the busy cycles) and by loads of which only one round
// is in flight: 128 samples of 20 x 20 x 256 from E2M1 15 us (52 MB written, 7 MB
// read, 3.9 TB/s).
constexpr int kReadPix = 16, kReadUnroll = 4;
struct CacheRead {
  CacheView c;
  const int32_t* slot;
  float* x;
  int N, n0, count, nCB, NQ, mb, nmt;  // quads of a row; samples of a tile, tiles along the samples
  FastDiv dNQ, dmb;
};

template <int F>
__global__ __launch_bounds__(256) void cache_read_kernel(const CacheRead a) {
  constexpr int RB = run_bytes_of(F);
  const int pt = (int)blockIdx.x / a.nmt, mt = (int)blockIdx.x - pt * a.nmt;
  const int p0 = pt * kReadPix, pe = min(kReadPix, a.c.P - p0);
  const int m0 = mt * a.mb;
  const int total = pe * a.mb * a.NQ, C = a.c.C;
  constexpr int U = kReadUnroll;
  for (int i0 = (int)threadIdx.x; i0 < total; i0 += 256 * U) {
    uint32_t w[U], S[U];
    float* to[U];
    int cnt[U];
#pragma unroll
    for (int k = 0; k < U; k++) {
      const int i = i0 + 256 * k;
      const int row = (int)fdiv((unsigned)i, a.dNQ), q = i - row * a.NQ;
      const int pp = (int)fdiv((unsigned)row, a.dmb), m = m0 + row - pp * a.mb;
      const bool ok = i < total && m < a.count;
      const int slot = ok ? a.slot[m] : -1;
      cnt[k] = ok ? min(4, C - 4 * q) : 0;
      to[k] = a.x + ((long long)(p0 + pp) * a.N + a.n0 + m) * C + 4 * q;
      w[k] = 0;
      S[k] = 0;
      if (slot >= 0 && slot < a.c.slots) {
        const long long src = (long long)slot * a.c.P + p0 + pp;
        const uint8_t* run = a.c.codes + (src * a.nCB + (q >> 3)) * RB;
        S[k] = a.c.scales[src * a.nCB + (q >> 3)];
        const int j = q & 7;
        if constexpr (RB == 32) w[k] = reinterpret_cast<const uint32_t*>(run)[j];
        else if constexpr (RB == 16) w[k] = reinterpret_cast<const uint16_t*>(run)[j];
        else {  // 24 bits at bit 24 j: one or two dwords of the run
          const uint32_t* d = reinterpret_cast<const uint32_t*>(run);
          const int b = 24 * j, at = b >> 5;
          const uint64_t both = (uint64_t)d[min(at + 1, 5)] << 32 | d[at];
          w[k] = (uint32_t)(both >> (b & 31));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < U; k++) {
      float v[4];
      values4<F>(w[k], scale_value(S[k]), v);
      store_run<4>(to[k], cnt[k], v);
    }
  }
}

hipError_t launch_cache_read(const CacheView& c, const int32_t* slot, int count, float* x, int N, int n0,
                             hipStream_t st) {
  CacheRead a{};
  a.c = c; a.slot = slot; a.x = x; a.N = N; a.n0 = n0; a.count = count;
  a.nCB = ceil_div(c.C, 32);
  a.NQ = ceil_div(c.C, 4);
  // one round of loads for every thread (two rounds: 64 samples' worth of
  // 4-bit codes a replay batch, 20 x 20 x 128 x 256, 17 instead of 12 us)
  const int rows = 256 * kReadUnroll / a.NQ;
  a.mb = rows / kReadPix;
  if (a.mb < 1) a.mb = 1;
  if (a.mb > count) a.mb = count;
  a.nmt = ceil_div(count, a.mb);
  a.dNQ = make_fastdiv((unsigned)a.NQ);
  a.dmb = make_fastdiv((unsigned)a.mb);
  const dim3 grid((unsigned)(ceil_div(c.P, kReadPix) * a.nmt));
  switch (c.fmt) {
    case 0: hipLaunchKernelGGL(cache_read_kernel<0>, grid, dim3(256), 0, st, a); break;
    case 1: hipLaunchKernelGGL(cache_read_kernel<1>, grid, dim3(256), 0, st, a); break;
    case 2: hipLaunchKernelGGL(cache_read_kernel<2>, grid, dim3(256), 0, st, a); break;
    case 3: hipLaunchKernelGGL(cache_read_kernel<3>, grid, dim3(256), 0, st, a); break;
    default: hipLaunchKernelGGL(cache_read_kernel<4>, grid, dim3(256), 0, st, a); break;
  }
  return launch_check();
}

// ---------------------------------------------------------------------------
// read, packed activation
// ---------------------------------------------------------------------------
// The values of half a stored run are the source of the packed rows; a block
// whose lines come back with their own format and scale gets its codes back,
// because the largest code of a line lies in the format's largest binade (or
// the line's scale byte is 0, and its values' too). Bound by decoding and
// encoding, whose instructions issue in 84% of the busy cycles: 128 samples of
// 20 x 20 x 256 from E3M2 to E4M3 squares 11 us (23 MB).
template <int FI, bool FULL>
struct CacheSrc {
  CacheView c;
  const int32_t* slot;
  int nCB;
  struct State {
    long long row0;  // first row of the sample's slot (of slot 0 where there is none)
    bool ok;
  };
  struct Raw {
    uint32_t w[FI <= 1 ? 4 : FI <= 3 ? 3 : 2], S;
  };
  __device__ void params(State&, int, int, int) const {}
  __device__ void rows(State& s, int n, int cnt) const {
    const int k = cnt > 0 ? slot[n] : -1;
    s.ok = k >= 0 && k < c.slots;
    s.row0 = s.ok ? (long long)k * c.P : 0;
  }
  __device__ void load(const State& s, Raw& r, int p, int, int c0, int) const {
    constexpr int NW = sizeof(r.w) / 4, RB = run_bytes_of(FI);
    const long long run = (s.row0 + p) * nCB + (c0 >> 5);
    const uint32_t* d = reinterpret_cast<const uint32_t*>(c.codes + run * RB + ((c0 >> 4) & 1) * (RB / 2));
#pragma unroll
    for (int i = 0; i < NW; i++) r.w[i] = d[i];
    r.S = c.scales[run];
  }
  // (no slot: codes 0 with scale byte 0)
  __device__ void words(const State& s, const Raw& r, uint32_t (&w)[4], uint32_t& S) const {
    S = s.ok ? r.S : 0u;
    uint32_t a[sizeof(r.w) / 4];
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.w) / 4); i++) a[i] = s.ok ? r.w[i] : 0u;
    if constexpr (FI <= 1) {
#pragma unroll
      for (int i = 0; i < 4; i++) w[i] = a[i];
    } else if constexpr (FI <= 3) {
      w[0] = a[0];
      w[1] = a[0] >> 24 | a[1] << 8;
      w[2] = a[1] >> 16 | a[2] << 16;
      w[3] = a[2] >> 8;
    } else {
      w[0] = a[0]; w[1] = a[0] >> 16;
      w[2] = a[1]; w[3] = a[1] >> 16;
    }
  }
  __device__ void values(const State& s, const Raw& r, int, int, int c0, float (&v)[16]) const {
    uint32_t w[4], S;  // four codes each
    words(s, r, w, S);
    const float sc = scale_value(S);
    const int cnt = c.C - c0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float q[4];
      values4<FI>(w[i], sc, q);
#pragma unroll
      for (int j = 0; j < 4; j++) v[4 * i + j] = FULL || 4 * i + j < cnt ? q[j] : 0.0f;
    }
  }
  __device__ void extra(int, int) const {}
};

namespace {
template <bool FULL>
hipError_t launch_read_mx(const CacheView& c, const int32_t* slot, const MxRows& g, int fmt, hipStream_t st) {
  const int nCB = ceil_div(c.C, 32);
  switch (c.fmt) {
    case 0: return launch_mx_rows(fmt, CacheSrc<0, FULL>{c, slot, nCB}, g, 0, st);
    case 1: return launch_mx_rows(fmt, CacheSrc<1, FULL>{c, slot, nCB}, g, 0, st);
    case 2: return launch_mx_rows(fmt, CacheSrc<2, FULL>{c, slot, nCB}, g, 0, st);
    case 3: return launch_mx_rows(fmt, CacheSrc<3, FULL>{c, slot, nCB}, g, 0, st);
    default: return launch_mx_rows(fmt, CacheSrc<4, FULL>{c, slot, nCB}, g, 0, st);
  }
}
}  // namespace

hipError_t launch_cache_read_mx(const CacheView& c, const int32_t* slot, int N, const MxOutView& out, hipStream_t st) {
  const MxRows g = mx_rows(out, c.P, N, c.C);
  return c.C % 16 == 0 ? launch_read_mx<true>(c, slot, g, out.fmt, st) : launch_read_mx<false>(c, slot, g, out.fmt, st);
}

}  // namespace mq
