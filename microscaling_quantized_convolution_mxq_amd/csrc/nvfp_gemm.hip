// nvfp_gemm.hip -- the three products of a convolution on two-level codes.
//
// An operand's value is q B T: element code, E4M3 scale of its 8 x 8 block,
// fp32 scale of the tensor. q B has at most 8 significant bits in every format
// (E4M3 and E2M3 elements 4, times 4 of the scale), so it is a bf16 exactly,
// and the products q B q' B' are exact in the bf16 matrix units; T T' multiplies
// the sums. A block of 8 x 8 has one scale for 8 values along either product's
// k, where the block-scaled matrix instructions take a power of two for 32, so
// values are made first:
//   1. both operands are written as bf16 with k contiguous, channels (weight
//      gradient: samples) padded with zeros;
//   2. a product gathers rows of 128 bytes (64 values of k) from them: of the
//      pixel that a tap reaches, or past the end of the buffer, which reads as
//      zeros, outside the image.
//   forward:   Y[(ho wo n)][co] = sum over (kh kw ci) of X[..] W[co][..]
//   data:      dX[(h w n)][ci] = sum over (kh kw co) of dY[..] W'[ci][..], the
//              rows in classes of equal (h mod stride, w mod stride), which
//              have the same taps
//   weight:    dW[co][(kh kw ci)] = sum over (ho wo n) of dY'[co][..] X'[ci][..]
//              with the operands transposed in step 1
// Few tiles with long sums are split along k into slices, whose sums a last
// kernel adds in a fixed order.
#include <math.h>

#include <algorithm>

#include "mma_core.h"
#include "mx_rows.h"
#include "train.h"

namespace mq {

namespace {

typedef float v2f __attribute__((ext_vector_type(2)));

// ---- values of codes ----------------------------------------------------------------------------
// Eight neighbouring codes, 32, 48 or 64 bits in two words, as floats.
template <int F>
__device__ __forceinline__ void decode8_words(uint32_t lo, uint32_t hi, float (&v)[8]) {
  if constexpr (Fmt<F>::bits == 8) {
    const uint32_t u[2] = {lo, hi};
#pragma unroll
    for (int i = 0; i < 2; i++) {
      v2f a, b;
      if constexpr (F == 0) {
        a = __builtin_amdgcn_cvt_pk_f32_fp8(u[i], false);
        b = __builtin_amdgcn_cvt_pk_f32_fp8(u[i], true);
      } else {
        a = __builtin_amdgcn_cvt_pk_f32_bf8(u[i], false);
        b = __builtin_amdgcn_cvt_pk_f32_bf8(u[i], true);
      }
      v[4 * i] = a[0]; v[4 * i + 1] = a[1]; v[4 * i + 2] = b[0]; v[4 * i + 3] = b[1];
    }
  } else if constexpr (Fmt<F>::bits == 6) {
    const uint64_t w = (uint64_t)lo | (uint64_t)hi << 32;
    // magnitude bits as the top of an fp32's: its exponent is off by 127 - bias, subnormals included
    constexpr float up = __builtin_bit_cast(float, (uint32_t)(254 - Fmt<F>::bias) << 23);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t c = (uint32_t)(w >> (6 * i));
      v[i] = __uint_as_float((c & 31u) << (23 - Fmt<F>::M) | (c & 32u) << 26) * up;
    }
  } else {
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.0f, 1),
              c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.0f, 3);
    v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1]; v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
  }
}
// The same from memory.
template <int F>
__device__ __forceinline__ void decode8(const uint8_t* p, float (&v)[8]) {
  if constexpr (Fmt<F>::bits == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    decode8_words<F>(w.x, w.y, v);
  } else if constexpr (Fmt<F>::bits == 6) {
    const uint16_t* const h = reinterpret_cast<const uint16_t*>(p);
    decode8_words<F>((uint32_t)h[0] | (uint32_t)h[1] << 16, h[2], v);
  } else {
    decode8_words<F>(*reinterpret_cast<const uint32_t*>(p), 0, v);
  }
}

// An operand as the quantizer wrote it: an [A][P][B] x C view, P the partner index.
struct Codes {
  const uint8_t *codes, *scales;
  int fmt, A, P, B, C;
  int rbytes, nPB, nCB;  // bytes of a row's codes; blocks along P and C
};

Codes codes_of(const NvfpView& t, int A, int P, int B, int C) {
  return Codes{t.codes, t.scales, t.fmt, A, P, B, C, (int)row_bytes(t.fmt, C), ceil_div(P, 8), ceil_div(C, 8)};
}

typedef unsigned short bits8 __attribute__((ext_vector_type(8)));  // eight 16-bit values

// Channels 8 ch .. 8 ch + 7 of row (ab, p) as bf16, or as f16 (which holds 4-bit elements times their scales too, 6 bits from
// 2^-10 to 2688); zeros past C.
template <int F>
__device__ __forceinline__ bits8 values8(const Codes& t, bool half, long long row, int ab, int p, int ch) {
  float v[8];
  const int c0 = 8 * ch;
  if (c0 < t.C) {
    decode8<F>(t.codes + row * t.rbytes + (c0 >> 5) * run_bytes_of(F) + (c0 & 31) * Fmt<F>::bits / 8, v);
    const float s = __builtin_amdgcn_cvt_f32_fp8(t.scales[((long long)ab * t.nPB + (p >> 3)) * t.nCB + ch], 0);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = c0 + i < t.C ? v[i] * s : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = 0.0f;
  }
  if (half) {
    half8 o;
#pragma unroll
    for (int i = 0; i < 8; i++) o[i] = (_Float16)v[i];
    return __builtin_bit_cast(bits8, o);
  }
  bhalf8 o;
#pragma unroll
  for (int i = 0; i < 8; i++) o[i] = (__bf16)v[i];
  return __builtin_bit_cast(bits8, o);
}

// f(the format as a constant); the format is the same for a whole workgroup
template <class L>
__host__ __device__ __forceinline__ void by_format(int fmt, L&& f) {
  switch (fmt) {
    case 0: f(std::integral_constant<int, 0>{}); break;
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 3: f(std::integral_constant<int, 3>{}); break;
    default: f(std::integral_constant<int, 4>{}); break;
  }
}

// An operand as 16-bit values, either
//   out[row][Cp], Cp a multiple of 64: 8 channels a thread, or
//   out[c][ab][Pp], Pp a multiple of 8: tiles of 64 channels x 64 of the (ab, p).
struct Task {
  Codes t;
  __bf16* out;
  bool across, half;     // half: f16 instead of bf16
  int groups;            // workgroups
  int n;                 // pieces of 8 channels
  FastDiv pieces, dP, dB;
  int Pp, S, tiles;      // S = A B Pp; tiles along S
  FastDiv dPp;
};

constexpr int kPieces = 2;  // of a thread, their loads together (8192 x 4096 and 4096 x 4096, 127 MB: 31.8 us, 37.1 with one)
template <int F>
__device__ __forceinline__ void make_rows(const Task& a, int group) {
  bits8 v[kPieces];
  long long to[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; u++) {
    const unsigned i = (unsigned)(group * kPieces + u) * 256u + threadIdx.x, j = min(i, (unsigned)a.n - 1);
    const unsigned row = fdiv(j, a.pieces), ch = j - row * a.pieces.d;
    const unsigned q = fdiv(row, a.dB), b = row - q * a.dB.d, aa = fdiv(q, a.dP), p = q - aa * a.dP.d;
    to[u] = i < (unsigned)a.n ? (long long)i * 8 : -1;
    v[u] = values8<F>(a.t, a.half, row, (int)(aa * a.dB.d + b), (int)p, (int)ch);
  }
#pragma unroll
  for (int u = 0; u < kPieces; u++)
    if (to[u] >= 0) *reinterpret_cast<bits8*>(a.out + to[u]) = v[u];
}

constexpr int kAcross = 66;  // a column of the tile (eight threads of one slot write 8 channels each, 264 dwords apart: eight banks)
template <int F>
__device__ __forceinline__ void make_across(const Task& a, int group, unsigned short* tile) {
  const int ct = group / a.tiles, s0 = (group - ct * a.tiles) * 64, c0 = ct * 64;
#pragma unroll
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int ch = i & 7, slot = i >> 3, s = s0 + slot;
    bits8 v = {0, 0, 0, 0, 0, 0, 0, 0};
    if (s < a.S) {
      const unsigned ab = fdiv((unsigned)s, a.dPp), p = (unsigned)s - ab * a.dPp.d;
      if ((int)p < a.t.P) {
        const unsigned aa = fdiv(ab, a.dB), b = ab - aa * a.dB.d;
        v = values8<F>(a.t, a.half, ((long long)aa * a.t.P + p) * a.dB.d + b, (int)ab, (int)p, (c0 >> 3) + ch);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; e++) tile[(8 * ch + e) * kAcross + slot] = v[e];
  }
  __syncthreads();
#pragma unroll
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int k = i & 7, c = i >> 3, s = s0 + 8 * k;
    if (c0 + c >= a.t.C || s >= a.S) continue;
    const uint32_t* const from = reinterpret_cast<const uint32_t*>(tile + c * kAcross + 8 * k);
    *reinterpret_cast<uint4*>(a.out + (long long)(c0 + c) * a.S + s) = make_uint4(from[0], from[1], from[2], from[3]);
  }
}

// Both operands in one launch.
__global__ __launch_bounds__(256) void nvfp_values_kernel(const Task a, const Task b) {
  __shared__ __attribute__((aligned(16))) unsigned short tile[64 * kAcross];
  const bool first = (int)blockIdx.x < a.groups;
  const Task& t = first ? a : b;
  const int group = first ? (int)blockIdx.x : (int)blockIdx.x - a.groups;
  by_format(t.t.fmt, [&](auto f) {
    constexpr int F = decltype(f)::value;
    if (t.across) make_across<F>(t, group, tile);
    else make_rows<F>(t, group);
  });
}

long long up(long long v, int m) { return (v + m - 1) / m * m; }

Task rows_task(const Codes& t, __bf16* out) {
  const int cp = (int)up(t.C, 64);
  Task a{};
  a.t = t; a.out = out;
  a.n = (int)((long long)t.A * t.P * t.B * (cp / 8));
  a.groups = ceil_div(a.n, 256 * kPieces);
  a.pieces = make_fastdiv(cp / 8); a.dP = make_fastdiv(t.P); a.dB = make_fastdiv(t.B);
  return a;
}
Task across_task(const Codes& t, __bf16* out, int pad) {
  Task a{};
  a.t = t; a.out = out; a.across = true;
  a.Pp = (int)up(t.P, pad);
  a.S = t.A * t.B * a.Pp;
  a.tiles = ceil_div(a.S, 64);
  a.groups = a.tiles * ceil_div(t.C, 64);
  a.dPp = make_fastdiv((unsigned)a.Pp); a.dB = make_fastdiv(t.B);
  return a;
}
hipError_t launch_values(const Task& a, const Task& b, hipStream_t st) {
  hipLaunchKernelGGL(nvfp_values_kernel, dim3((unsigned)(a.groups + b.groups)), dim3(256), 0, st, a, b);
  return launch_check();
}

// ---- products -----------------------------------------------------------------------------------
// A value that all lanes share, in a scalar register (quotients are computed in
// vector ones, and a load's address from those is a loop over its values).
__device__ __forceinline__ int shared(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Rows of an image of pixels, each the channels (64 cb) of a pixel's sample, moved by the taps of a step. Output row (r, c, n)
// starts at pixel (r sr + r0, c sc + c0), and tap (i, j) is at (+-i, +-j) from there.
struct Gather {
  const __bf16* p;
  long long bytes;
  int H, W, N, row;      // row: bytes of a row (pixel and sample)
  int Wr, M;             // columns of the output's pixels, output rows
  int sr, sc, r0, c0, dir;
  FastDiv dN, dW;
};
// The steps of a sum over taps (i, j) and blocks of 64 channels; the other operand's rows have taps (k0 + s i) KW + l0 + s j.
struct Taps {
  int ni, nj, nc;  // taps, and blocks of 64 channels
  int k0, l0, si, sj, KW;
};

template <int L, int NW>
struct GatherLoader {
  static_assert(NW % 2 == 0, "one chunk a lane");
  __amdgpu_buffer_rsrc_t rsrc;
  int off[L], h[L], w[L];
  int H, W, pix, dir, nj, nc, i, j, cb;
  __device__ void init(const Gather& g, const Taps& t, int row0, int step0, int wave, int lane) {
    rsrc = mma_rsrc(g.p, g.bytes);
    H = g.H; W = g.W; pix = g.N * g.row; dir = g.dir; nj = t.nj; nc = t.nc;
    const int tap = step0 / t.nc;
    cb = step0 - tap * t.nc; i = tap / t.nj; j = tap - i * t.nj;
#pragma unroll
    for (int k = 0; k < L; k++) {
      const int m = row0 + lane_row<NW>(wave, lane, k);
      const unsigned px = fdiv((unsigned)m, g.dN), n = (unsigned)m - px * g.dN.d, r = fdiv(px, g.dW), c = px - r * g.dW.d;
      h[k] = (int)r * g.sr + g.r0;
      w[k] = (int)c * g.sc + g.c0;
      off[k] = (int)(((unsigned)(h[k] * g.W + w[k]) * (unsigned)g.N + n) * (unsigned)g.row) + lane_chunk(wave, lane) * 16;
      if (m >= g.M) h[k] = -(1 << 20);  // (no tap leads back into the image from there)
    }
  }
  // (steps are asked for in order)
  __device__ void issue(int, uint8_t* lds, int wave) {
    const int di = dir * i, dj = dir * j, move = (di * W + dj) * pix;
#pragma unroll
    for (int k = 0; k < L; k++) {
      const bool in = (unsigned)(h[k] + di) < (unsigned)H && (unsigned)(w[k] + dj) < (unsigned)W;
      load_lds16(rsrc, lds + (wave + NW * k) * 1024, in ? off[k] + move : kBeyond, cb * kPiece);
    }
    if (++cb == nc) {
      cb = 0;
      if (++j == nj) { j = 0; i++; }
    }
  }
};

template <int L, int NW>
struct TapLoader {
  RowLoader<L, NW> rows;
  int nj, nc, i, j, cb;
  Taps t;
  __device__ void init(const void* p, long long bytes, int row0, int n, int pitch, const Taps& taps, int step0, int wave, int lane) {
    rows.init(p, bytes, row0, n, pitch, wave, lane);
    t = taps;
    const int tap = shared(step0 / t.nc);
    cb = step0 - tap * t.nc; i = shared(tap / t.nj); j = tap - i * t.nj;
  }
  __device__ void issue(int, uint8_t* lds, int wave) {
    rows.issue(shared(((t.k0 + t.si * i) * t.KW + t.l0 + t.sj * j) * t.nc + cb), lds, wave);
    if (++cb == t.nc) {
      cb = 0;
      if (++j == t.nj) { j = 0; i++; }
    }
  }
};

// dY' [co][pixel][Np]: rows of `pieces` 16-byte pieces, which need not end with a step
template <int L, int NW>
struct EndLoader {
  static_assert(NW % 2 == 0, "one chunk a lane");
  RowLoader<L, NW> rows;
  int pieces, chunk;
  __device__ void init(const void* p, long long bytes, int row0, int n, int count, int wave, int lane) {
    rows.init(p, bytes, row0, n, count * 16, wave, lane);
    pieces = count;
    chunk = lane_chunk(wave, lane);
  }
  __device__ void issue(int step, uint8_t* lds, int wave) const {
    const bool in = step * 8 + chunk < pieces;
#pragma unroll
    for (int j = 0; j < L; j++)
      load_lds16(rows.rsrc, lds + (wave + NW * j) * 1024, in ? rows.off[j] : kBeyond, step * kPiece);
  }
};

// X' [ci][H][W][Np] for the columns (kh, kw, ci) of dW: piece q of the sum is samples 8 n8 .. of output pixel q / (Np / 8)
struct Shift {
  const __bf16* p;
  long long bytes;
  int H, W, Cin, KW, Np, sr, sc, pr, pc;
  int cols, pieces;  // columns of dW; pieces of a sum
  FastDiv dC, dK, dN, dW;  // by Cin, KW, Np / 8 and Wo
};
template <int L, int NW>
struct ShiftLoader {
  static_assert(NW % 2 == 0, "one chunk a lane");
  __amdgpu_buffer_rsrc_t rsrc;
  int off[L], h[L], w[L], chunk;
  const Shift* s;
  __device__ void init(const Shift& g, int col0, int wave, int lane) {
    rsrc = mma_rsrc(g.p, g.bytes);
    s = &g;
    chunk = lane_chunk(wave, lane);
#pragma unroll
    for (int k = 0; k < L; k++) {
      const int col = col0 + lane_row<NW>(wave, lane, k);
      const unsigned tap = fdiv((unsigned)col, g.dC), ci = (unsigned)col - tap * g.dC.d, kh = fdiv(tap, g.dK), kw = tap - kh * g.dK.d;
      h[k] = (int)kh - g.pr;
      w[k] = (int)kw - g.pc;
      off[k] = (int)((unsigned)(((int)ci * g.H + h[k]) * g.W + w[k]) * (unsigned)(g.Np * 2));
      if (col >= g.cols) h[k] = -(1 << 20);
    }
  }
  __device__ void issue(int step, uint8_t* lds, int wave) const {
    const unsigned q = step * 8 + chunk, px = fdiv(q, s->dN), n8 = q - px * s->dN.d, r = fdiv(px, s->dW), c = px - r * s->dW.d;
    const int w0 = (int)c * s->sc, h0 = (int)q < s->pieces ? (int)r * s->sr : -(1 << 20);
    const int at = (int)((r * (unsigned)(s->sr * s->W) + (unsigned)w0) * (unsigned)(s->Np * 2) + n8 * 16u);
#pragma unroll
    for (int k = 0; k < L; k++) {
      const bool in = (unsigned)(h[k] + h0) < (unsigned)s->H && (unsigned)(w[k] + w0) < (unsigned)s->W;
      load_lds16(rsrc, lds + (wave + NW * k) * 1024, in ? off[k] + at : kBeyond, 0);
    }
  }
};

// Sums times the tensors' scales: the product of the two in fp64 as a mantissa and a power of two, as it may leave fp32's range.
struct Scale {
  float m;
  int e;
  __device__ float operator()(float v) const { return ldexpf(v * m, e); }
};
__device__ __forceinline__ Scale scale_of(const float* a, const float* b) {
  Scale s;
  s.m = (float)frexp((double)*a * (double)*b, &s.e);
  return s;
}

struct Class {
  Gather g;
  Taps t;
  int h0, w0;  // its pixels are (r sh + h0, c sw + w0)
  int tiles;
};
constexpr int kClasses = 8;  // of a launch

struct ConvArgs {
  const __bf16* b;
  long long b_bytes;
  int b_pitch, cols;  // bytes of a row of the other operand; its rows, the output's columns
  float* out;         // or the slices
  const float *ta, *tb;
  int slices, tiles;
  long long slice;    // values of a slice
  int sh, sw, W, N;   // where a class's rows are in the output
  int nclass;
  bool classes;       // rows go by classes (backward data)
  // the gathered operand's codes, for the kernel that makes its values itself
  const uint8_t *codes, *scales;
  long long codes_bytes, scales_bytes;
  int rbytes, runs, nPB, nCB;  // bytes and 32-channel runs of a row, blocks along samples and channels
  Class k[kClasses];
};

// A wave's results through LDS, 32 rows at a time, to whole pieces of rows: `rows` has the tile's rows in the output (-1: none).
template <class S, int MOST = 2>
__device__ __forceinline__ void store_results(float* strips, const int* rows, v16f (&acc)[S::TM][S::TN], const MmaWave<S>& me,
                                              const Scale& scale, float* out, int cols, int j0) {
  constexpr int TJ = S::TN < MOST ? S::TN : MOST, WIDE = TJ * 32, PITCH = WIDE + 8;  // (rows r and r + 4 are written together: the other half of the banks)
  static_assert(S::TN % TJ == 0, "strips");
  const int lane = me.lane, wm = me.wave / S::WN, wn = me.wave % S::WN;
  float* const strip = strips + me.wave * 32 * PITCH;
  constexpr int LPR = WIDE / 4, RPI = 64 / LPR;  // lanes of a row, rows of a store
  const int c = (lane % LPR) * 4;
#pragma unroll
  for (int i = 0; i < S::TM; i++)
#pragma unroll
    for (int j0t = 0; j0t < S::TN; j0t += TJ) {
      const int col = j0 + wn * S::TN * 32 + j0t * 32 + c;
#pragma unroll
      for (int j = 0; j < TJ; j++)
#pragma unroll
        for (int e = 0; e < 16; e++)
          strip[(8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * PITCH + j * 32 + (lane & 31)] = scale(acc[i][j0t + j][e]);
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the strip is written (one wave's)
      asm volatile("" ::: "memory");
#pragma unroll
      for (int r = 0; r < 32; r += RPI) {
        const int rr = r + lane / LPR;
        const int row = rows[(wm * S::TM + i) * 32 + rr];
        const f4u v = *reinterpret_cast<const f4u*>(strip + rr * PITCH + c);
        if (row < 0 || col >= cols) continue;
        float* const to = out + (long long)row * cols + col;
        if (col + 4 <= cols) {
          __builtin_nontemporal_store(v, reinterpret_cast<f4u*>(to));
        } else {
#pragma unroll
          for (int e = 0; e < 3; e++)
            if (col + e < cols) to[e] = v[e];
        }
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);  // (and read, before the next one)
      asm volatile("" ::: "memory");
    }
}

template <class S>
constexpr int strips_of() {  // bytes of the strips; the tile's rows are behind them
  constexpr int n = S::NW * 32 * ((S::TN < 2 ? 1 : 2) * 32 + 8) * 4;
  static_assert(n + S::BM * 4 <= S::LDS, "the strips and the rows take the ring's place");
  return n;
}
// The output's rows of a tile's rows.
template <class S>
__device__ __forceinline__ void fill_rows(const ConvArgs& a, const Class& k, int i0, int* rows) {
  for (int r = threadIdx.x; r < S::BM; r += S::THREADS) {
    const int m = i0 + r;
    int row = m < k.g.M ? m : -1;
    if (a.classes && row >= 0) {
      const unsigned px = fdiv((unsigned)m, k.g.dN), n = (unsigned)m - px * k.g.dN.d, pr = fdiv(px, k.g.dW), pc = px - pr * k.g.dW.d;
      row = (((int)pr * a.sh + k.h0) * a.W + (int)pc * a.sw + k.w0) * a.N + (int)n;
    }
    rows[r] = row;
  }
}
template <class S>
constexpr bool wide_of() {
  return S::TM * S::TN >= 8 && S::NW == 4;
}
template <class S>
constexpr int waves_of() {  // a SIMD's, for the register budget
  return wide_of<S>() ? 1 : 2;
}

template <class S>
__global__ __launch_bounds__(S::THREADS, waves_of<S>()) void nvfp_conv_kernel(const ConvArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  const MmaWave<S> me;
  const int lane = me.lane, wave = me.wave;
  const int b = xcd_tile(blockIdx.x, gridDim.x), z = b / a.tiles, at = b - z * a.tiles;
  // the classes of one place side by side: they read the same rows, and every XCD has as many of the long sums
  const int tile = at / a.nclass;
  const Class& k = a.k[at - tile * a.nclass];
  if (tile >= k.tiles) return;
  const int tn = (a.cols + S::BN - 1) / S::BN;
  const int ti = tile / tn, i0 = ti * S::BM, j0 = (tile - ti * tn) * S::BN;
  const int steps = k.t.ni * k.t.nj * k.t.nc, s0 = (int)((long long)steps * z / a.slices),
            s1 = (int)((long long)steps * (z + 1) / a.slices);
  v16f acc[S::TM][S::TN];
  mma_zero<S>(acc);
  if (s1 > s0) {
    GatherLoader<S::LA, S::NW> la;
    TapLoader<S::LB, S::NW> lb;
    la.init(k.g, k.t, i0, s0, wave, lane);
    lb.init(a.b, a.b_bytes, j0, a.cols, a.b_pitch, k.t, s0, wave, lane);
    if constexpr (wide_of<S>()) mma_loop_wide<Bf16, S>(lds, la, lb, s0, s1 - s0, me, acc);
    else mma_loop<Bf16, S>(lds, la, lb, s0, s1 - s0, s1 - s0, me, acc);
  }
  stage_ready<0>();  // the ring is free
  int* const rows = reinterpret_cast<int*>(lds + strips_of<S>());
  fill_rows<S>(a, k, i0, rows);
  __syncthreads();
  Scale scale{1.0f, 0};
  if (a.slices == 1) scale = scale_of(a.ta, a.tb);
  store_results<S>(reinterpret_cast<float*>(lds), rows, acc, me, scale, a.out + (a.slices == 1 ? 0 : z * a.slice), a.cols, j0);
}

// ---- the same from codes ------------------------------------------------------------------------
// The gathered operand stays in codes as far as the registers of the wave that
// multiplies them, a quarter (4 bit) or half of the bytes through L2 and LDS,
// and no pass over it before. A step is two runs of 32 channels of every row; a
// lane takes a run of its row (its eight 16-byte pieces of 8 channels are the
// products' k, which both operands may take in any order) with the run's four
// block scales in one dword, and makes 8 values with 16 instructions while the
// other waves multiply. Each wave has all columns, so no value is made twice in
// a workgroup. The other operand, small, comes as bf16.
// Codes are read from LDS as vectors: for a struct the compiler waits until
// every load is done, those of later steps too.
// The input gradient of 3 x 3, stride 2 (160 x 160 x 32 x 128 from 80 x 80 x 32 x
// 256, E2M1): 149 us once the clock has settled (140 at the least, 190 to 207 for
// some milliseconds after the first calls), 288 by the kernel above with its pass over
// both; a call with the weights' pass 154, of E5M2 by E4M3 168. Its products alone
// are 84 us at the rate of a large matrix product, its stores 79 at a copy's: at two
// waves a SIMD (registers for the sums) they overlap by half.
// 3 x 3 on 80 x 80 x 16 x 64 to 64 channels: 18.7 us (19.2 and a pass of 6.4 by the
// kernel above, here 4.0), of which 10 remain with one step of the nine; with
// tiles of 128 rows the same.
template <int F>
struct CodeRows {
  static constexpr int RUN = run_bytes_of(F), SLOTS = 2 * RUN / 16;  // 16-byte slots of a row: 2 (4 bit) or 4 (8 bit)
  static constexpr int ROW = 16 * SLOTS;
  // a row's slots are permuted so that sixteen rows' reads of one slot lie in different banks
  __device__ static int swizzle(int row) { return SLOTS == 2 ? (row >> 3) & 1 : (row >> 2) & 3; }
};

template <int BM_, int BN_, int ST_, int F>
struct CodeShape : MmaShape<BM_, BN_, 4, 1, ST_> {
  typedef MmaShape<BM_, BN_, 4, 1, ST_> Base;
  static constexpr int SCALES = BM_ * CodeRows<F>::ROW, OTHER = SCALES + BM_ * 8;  // offsets in a stage
  static constexpr int STAGE = OTHER + BN_ * kPiece, LDS = ST_ * STAGE;
  static constexpr int LC = BM_ * CodeRows<F>::SLOTS / 64 / 4, LS = BM_ * 2 / 64 / 4, LB = Base::LB;  // loads of a wave: codes, scales, others
};

__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, uint8_t* lds, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (mma_lds_t)lds, 4, voff, soff, 0, 0);
}

template <int F, int LC, int LS, int SCALES>
struct CodeLoader {
  typedef CodeRows<F> R;
  __amdgpu_buffer_rsrc_t codes, scales;
  int coff[LC], ch[LC], cw[LC], soff[LS], sh[LS], sw[LS];
  int H, W, cpix, spix, dir, nj, nc, i, j, cb, crun[LC], runs, nCB;
  __device__ void init(const ConvArgs& a, const Gather& g, const Taps& t, int row0, int step0, int wave, int lane) {
    H = g.H; W = g.W; dir = g.dir; nj = t.nj; nc = t.nc;
    cpix = g.N * a.rbytes; spix = a.nPB * a.nCB; runs = a.runs; nCB = a.nCB;
    const int tap = shared(step0 / t.nc);
    cb = step0 - tap * t.nc; i = shared(tap / t.nj); j = tap - i * t.nj;
    auto place = [&](int m, int& h, int& w, unsigned& n) {
      const unsigned px = fdiv((unsigned)m, g.dN), r = fdiv(px, g.dW), c = px - r * g.dW.d;
      n = (unsigned)m - px * g.dN.d;
      h = (int)r * g.sr + g.r0;
      w = (int)c * g.sc + g.c0;
    };
#pragma unroll
    for (int k = 0; k < LC; k++) {
      const int local = (wave + 4 * k) * (64 / R::SLOTS) + lane / R::SLOTS, m = row0 + local;
      const int slot = (lane % R::SLOTS) ^ R::swizzle(local);
      unsigned n;
      place(m, ch[k], cw[k], n);
      crun[k] = slot * 16 / R::RUN;
      coff[k] = (int)((unsigned)(ch[k] * g.W + cw[k]) * (unsigned)cpix + n * (unsigned)a.rbytes) + slot * 16;
      if (m >= g.M) ch[k] = -(1 << 20);
    }
#pragma unroll
    for (int k = 0; k < LS; k++) {
      const int m = row0 + (wave + 4 * k) * 32 + (lane >> 1);
      unsigned n;
      place(m, sh[k], sw[k], n);
      soff[k] = (int)((unsigned)(sh[k] * g.W + sw[k]) * (unsigned)spix + (n >> 3) * (unsigned)a.nCB) + (lane & 1) * 4;
      if (m >= g.M) sh[k] = -(1 << 20);
    }
  }
  // (steps are asked for in order)
  __device__ void issue(uint8_t* lds, int wave, int lane) {
    const int di = dir * i, dj = dir * j, at = di * W + dj, cmove = at * cpix, smove = at * spix;
#pragma unroll
    for (int k = 0; k < LC; k++) {
      const bool in = (unsigned)(ch[k] + di) < (unsigned)H && (unsigned)(cw[k] + dj) < (unsigned)W && 2 * cb + crun[k] < runs;
      load_lds16(codes, lds + (wave + 4 * k) * 1024, in ? coff[k] + cmove : kBeyond, shared(cb * 2 * R::RUN));
    }
#pragma unroll
    for (int k = 0; k < LS; k++) {
      const bool in = (unsigned)(sh[k] + di) < (unsigned)H && (unsigned)(sw[k] + dj) < (unsigned)W && 8 * cb + (lane & 1) * 4 < nCB;
      load_lds4(scales, lds + SCALES + (wave + 4 * k) * 256, in ? soff[k] + smove : kBeyond, shared(cb * 8));
    }
    if (++cb == nc) {
      cb = 0;
      if (++j == nj) { j = 0; i++; }
    }
  }
};

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Eight values of piece kk of a run: words `w` of the run's codes, the four
// scales in `s`. As f16, 4-bit elements take 4 conversions and 4 packed
// products; as bf16, whose products have no packed form, twice as many.
template <int F>
__device__ __forceinline__ half8 piece_values(const uint32_t* w, uint32_t s, int kk, half8) {
  static_assert(F == 4, "4-bit elements");
  const uint32_t c = w[kk];
  const half2v two = kk < 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s, 1.0f, false) : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s, 1.0f, true);
  const half2v f = {two[kk & 1], two[kk & 1]};
  const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 0) * f, b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 1) * f,
               d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 2) * f, e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 3) * f;
  return half8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}
template <int F>
__device__ __forceinline__ bhalf8 piece_values(const uint32_t* w, uint32_t s, int kk, bhalf8) {
  float v[8];
  if constexpr (F == 4) {
    const uint32_t c = w[kk];
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1),
              d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1]; v[4] = d[0]; v[5] = d[1]; v[6] = e[0]; v[7] = e[1];
  } else {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const uint32_t c = w[2 * kk + h];
      const v2f a = F == 0 ? __builtin_amdgcn_cvt_pk_f32_fp8(c, false) : __builtin_amdgcn_cvt_pk_f32_bf8(c, false),
                b = F == 0 ? __builtin_amdgcn_cvt_pk_f32_fp8(c, true) : __builtin_amdgcn_cvt_pk_f32_bf8(c, true);
      v[4 * h] = a[0]; v[4 * h + 1] = a[1]; v[4 * h + 2] = b[0]; v[4 * h + 3] = b[1];
    }
  }
  float f;
  switch (kk) {  // (a constant where this is called)
    case 0: f = __builtin_amdgcn_cvt_f32_fp8(s, 0); break;
    case 1: f = __builtin_amdgcn_cvt_f32_fp8(s, 1); break;
    case 2: f = __builtin_amdgcn_cvt_f32_fp8(s, 2); break;
    default: f = __builtin_amdgcn_cvt_f32_fp8(s, 3); break;
  }
  bhalf8 o;
#pragma unroll
  for (int e = 0; e < 8; e++) o[e] = (__bf16)(v[e] * f);
  return o;
}

// Tiles t of a launch for a workgroup that takes several: each XCD has a contiguous range of them.
struct TileWalk {
  int at, end, step;
  __device__ explicit TileWalk(int total) {
    const int x = blockIdx.x & 7, q = total >> 3, r = total & 7;
    at = x * q + min(x, r);
    end = at + q + (x < r ? 1 : 0);
    at += blockIdx.x >> 3;
    step = ((int)gridDim.x + 7 - x) >> 3;
  }
};

// Workgroups stay and walk over the tiles: one for each left the chip half
// empty, as sums are short (a workgroup of four waves lived 20 us, and a place
// waited as long for the next). The first loads of a tile are under way while
// the results of the one before are stored, from the end of the ring.
__device__ __forceinline__ v16f multiply(half8 x, half8 y, v16f c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, c, 0, 0, 0); }
__device__ __forceinline__ v16f multiply(bhalf8 x, bhalf8 y, v16f c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, c, 0, 0, 0); }

template <class S, int F, class V>
__global__ __launch_bounds__(256, 2) void nvfp_codes_kernel(const ConvArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  typedef CodeRows<F> R;
  constexpr int ST = S::ST, TM = S::TM, TN = S::TN, LPS = S::LC + S::LS + S::LB;
  constexpr int STRIPS = 4 * 32 * 40 * 4, KEPT = STRIPS + S::BM * 4;  // strips of 32 columns, and the tile's rows
  constexpr int FREE = (S::LDS - KEPT) / S::STAGE, PRE = FREE < ST - 1 ? FREE : ST - 1;
  static_assert(PRE >= 1, "a stage beside the strips");
  constexpr int STORES = TM * TN * 4;  // of a wave with a whole tile
  int held = 0;  // steps of the present tile whose loads stand before such stores
  float* const strips = reinterpret_cast<float*>(lds + S::LDS - KEPT);
  int* const rows = reinterpret_cast<int*>(lds + S::LDS - S::BM * 4);
  const MmaWave<S> me;
  const int lane = me.lane, wave = me.wave;
  const int r = lane & 31, q = lane >> 5, sw = (r >> 1) & 7;
  const int tn = (a.cols + S::BN - 1) / S::BN;
  Scale scale{1.0f, 0};
  if (a.slices == 1) scale = scale_of(a.ta, a.tb);

  TileWalk walk(a.tiles * a.slices);
  CodeLoader<F, S::LC, S::LS, S::SCALES> la;
  RowLoader<S::LB, 4> lb;
  int first = 0, down = 0, right = 0;  // the other operand's row of a step: (first + i down + j right) nc + cb
  int which = 0, i0 = 0, j0 = 0, z = 0, n = 0;
  const __amdgpu_buffer_rsrc_t codes = mma_rsrc(a.codes, a.codes_bytes), scales = mma_rsrc(a.scales, a.scales_bytes),
                               other = mma_rsrc(a.b, a.b_bytes);
  auto issue = [&](int slot) {
    uint8_t* const to = lds + shared(slot * S::STAGE);
    la.codes = codes; la.scales = scales; lb.rsrc = other;  // (the same for all tiles)
    lb.issue(shared((first + la.i * down + la.j * right) * la.nc + la.cb), to + S::OTHER, wave);
    la.issue(to, wave, lane);
  };
  // the next tile and its first loads; false: there is none
  auto next = [&]() {
    for (; walk.at < walk.end; walk.at += walk.step) {
      z = shared(walk.at / a.tiles);
      const int at = walk.at - z * a.tiles, tile = shared(at / a.nclass);
      // (turned from place to place, or a workgroup whose step is a multiple of their number would always meet the same class)
      which = shared((at + tile + (tile >> 4)) % a.nclass);
      const Class& k = a.k[which];
      if (tile >= k.tiles) continue;
      const int ti = shared(tile / tn), steps = k.t.ni * k.t.nj * k.t.nc, s0 = shared((int)((long long)steps * z / a.slices));
      i0 = ti * S::BM;
      j0 = (tile - ti * tn) * S::BN;
      n = shared((int)((long long)steps * (z + 1) / a.slices)) - s0;
      if (n > 0) {
        la.init(a, k.g, k.t, i0, s0, wave, lane);
        lb.init(a.b, a.b_bytes, j0, a.cols, a.b_pitch, wave, lane);
        first = k.t.k0 * k.t.KW + k.t.l0; down = k.t.si * k.t.KW; right = k.t.sj;
#pragma unroll
        for (int s = 0; s < PRE; s++)
          if (s < n) issue(s);
      }
      walk.at += walk.step;
      return true;
    }
    return false;
  };

  bool more = next();
  while (more) {
    v16f acc[TM][TN];
    mma_zero<S>(acc);
#pragma unroll
    for (int s = PRE; s < ST - 1; s++)
      if (s < n) issue(s);
    int slot = 0, fill = ST - 1;
    for (int s = 0; s < n; s++) {
      if (s + ST - 2 >= n) stage_ready<0>();
      else if (s < held) stage_ready<(ST - 2) * LPS + STORES>();
      else stage_ready<(ST - 2) * LPS>();
      if (s + ST - 1 < n) issue(fill);
      const uint8_t* const from = lds + slot * S::STAGE;
      uint32_t w[TM][R::RUN / 4], sc[TM];
#pragma unroll
      for (int i = 0; i < TM; i++) {
        const int row = (wave * TM + i) * 32 + r;
#pragma unroll
        for (int h = 0; h < R::RUN / 16; h++)
          *reinterpret_cast<u32x4*>(&w[i][4 * h]) =
              *reinterpret_cast<const u32x4*>(from + row * R::ROW + (((q * (R::RUN / 16) + h) ^ R::swizzle(row)) << 4));
        sc[i] = *reinterpret_cast<const uint32_t*>(from + S::SCALES + row * 8 + q * 4);
      }
#pragma unroll
      for (int kk = 0; kk < 4; kk++) {
        V x[TM], y[TN];
#pragma unroll
        for (int j = 0; j < TN; j++)
          y[j] = *reinterpret_cast<const V*>(from + S::OTHER + (32 * j + r) * kPiece + (((4 * q + kk) ^ sw) << 4));
#pragma unroll
        for (int i = 0; i < TM; i++) x[i] = piece_values<F>(w[i], sc[i], kk, V{});
#pragma unroll
        for (int i = 0; i < TM; i++)
#pragma unroll
          for (int j = 0; j < TN; j++) acc[i][j] = multiply(x[i], y[j], acc[i][j]);
      }
      slot = slot + 1 == ST ? 0 : slot + 1;
      fill = fill + 1 == ST ? 0 : fill + 1;
    }
    stage_ready<0>();  // the ring is free
    fill_rows<S>(a, a.k[which], i0, rows);
    float* const out = a.out + (a.slices == 1 ? 0 : z * a.slice);
    const int c0 = j0;
    // Where every lane stores, every wave does so STORES times, and the stages asked for before that are waited for with the
    // stores under way.
    held = i0 + S::BM <= a.k[which].g.M && j0 + S::BN <= a.cols ? PRE : 0;
    more = next();
    lds_ready();  // the rows are known
    store_results<S, 1>(strips, rows, acc, me, scale, out, a.cols, c0);
    if (PRE < ST - 1) lds_ready();  // (the strips are read: loads may go there)
  }
}

// ---- a linear layer for a few rows --------------------------------------------------------------
// Y[n][co] for up to 8 samples, bound by reading W's codes once: no values are
// written, no matrix units (a tile of 64 rows would be empty). A lane takes the
// same run of 32 channels of R rows of W and of every sample; the products of
// the codes' own values (exact in fp32) are summed over a block's 8 channels and
// then take the two block scales, so a scale costs an eighth of a product. The
// four rows lie in one block of 8 along Cout, so they share the scales, and all
// samples lie in one along N. Waves of a workgroup share the channels between
// them where these are many.
// 4096 x 4096 E2M1 at one sample: 5.1 us on the device (8.9 MB of codes and
// scales, 1.75 TB/s: one round of loads, so their latency) against 12.7 through
// the tiles, whose values of W alone are 33.5 MB written and read. A call with its
// host part is 9.2 us at 1 and 2 samples, 9.6 at 4 and 14.6 at 8, through the
// tiles 25 us at any of them.
// Operands of two formats take it at one sample only: to decode the second by a
// switch in the loop over samples needs more registers than there are.
constexpr int kRowR = 4;

// A run's 32 codes in registers.
template <int F>
struct Run {
  static constexpr int WORDS = run_bytes_of(F) / 4;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < WORDS; i += 2) *reinterpret_cast<uint2*>(w + i) = *reinterpret_cast<const uint2*>(p + 4 * i);
  }
  // the values of block b's eight codes
  __device__ __forceinline__ void values(int b, float (&v)[8]) const {
    if constexpr (Fmt<F>::bits == 8) decode8_words<F>(w[2 * b], w[2 * b + 1], v);
    else if constexpr (Fmt<F>::bits == 4) decode8_words<F>(w[b], 0, v);
    else if (b & 1) decode8_words<F>(w[3 * (b / 2) + 1] >> 16 | w[3 * (b / 2) + 2] << 16, w[3 * (b / 2) + 2] >> 16, v);
    else decode8_words<F>(w[3 * (b / 2)], w[3 * (b / 2) + 1] & 0xffffu, v);
  }
};

// SAME: both operands have the format FW (else x's is looked up, and M is 1).
template <int FW, bool SAME, int M>
__global__ __launch_bounds__(256, M == 8 ? 2 : 4) void nvfp_few_rows_kernel(const Codes x, const Codes w, const float* ta, const float* tb,
                                                                float* y, int N, int cols, int along) {
  __shared__ float sums[4][M][kRowR];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % along, co0 = (blockIdx.x * (4 / along) + wave / along) * kRowR;
  const int runs = (w.C + 31) / 32;
  float acc[M][kRowR];
#pragma unroll
  for (int m = 0; m < M; m++)
#pragma unroll
    for (int r = 0; r < kRowR; r++) acc[m][r] = 0;
  for (int run = part * 64 + lane; run < runs && co0 < cols; run += 64 * along) {
    Run<FW> wr[kRowR], xr[SAME ? M : 1];
#pragma unroll
    for (int r = 0; r < kRowR; r++) wr[r].load(w.codes + (long long)min(co0 + r, cols - 1) * w.rbytes + run * run_bytes_of(FW));
    if constexpr (SAME)
#pragma unroll
      for (int m = 0; m < M; m++) xr[m].load(x.codes + (long long)min(m, N - 1) * x.rbytes + run * run_bytes_of(FW));
    float s[4];
#pragma unroll
    for (int b = 0; b < 4; b++) {  // the run's blocks (the last run may have fewer)
      const bool in = 4 * run + b < w.nCB;
      const int at = in ? 4 * run + b : 0;
      s[b] = __builtin_amdgcn_cvt_f32_fp8(w.scales[(long long)(co0 >> 3) * w.nCB + at], 0) *
             __builtin_amdgcn_cvt_f32_fp8(x.scales[at], 0);
      s[b] = in ? s[b] : 0.0f;
    }
#pragma unroll
    for (int b = 0; b < 4; b++) {
      float v[kRowR][8];
#pragma unroll
      for (int r = 0; r < kRowR; r++) wr[r].values(b, v[r]);
#pragma unroll
      for (int m = 0; m < M; m++) {
        float u[8];
        if constexpr (SAME) {
          xr[m].values(b, u);
        } else {
          by_format(x.fmt, [&](auto f) {
            constexpr int F = decltype(f)::value;
            decode8<F>(x.codes + (long long)min(m, N - 1) * x.rbytes + run * run_bytes_of(F) + b * Fmt<F>::bits, u);
          });
        }
#pragma unroll
        for (int r = 0; r < kRowR; r++) {
          float d = u[0] * v[r][0];
#pragma unroll
          for (int e = 1; e < 8; e++) d = __builtin_fmaf(u[e], v[r][e], d);
          acc[m][r] = __builtin_fmaf(d, s[b], acc[m][r]);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < M; m++)
#pragma unroll
    for (int r = 0; r < kRowR; r++) {
#pragma unroll
      for (int off = 1; off < 64; off *= 2) acc[m][r] += __shfl_xor(acc[m][r], off);
      if (lane == 0) sums[wave][m][r] = acc[m][r];
    }
  __syncthreads();
  if (part != 0 || lane >= M * kRowR) return;
  const int m = lane / kRowR, r = lane % kRowR;
  if (m >= N || co0 + r >= cols) return;
  float s = sums[wave][m][r];
  for (int k = 1; k < along; k++) s += sums[wave + k][m][r];
  const Scale scale = scale_of(ta, tb);
  y[(long long)m * cols + co0 + r] = scale(s);
}

struct WeightArgs {
  const __bf16* dy;
  long long dy_bytes;
  Shift x;
  int rows;
  float* out;
  const float *ta, *tb;
  int slices, tiles, steps;
  long long slice;
};

// dW: the sums run over output pixels and samples, so both operands come with
// those contiguous (X' moved by a tap's pixels, as whole pieces of 8 samples).
// Bound by the loop: 62 us for 60 GFLOP (975 TFLOP/s) at 3 x 3 x 256 to 256
// channels on 20 x 20 x 128, of it about 7 for the slices' 33 MB; the operands'
// pass before is 17 us (65 MB) and the join behind 8.
template <class S>
__global__ __launch_bounds__(S::THREADS, 2) void nvfp_weight_kernel(const WeightArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  const MmaWave<S> me;
  const int lane = me.lane, wave = me.wave;
  const int b = xcd_tile(blockIdx.x, gridDim.x), z = b / a.tiles, tile = b - z * a.tiles;
  const int tn = (a.x.cols + S::BN - 1) / S::BN;
  const int ti = tile / tn, i0 = ti * S::BM, j0 = (tile - ti * tn) * S::BN;
  const int s0 = (int)((long long)a.steps * z / a.slices), s1 = (int)((long long)a.steps * (z + 1) / a.slices);
  v16f acc[S::TM][S::TN];
  mma_zero<S>(acc);
  EndLoader<S::LA, S::NW> la;
  ShiftLoader<S::LB, S::NW> lb;
  la.init(a.dy, a.dy_bytes, i0, a.rows, a.x.pieces, wave, lane);
  lb.init(a.x, j0, wave, lane);
  mma_loop<Bf16, S>(lds, la, lb, s0, s1 - s0, s1 - s0, me, acc);
  stage_ready<0>();
  int* const rows = reinterpret_cast<int*>(lds + strips_of<S>());
  for (int r = threadIdx.x; r < S::BM; r += S::THREADS) rows[r] = i0 + r < a.rows ? i0 + r : -1;
  __syncthreads();
  Scale scale{1.0f, 0};
  if (a.slices == 1) scale = scale_of(a.ta, a.tb);
  store_results<S>(reinterpret_cast<float*>(lds), rows, acc, me, scale, a.out + (a.slices == 1 ? 0 : z * a.slice), a.x.cols, j0);
}

// The slices' sums, added in order (fp64), times the tensors' scales: bound by
// the slices' bytes, with four of a thread's loads under way.
template <class V>
__global__ __launch_bounds__(256) void nvfp_join_kernel(const V* part, V* out, long long n, int slices, const float* ta, const float* tb) {
  constexpr int PER = sizeof(V) / 4;
  const Scale scale = scale_of(ta, tb);
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    double s[PER] = {};
    auto add = [&](const V& v) {
#pragma unroll
      for (int e = 0; e < PER; e++) s[e] += reinterpret_cast<const float*>(&v)[e];
    };
    int z = 0;
    for (; z + 4 <= slices; z += 4) {
      V v[4];
#pragma unroll
      for (int k = 0; k < 4; k++) v[k] = part[(z + k) * n + i];
#pragma unroll
      for (int k = 0; k < 4; k++) add(v[k]);
    }
    for (; z < slices; z++) add(part[z * n + i]);
    V o;
#pragma unroll
    for (int e = 0; e < PER; e++) reinterpret_cast<float*>(&o)[e] = scale((float)s[e]);
    out[i] = o;
  }
}

// ---- plans --------------------------------------------------------------------------------------
typedef MmaShape<256, 256, 2, 2, 2> Big;
typedef MmaShape<128, 128, 2, 2, 2> Mid;
typedef MmaShape<256, 64, 4, 1, 2> Tall;
typedef MmaShape<64, 64, 2, 2, 3> Small;
enum { kBig, kMid, kTall, kSmall };

// Tiles by the output's extents, and slices along k where these tiles do not
// fill the chip. Large ones read less and multiply at a better rate, as long as
// there are tiles for most compute units:
//   8192 x 4096 x 4096: 240 us (1145 TFLOP/s) in tiles of 256 x 256, 286 of 128 x 128;
//   dW of 3 x 3 x 256 from 20 x 20 x 128 x 256 (256 x 2304, sums of 51200): 62 us
//   in tiles of 128 x 128 by 14 slices, 129 of 64 x 64; 256 x 128 the same as 128 x 128;
//   3 x 3 on 80 x 80 x 16 x 64 to 64 channels: 19.2 us in tiles of 256 x 64, 22.4 of 64 x 64.
struct Plan {
  int shape, slices;
};
const int kBM[4] = {256, 128, 256, 64}, kBN[4] = {256, 128, 64, 64};
Plan plan_of(int op, long long M, long long N, long long steps) {
  auto tiles = [&](int s) { return (long long)ceil_div(M, kBM[s]) * ceil_div(N, kBN[s]); };
  Plan p{kSmall, 1};
  if (op < 2 && N > 128 && M > 128 && tiles(kBig) >= 200) p.shape = kBig;
  else if (N <= 64 && M >= 256 && tiles(kTall) >= 200) p.shape = kTall;
  else if (N > 64 && M > 64 && tiles(kMid) * std::max(1LL, steps / 8) >= 256) p.shape = kMid;
  const long long want = 512 / std::max(1LL, tiles(p.shape));
  // slices of eight steps at least, and no more sums than operands' bytes by far
  if (want >= 2) p.slices = (int)std::max(1LL, std::min({want, steps / 8, 64LL}));
  return p;
}

template <int OP, class F>
void with_shape(int s, F&& f) {
  switch (s) {
    case kBig:
      if constexpr (OP < 2) f(Big{});  // (the weight gradient's loader leaves no registers for it)
      break;
    case kMid: f(Mid{}); break;
    case kTall: f(Tall{}); break;
    default: f(Small{}); break;
  }
}

// The kernel that takes codes: 4- and 8-bit elements whose rows of scales are
// whole dwords, at most two tiles of columns (a value is made for each), and
// rows enough for its tall tiles (figures of both kernels are at this one). 0
// slices: the other kernel.
int code_slices(int op, int fmt, long long M, long long cols, int channels, long long steps) {
  if (op > 1 || (fmt > 1 && fmt != 4) || cols > 256 || ceil_div(channels, 8) % 4 != 0 || M < 4096) return 0;
  const long long t = (long long)ceil_div(M, 256) * ceil_div(cols, cols <= 64 ? 64 : 128);
  return (int)std::max(1LL, std::min({512 / std::max(1LL, t), steps / 8, 64LL}));
}
template <class F>
void with_code_shape(int fmt, bool half, bool narrow, F&& f) {
  auto both = [&](auto fm, auto v) {
    constexpr int E = decltype(fm)::value, ST = E == 4 ? 3 : 2;
    if (narrow) f(CodeShape<256, 64, ST, E>{}, fm, v);
    else f(CodeShape<256, 128, ST, E>{}, fm, v);
  };
  if (fmt == 0) both(std::integral_constant<int, 0>{}, bhalf8{});
  else if (fmt == 1) both(std::integral_constant<int, 1>{}, bhalf8{});
  else if (half) both(std::integral_constant<int, 4>{}, half8{});
  else both(std::integral_constant<int, 4>{}, bhalf8{});
}

struct Sizes {
  long long a, b, part;  // bytes of the operands and the slices
  Plan plan;
  int code_slices;
};

// the longest sum of a class of rows
int class_taps(int k, int stride) { return ceil_div(k, stride); }

Sizes sizes_of(const Conv& c, int op, int fa) {
  const long long ho = c.ho(), wo = c.wo(), taps = (long long)c.kh * c.kw;
  Sizes s{};
  long long out;
  if (op == 0) {
    const long long cp = up(c.cin, 64);
    s.a = (long long)c.h * c.w * c.n * cp * 2;
    s.b = c.cout * taps * cp * 2;
    s.plan = plan_of(op, ho * wo * c.n, c.cout, taps * (cp / 64));
    s.code_slices = code_slices(op, fa, ho * wo * c.n, c.cout, c.cin, taps * (cp / 64));
    out = ho * wo * c.n * c.cout;
  } else if (op == 1) {
    const long long kp = up(c.cout, 64);
    s.a = ho * wo * c.n * kp * 2;
    s.b = c.cin * taps * kp * 2;
    const long long steps = (long long)class_taps(c.kh, c.sh) * class_taps(c.kw, c.sw) * (kp / 64);
    s.plan = plan_of(op, (long long)c.h * c.w * c.n, c.cin, steps);
    s.code_slices = code_slices(op, fa, (long long)c.h * c.w * c.n, c.cin, c.cout, steps);
    out = (long long)c.h * c.w * c.n * c.cin;
  } else {
    const long long np = up(c.n, 8);
    s.a = c.cout * ho * wo * np * 2;
    s.b = (long long)c.cin * c.h * c.w * np * 2;
    s.plan = plan_of(op, c.cout, taps * c.cin, (ho * wo * np + 63) / 64);
    out = c.cout * taps * c.cin;
  }
  const int slices = std::max(s.plan.slices, s.code_slices);
  s.part = slices > 1 ? out * 4 * slices : 0;
  return s;
}

}  // namespace

bool nvfp_gemm_ok(const Conv& c, int op) {
  const Sizes s = sizes_of(c, op, 2);
  return s.a < kBeyond && s.b < kBeyond;
}

size_t nvfp_gemm_workspace_bytes(const Conv& c, int op, int fa) {
  const Sizes s = sizes_of(c, op, fa);
  return (size_t)(up(s.a, 256) + up(s.b, 256) + s.part);
}

static hipError_t join(int slices, const float* part, float* out, long long n, const float* ta, const float* tb, hipStream_t st) {
  if (slices == 1) return hipSuccess;
  const auto go = [&](auto kern, auto v, long long count) {
    typedef decltype(v) V;
    hipLaunchKernelGGL(kern, dim3((unsigned)std::min<long long>(ceil_div(count, 256), 4096)), dim3(256), 0, st,
                       reinterpret_cast<const V*>(part), reinterpret_cast<V*>(out), count, slices, ta, tb);
  };
  if (n % 2 == 0 && (uintptr_t)out % 8 == 0) go(nvfp_join_kernel<float2>, float2{}, n / 2);
  else go(nvfp_join_kernel<float>, 0.0f, n);
  return launch_check();
}

// Bytes at any address to whole dwords.
__global__ __launch_bounds__(256) void nvfp_align_kernel(const uint8_t* from, uint32_t* to, int n) {
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
    const uint8_t* const p = from + 4 * (long long)i;
    to[i] = (uint32_t)p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16 | (uint32_t)p[3] << 24;
  }
}

// The gathered operand's codes where their kernel takes them, a rule on sizes and formats alone, so that no result depends on
// an address: scales that start between dwords are copied first, to `spare`, the place of the 16-bit values that this kernel
// does without (16 bytes for each scale's at least; rows of scales are whole dwords).
static hipError_t use_codes(ConvArgs& a, const Sizes& s, const Codes& t, void* spare, hipStream_t st, bool& codes) {
  codes = s.code_slices != 0;
  if (!codes) return hipSuccess;
  a.codes = t.codes; a.scales = t.scales;
  const long long pixels = (long long)t.A * t.B;
  a.codes_bytes = pixels * t.P * t.rbytes; a.scales_bytes = pixels * t.nPB * t.nCB;
  a.rbytes = t.rbytes; a.runs = ceil_div(t.C, 32); a.nPB = t.nPB; a.nCB = t.nCB;
  if (((uintptr_t)t.scales & 3u) == 0) return hipSuccess;
  a.scales = static_cast<const uint8_t*>(spare);
  const int n = (int)(a.scales_bytes / 4);
  hipLaunchKernelGGL(nvfp_align_kernel, dim3((unsigned)std::min(ceil_div(n, 256), 2048)), dim3(256), 0, st, t.scales,
                     static_cast<uint32_t*>(spare), n);
  return launch_check();
}

template <int OP>
static hipError_t launch_tiles(const ConvArgs& a, const Sizes& s, int fmt, bool half, hipStream_t st) {
  const dim3 grid((unsigned)(a.tiles * a.slices));
  if (a.codes)
    with_code_shape(fmt, half, a.cols <= 64, [&](auto shape, auto f, auto v) {
      const auto kern = nvfp_codes_kernel<decltype(shape), decltype(f)::value, decltype(v)>;
      static const int resident = resident_groups(reinterpret_cast<const void*>(kern), 256) / 8 * 8;
      hipLaunchKernelGGL(kern, dim3((unsigned)std::min(a.tiles * a.slices, std::max(8, resident))), dim3(256), 0, st, a);
    });
  else
    with_shape<OP>(s.plan.shape, [&](auto shape) {
      typedef decltype(shape) S;
      hipLaunchKernelGGL(nvfp_conv_kernel<S>, grid, dim3(S::THREADS), 0, st, a);
    });
  return launch_check();
}
static int tiles_for(const ConvArgs& a, const Sizes& s, int M) {
  if (a.codes) return ceil_div(M, 256) * ceil_div(a.cols, a.cols <= 64 ? 64 : 128);
  return ceil_div(M, kBM[s.plan.shape]) * ceil_div(a.cols, kBN[s.plan.shape]);
}

// Whether the kernel for a few rows takes it: a linear layer.
static bool few_rows(const Conv& c, bool same) {
  return c.n <= (same ? 8 : 1) && c.h == 1 && c.w == 1 && c.kh == 1 && c.kw == 1;
}

static hipError_t launch_few_rows(const Conv& c, const NvfpView& x, const NvfpView& w, float* y, hipStream_t st) {
  const Codes xc = codes_of(x, 1, c.n, 1, c.cin), wc = codes_of(w, 1, c.cout, 1, c.cin);
  const int pieces = ceil_div(c.cin, 2048), along = pieces >= 4 ? 4 : (pieces >= 2 ? 2 : 1);
  const dim3 grid((unsigned)ceil_div(c.cout, kRowR * (4 / along)));
  by_format(w.fmt, [&](auto f) {
    constexpr int F = decltype(f)::value;
    const auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, xc, wc, x.tensor, w.tensor, y, c.n, c.cout, along);
    };
    if (x.fmt != w.fmt) go(nvfp_few_rows_kernel<F, false, 1>);
    else if (c.n == 1) go(nvfp_few_rows_kernel<F, true, 1>);
    else if (c.n == 2) go(nvfp_few_rows_kernel<F, true, 2>);
    else if (c.n <= 4) go(nvfp_few_rows_kernel<F, true, 4>);
    else go(nvfp_few_rows_kernel<F, true, 8>);
  });
  return launch_check();
}

hipError_t launch_nvfp_forward(const Conv& c, const NvfpView& x, const NvfpView& w, float* y, void* ws, hipStream_t st) {
  if (few_rows(c, x.fmt == w.fmt)) return launch_few_rows(c, x, w, y, st);
  const Sizes s = sizes_of(c, 0, x.fmt);
  const int cp = (int)up(c.cin, 64), taps = c.kh * c.kw, ho = c.ho(), wo = c.wo();
  __bf16* const xb = static_cast<__bf16*>(ws);
  __bf16* const wb = reinterpret_cast<__bf16*>(static_cast<char*>(ws) + up(s.a, 256));
  float* const part = reinterpret_cast<float*>(static_cast<char*>(ws) + up(s.a, 256) + up(s.b, 256));
  ConvArgs a{};
  const Codes xc = codes_of(x, c.h * c.w, c.n, 1, c.cin);
  bool codes;
  hipError_t e = use_codes(a, s, xc, xb, st, codes);
  if (e != hipSuccess) return e;
  const bool half = codes && x.fmt == 4 && w.fmt == 4;
  Task wt = rows_task(codes_of(w, 1, c.cout, taps, c.cin), wb);
  wt.half = half;
  e = launch_values(wt, codes ? Task{} : rows_task(xc, xb), st);
  if (e != hipSuccess) return e;
  a.b = wb; a.b_bytes = s.b; a.b_pitch = taps * cp * 2; a.cols = c.cout;
  a.slices = codes ? s.code_slices : s.plan.slices; a.slice = (long long)ho * wo * c.n * c.cout;
  a.out = a.slices > 1 ? part : y;
  a.ta = x.tensor; a.tb = w.tensor;
  a.nclass = 1;
  Class& k = a.k[0];
  k.g = Gather{xb, s.a, c.h, c.w, c.n, cp * 2, wo, ho * wo * c.n, c.sh, c.sw, -c.ph, -c.pw, 1, make_fastdiv(c.n), make_fastdiv(wo)};
  k.t = Taps{c.kh, c.kw, cp / 64, 0, 0, 1, 1, c.kw};
  k.tiles = a.tiles = tiles_for(a, s, k.g.M);
  if ((e = launch_tiles<0>(a, s, x.fmt, half, st)) != hipSuccess) return e;
  return join(a.slices, part, y, a.slice, a.ta, a.tb, st);
}

hipError_t launch_nvfp_backward_data(const Conv& c, const NvfpView& dy, const NvfpView& w, float* dx, void* ws, hipStream_t st) {
  const Sizes s = sizes_of(c, 1, dy.fmt);
  const int kp = (int)up(c.cout, 64), taps = c.kh * c.kw, ho = c.ho(), wo = c.wo();
  __bf16* const yb = static_cast<__bf16*>(ws);
  __bf16* const wb = reinterpret_cast<__bf16*>(static_cast<char*>(ws) + up(s.a, 256));
  float* const part = reinterpret_cast<float*>(static_cast<char*>(ws) + up(s.a, 256) + up(s.b, 256));
  ConvArgs a{};
  const Codes yc = codes_of(dy, ho * wo, c.n, 1, c.cout);
  bool codes;
  hipError_t e = use_codes(a, s, yc, yb, st, codes);
  if (e != hipSuccess) return e;
  const bool half = codes && dy.fmt == 4 && w.fmt == 4;
  Task wt = across_task(codes_of(w, 1, c.cout, taps, c.cin), wb, 64);
  wt.half = half;
  e = launch_values(wt, codes ? Task{} : rows_task(yc, yb), st);
  if (e != hipSuccess) return e;
  a.b = wb; a.b_bytes = s.b; a.b_pitch = taps * kp * 2; a.cols = c.cin;
  a.slices = codes ? s.code_slices : s.plan.slices; a.slice = (long long)c.h * c.w * c.n * c.cin;
  a.out = a.slices > 1 ? part : dx;
  a.ta = dy.tensor; a.tb = w.tensor;
  a.sh = c.sh; a.sw = c.sw; a.W = c.w; a.N = c.n;
  a.classes = c.sh > 1 || c.sw > 1;
  const int nh = std::min(c.sh, c.h), nw = std::min(c.sw, c.w);
  int most = 0;
  for (int q = 0; q < nh * nw; q++) {
    const int h = q / nw, v = q % nw, k0 = (h + c.ph) % c.sh, l0 = (v + c.pw) % c.sw;
    const int rows = ceil_div(c.h - h, c.sh), cols = ceil_div(c.w - v, c.sw);
    Class& k = a.k[a.nclass];
    k = Class{};
    k.h0 = h; k.w0 = v;
    k.g = Gather{yb, s.a, ho, wo, c.n, kp * 2, cols, rows * cols * c.n, 1, 1, (h + c.ph - k0) / c.sh, (v + c.pw - l0) / c.sw, -1,
                 make_fastdiv(c.n), make_fastdiv(cols)};
    k.t = Taps{k0 < c.kh ? ceil_div(c.kh - k0, c.sh) : 0, l0 < c.kw ? ceil_div(c.kw - l0, c.sw) : 0, kp / 64, k0, l0, c.sh, c.sw, c.kw};
    if (k.t.ni == 0 || k.t.nj == 0) k.t.ni = 0, k.t.nj = 1;  // (no tap reaches these pixels: zeros)
    k.tiles = tiles_for(a, s, k.g.M);
    most = std::max(most, k.tiles);
    if (++a.nclass < kClasses && q + 1 < nh * nw) continue;
    a.tiles = most * a.nclass;
    if ((e = launch_tiles<1>(a, s, dy.fmt, half, st)) != hipSuccess) return e;
    a.nclass = most = 0;
  }
  return join(a.slices, part, dx, a.slice, a.ta, a.tb, st);
}

hipError_t launch_nvfp_backward_weight(const Conv& c, const NvfpView& dy, const NvfpView& x, float* dw, void* ws, hipStream_t st) {
  const Sizes s = sizes_of(c, 2, dy.fmt);
  const int np = (int)up(c.n, 8), taps = c.kh * c.kw, ho = c.ho(), wo = c.wo();
  __bf16* const yb = static_cast<__bf16*>(ws);
  __bf16* const xb = reinterpret_cast<__bf16*>(static_cast<char*>(ws) + up(s.a, 256));
  float* const part = reinterpret_cast<float*>(static_cast<char*>(ws) + up(s.a, 256) + up(s.b, 256));
  hipError_t e = launch_values(across_task(codes_of(dy, ho * wo, c.n, 1, c.cout), yb, 8),
                               across_task(codes_of(x, c.h * c.w, c.n, 1, c.cin), xb, 8), st);
  if (e != hipSuccess) return e;
  WeightArgs a{};
  a.dy = yb; a.dy_bytes = s.a; a.rows = c.cout;
  a.x = Shift{xb, s.b, c.h, c.w, c.cin, c.kw, np, c.sh, c.sw, c.ph, c.pw, taps * c.cin, ho * wo * (np / 8), make_fastdiv(c.cin),
              make_fastdiv(c.kw), make_fastdiv(np / 8), make_fastdiv(wo)};
  a.slices = s.plan.slices; a.slice = (long long)c.cout * taps * c.cin;
  a.out = a.slices > 1 ? part : dw;
  a.ta = dy.tensor; a.tb = x.tensor;
  a.steps = ceil_div(a.x.pieces, 8);
  a.tiles = ceil_div(c.cout, kBM[s.plan.shape]) * ceil_div(a.x.cols, kBN[s.plan.shape]);
  with_shape<2>(s.plan.shape, [&](auto shape) {
    typedef decltype(shape) S;
    hipLaunchKernelGGL(nvfp_weight_kernel<S>, dim3((unsigned)(a.tiles * a.slices)), dim3(S::THREADS), 0, st, a);
  });
  if ((e = launch_check()) != hipSuccess) return e;
  return join(a.slices, part, dw, a.slice, a.ta, a.tb, st);
}

}  // namespace mq
