// newton.hip -- the orthogonalised weight update: X0 = U / (|U|_F + eps), then
//   A = X X^T,  B = a I + b A + c A^2,  X <- B X
// for a number of steps, with U the gradient or the momentum that the first
// pass updates. X is m x n with m <= n (the transpose of a tall matrix).
//
// The result has fp32's accuracy: every product's factors are f16 pairs
// (mma_core.h), summed in fp32 by the f16 matrix units, which at three
// products for one are five times as fast as the fp32 ones. Values are stored
// times the largest power of two that keeps them within f16's range: the steps
// are refused unless |X| and |A| stay below 2 and |B| below 4 (the polynomial's
// range, checked on the host), so X and A are stored times 2^15 and B times
// 2^14. A stored value is off by 2^-22 of itself, or, as low parts may be f16
// subnormals, by 2^-40 (B: 2^-39): more than that for entries below 2^-18 (2^-17),
// which are about one in a hundred of X0 at 2048 x 4096.
// A and A^2 are symmetric: tiles on and above the diagonal are computed, and
// written on both sides. X is kept in both orientations ([m][n] for A, [n][m]
// for the product with B), since an operand's rows run along k.
// The matrices of a call share the launches of a product, one for each size of
// tile that it needs (a network's layers are small).
// 2048 x 4096, 5 steps: 1090 us, 830 TFLOP/s of f16 products with everything; 27
// layers of 16 x 27 to 256 x 1152: 149 us, 17 kernels of 7 to 11 us one after the
// other, which launches and the first loads and last stores take.
#include <math.h>

#include <algorithm>

#include "mma_core.h"
#include "mqconv_train.h"
#include "train.h"

namespace mq {

namespace {

constexpr float kUp = 32768.0f;  // 2^15
constexpr int kMaxParts = 1024;  // fp64 partial sums of squares of a matrix

struct Mat {
  const float* g;
  float *mom, *out;
  long long at;            // byte offset of its planes in the workspace
  long long part;          // its slices' sums, from Group::part on
  int rows, cols, mp, np;  // mp, np: the smaller and the larger extent, rounded up to 32
  int chunk;               // elements of a partial sum
  float scale;             // factor of the orthogonalised matrix in the weight's update
};

struct Group {
  Mat m[kUpdateGroup];
  int start[kUpdateGroup + 1];  // first workgroup of every matrix
  int tiles[kUpdateGroup], slices[kUpdateGroup];  // of the present product
  float4* part;                 // sums of slices
  int count;
  uint8_t* ws;
  double* parts;  // [count][kMaxParts]
  const float* rate;
  float a, b, c, eps, momentum, decay, lr;
  bool nesterov, update;
  int from;  // which of the two [n][m] copies of X is read
};

// planes of a matrix: X [m][n], two copies of its transpose, A and B [m][m]
__host__ __device__ inline long long plane_x(const Mat& m) { return (long long)m.mp * m.np * 4; }
__host__ __device__ inline long long plane_a(const Mat& m) { return (long long)m.mp * m.mp * 4; }
inline long long planes_bytes(const Mat& m) { return 3 * plane_x(m) + 2 * plane_a(m); }
__device__ __forceinline__ uint8_t* x_of(const Group& g, const Mat& m) { return g.ws + m.at; }
__device__ __forceinline__ uint8_t* xt_of(const Group& g, const Mat& m, int k) { return g.ws + m.at + (1 + k) * plane_x(m); }
__device__ __forceinline__ uint8_t* a_of(const Group& g, const Mat& m, int k) {
  return g.ws + m.at + 3 * plane_x(m) + k * plane_a(m);
}

// The matrix of workgroup b, and its number within that. A lane compares with
// one start: one after the other they cost 3 us at 27 matrices.
__device__ __forceinline__ int matrix_of(const Group& g, int b, int& local) {
  const int lane = threadIdx.x & 63;
  const bool behind = lane + 1 < g.count && b >= g.start[lane + 1 < kUpdateGroup ? lane + 1 : 0];
  const int i = __builtin_amdgcn_readfirstlane(__builtin_popcountll(__builtin_amdgcn_ballot_w64(behind)));
  local = b - g.start[i];
  return i;
}

__device__ __forceinline__ float direction(const Group& g, float grad, float mom) {
  return !g.update ? grad : (g.nesterov ? __builtin_fmaf(g.momentum, mom, grad) : mom);
}

// Partial sums of squares of U; the momentum is updated on the way.
__global__ __launch_bounds__(256) void norm_kernel(const Group g) {
  __shared__ double red[4];
  int part;
  const int k = matrix_of(g, blockIdx.x, part);
  const Mat& m = g.m[k];
  const long long n = (long long)m.rows * m.cols, i0 = (long long)part * m.chunk, i1 = min(n, i0 + m.chunk);
  double s = 0;
  constexpr int L = 8;  // elements whose loads are under way together
  for (long long at = i0; at < i1; at += 256 * L) {
    float u[L], mom[L];
#pragma unroll
    for (int k = 0; k < L; k++) {
      const long long i = at + 256 * k + threadIdx.x;
      u[k] = i < i1 ? m.g[i] : 0.0f;
      mom[k] = g.update && i < i1 ? m.mom[i] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < L; k++) {
      const long long i = at + 256 * k + threadIdx.x;
      if (g.update) {
        mom[k] = __builtin_fmaf(g.momentum, mom[k], u[k]);
        if (i < i1) m.mom[i] = mom[k];
      }
      const double v = direction(g, u[k], mom[k]);
      s = __builtin_fma(v, v, s);
    }
  }
#pragma unroll
  for (int off = 1; off < 64; off *= 2) s += __shfl_xor(s, off);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) g.parts[(long long)k * kMaxParts + part] = (red[0] + red[1]) + (red[2] + red[3]);
}

struct Pair {
  _Float16 hi, lo;
};
__device__ __forceinline__ Pair split(float v) {
  Pair p;
  p.hi = (_Float16)v;
  p.lo = (_Float16)(v - (float)p.hi);
  return p;
}
// byte offset of element (r, c)'s high part in planes of `ld` columns; the low part is 64 bytes behind it
__device__ __forceinline__ long long at_of(int r, int c, int ld) {
  return (long long)r * ld * 4 + (c >> 5) * kPiece + (c & 31) * 2;
}

constexpr int kTile = 64;  // of the first pass

// X0 in both orientations, zeros in the padding.
__global__ __launch_bounds__(256) void init_kernel(const Group g) {
  __shared__ float tile[kTile][kTile + 1];
  __shared__ double red[4];
  int local;
  const Mat& m = g.m[matrix_of(g, blockIdx.x, local)];
  const int k = (int)(&m - g.m);
  const long long n = (long long)m.rows * m.cols;
  const int parts = (int)((n + m.chunk - 1) / m.chunk);
  const int nx = (m.np + kTile - 1) / kTile;
  const int i0 = local / nx * kTile, j0 = local % nx * kTile;  // tile of X
  const bool tall = m.rows > m.cols;
  // read along the matrix's own rows, all loads before the sum of squares
  const int r0 = tall ? j0 : i0, c0 = (tall ? i0 : j0) + (threadIdx.x & 63);
  constexpr int L = kTile * kTile / 256;
  float u[L], mom[L];
#pragma unroll
  for (int t = 0; t < L; t++) {
    const int r = r0 + 4 * t + (threadIdx.x >> 6);
    const long long i = (long long)r * m.cols + c0;
    const bool in = r < m.rows && c0 < m.cols;
    u[t] = in ? m.g[i] : 0.0f;
    mom[t] = g.update && in ? m.mom[i] : 0.0f;
  }
  double s = 0;
  for (int i = threadIdx.x; i < parts; i += 256) s += g.parts[(long long)k * kMaxParts + i];
#pragma unroll
  for (int off = 1; off < 64; off *= 2) s += __shfl_xor(s, off);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  const double inv = (double)kUp / (sqrt((red[0] + red[1]) + (red[2] + red[3])) + (double)g.eps);
#pragma unroll
  for (int t = 0; t < L; t++) tile[4 * t + (threadIdx.x >> 6)][threadIdx.x & 63] = (float)((double)direction(g, u[t], mom[t]) * inv);
  __syncthreads();
  uint8_t* const x = x_of(g, m);
  uint8_t* const xt = xt_of(g, m, 0);
  for (int t = threadIdx.x; t < 2 * kTile * (kTile / 8); t += 256) {
    // eight neighbours along k of one row, of X and then of its transpose
    const bool second = t >= kTile * (kTile / 8);
    const int u = second ? t - kTile * (kTile / 8) : t, r = u / (kTile / 8), c = u % (kTile / 8) * 8;
    const int row = (second ? j0 : i0) + r, col = (second ? i0 : j0) + c;
    if (row >= (second ? m.np : m.mp) || col >= (second ? m.mp : m.np)) continue;
    half8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const Pair p = split(second != tall ? tile[c + e][r] : tile[r][c + e]);
      hi[e] = p.hi;
      lo[e] = p.lo;
    }
    uint8_t* const to = (second ? xt : x) + at_of(row, col, second ? m.mp : m.np);
    *reinterpret_cast<half8*>(to) = hi;
    *reinterpret_cast<half8*>(to + 64) = lo;
  }
}

enum { kGram, kPoly, kApply, kLast };

// Tile k of a symmetric product: those of t x u tiles, q columns of tiles as wide as a row of tiles is high, that lie on or
// above the diagonal. (The blocks on it are whole, so theirs is a store of one side alone.)
__device__ __forceinline__ void triangle(int k, int u, int q, int& i, int& j) {
  i = 0;
  while (k >= u - i * q) {
    k -= u - i * q;
    i++;
  }
  j = i * q + k;
}

// What becomes of 32 x 32 sums, rows r0 .. and columns c0 .. of the product of kind KIND, as the matrix units leave them.
struct Last {
  bool tall;
  float keep, step;
  int real_m, real_n;
};
__device__ __forceinline__ Last last_of(const Group& g, const Mat& m) {
  const float lr = g.rate ? g.lr * *g.rate : g.lr;
  return Last{m.rows > m.cols, __builtin_fmaf(-lr, g.decay, 1.0f), -lr * m.scale, min(m.rows, m.cols), max(m.rows, m.cols)};
}
// Sums go through LDS, [column][row] of 32 x 32, to whole pieces of rows (128
// bytes of high and low parts) in either orientation. The code behind that is a
// loop over a wave's blocks and both orientations: it runs once a tile, so
// written out it only costs instruction fetches.
constexpr int kStrip = 36, kStripFloats = 32 * kStrip;
__device__ __forceinline__ void leave(const v16f& s, float* strip, int lane) {
#pragma unroll
  for (int e = 0; e < 4; e++)
    *reinterpret_cast<float4*>(strip + (lane & 31) * kStrip + 8 * e + 4 * (lane >> 5)) =
        make_float4(s[4 * e], s[4 * e + 1], s[4 * e + 2], s[4 * e + 3]);
}
template <int KIND>
__device__ __forceinline__ void finish(const Group& g, const Mat& m, const Last& last, int r0, int c0, bool both, int lane,
                                       const float* strip) {
  const int mp = m.mp, np = m.np;
  if (r0 >= mp || c0 >= (KIND <= kPoly ? mp : np)) return;  // (whole waves)
  if constexpr (KIND == kLast) {
    const int col = c0 + (lane & 31), row = r0 + (lane >> 5);
    const long long down = last.tall ? 1 : m.cols, right = last.tall ? m.cols : 1;
    float old[16];
    if (g.update) {  // (all under way together, so none under a condition: places past the end read the last one)
#pragma unroll
      for (int e = 0; e < 16; e++) old[e] = m.out[min(row + 2 * e, last.real_m - 1) * down + min(col, last.real_n - 1) * right];
    }
#pragma unroll
    for (int e = 0; e < 16; e++) {
      const float o = strip[(lane & 31) * kStrip + (lane >> 5) + 2 * e] * (2.0f / kUp / kUp);
      if (row + 2 * e < last.real_m && col < last.real_n)
        m.out[(row + 2 * e) * down + col * right] = g.update ? __builtin_fmaf(last.step, o, old[e] * last.keep) : o;
    }
  } else {
    const int c = (lane & 3) * 8;
    uint8_t* const rows = KIND == kApply ? x_of(g, m) : a_of(g, m, KIND == kPoly ? 1 : 0);
    uint8_t* const across = KIND == kApply ? xt_of(g, m, g.from ^ 1) : rows;
    const uint8_t* const from = a_of(g, m, 0);
    // the rows of the block's transpose and then its own: a lane has the high or the low parts of eight neighbours
#pragma unroll 1
    for (int side = 0; side < (KIND == kApply || both ? 2 : 1); side++) {
      const int row0 = side ? r0 : c0, col0 = side ? c0 : r0, ld = KIND == kApply && side ? np : mp;
      const int step = side ? kStrip : 1, next = side ? 1 : kStrip;
      uint8_t* const to = (side ? rows : across) + at_of(row0 + (lane >> 3), col0 + c, ld) + (lane & 4) * 16;
      const float* const in = strip + (lane >> 3) * next + c * step;
      half8 hi[4], lo[4];
      if constexpr (KIND == kPoly)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const uint8_t* const p = from + at_of(row0 + 8 * i + (lane >> 3), col0 + c, ld);
          hi[i] = *reinterpret_cast<const half8*>(p);
          lo[i] = *reinterpret_cast<const half8*>(p + 64);
        }
#pragma unroll
      for (int i = 0; i < 4; i++) {
        half8 out;
#pragma unroll
        for (int e = 0; e < 8; e++) {
          float v = in[8 * i * next + e * step];
          if constexpr (KIND == kGram) {
            v *= 1.0f / kUp;
          } else if constexpr (KIND == kApply) {
            v *= 2.0f / kUp;
          } else {
            // b A + c A^2, and a on the diagonal, so that the next product is a whole step
            const int r = row0 + 8 * i + (lane >> 3);
            v = __builtin_fmaf(g.b * 0.5f, (float)hi[i][e] + (float)lo[i][e], v * (g.c * (0.5f / kUp)));
            if (r == col0 + c + e && r < last.real_m) v += g.a * (0.5f * kUp);
          }
          const Pair p = split(v);
          out[e] = lane & 4 ? p.lo : p.hi;
        }
        *reinterpret_cast<half8*>(to + (long long)i * 32 * ld) = out;
      }
    }
  }
}

// The place of tile `tile` of a matrix's product.
template <int KIND, class S>
__device__ __forceinline__ void place(const Mat& m, int tile, int& i0, int& j0, bool& both) {
  int ti, tj;
  if constexpr (KIND <= kPoly) {
    constexpr int Q = S::BM / S::BN;
    triangle(tile, (m.mp + S::BN - 1) / S::BN, Q, ti, tj);
    both = tj >= (ti + 1) * Q;
  } else {
    const int tm = (m.mp + S::BM - 1) / S::BM;  // neighbours: tiles of one column, which share X's rows
    tj = tile / tm;
    ti = tile - tj * tm;
    both = false;
  }
  i0 = ti * S::BM;
  j0 = tj * S::BN;
}

template <int KIND, class S>
__global__ __launch_bounds__(S::THREADS, S::TM * S::TN >= 8 ? 1 : 2) void newton_kernel(const Group g) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  const MmaWave<S> me;
  const int lane = me.lane, wave = me.wave;
  int local;
  const int which = matrix_of(g, xcd_tile(blockIdx.x, gridDim.x), local);
  const Mat& m = g.m[which];
  const int slices = g.slices[which], nt = g.tiles[which], z = local / nt, tile = local - z * nt;
  int i0, j0;
  bool both;
  place<KIND, S>(m, tile, i0, j0, both);
  const int mp = m.mp, k = KIND == kGram ? m.np : mp, rows_r = KIND <= kPoly ? mp : m.np;
  const uint8_t* const left = KIND == kGram ? x_of(g, m) : a_of(g, m, KIND == kPoly ? 0 : 1);
  const uint8_t* const right = KIND <= kPoly ? left : xt_of(g, m, g.from);
  RowLoader<S::LA, S::NW> la;
  RowLoader<S::LB, S::NW> lb;
  la.init(left, (long long)mp * k * 4, i0, mp, k * 4, wave, lane);
  lb.init(right, (long long)rows_r * k * 4, j0, rows_r, k * 4, wave, lane);
  v16f acc[S::TM][S::TN];
  mma_zero<S>(acc);
  const int all = k / 32, s0 = (int)((long long)all * z / slices), steps = (int)((long long)all * (z + 1) / slices) - s0;
  if constexpr (S::TM * S::TN >= 8) mma_loop_wide<Split, S>(lds, la, lb, s0, steps, me, acc);
  else mma_loop<Split, S>(lds, la, lb, s0 + me.first(steps), me.count(steps), me.most(steps), me, acc);
  __syncthreads();  // (the rings are free)
  if (me.group != 0) return;
  if (slices > 1) {
    // lane by lane: the kernel behind this one has the same order
    float4* const to = g.part + m.part + ((long long)tile * slices + z) * (S::BM * S::BN / 4) + wave * (S::TM * S::TN * 256) + lane;
#pragma unroll
    for (int i = 0; i < S::TM; i++)
#pragma unroll
      for (int j = 0; j < S::TN; j++, __builtin_amdgcn_sched_barrier(0))
#pragma unroll
        for (int e = 0; e < 4; e++)
          to[((i * S::TN + j) * 4 + e) * 64] =
              make_float4(acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]);
    return;
  }
  static_assert(S::NW * S::TM * S::TN * kStripFloats * 4 <= S::LDS, "strips");
  float* const strips = reinterpret_cast<float*>(lds) + wave * (S::TM * S::TN * kStripFloats);
#pragma unroll
  for (int i = 0; i < S::TM; i++)
#pragma unroll
    for (int j = 0; j < S::TN; j++, __builtin_amdgcn_sched_barrier(0)) leave(acc[i][j], strips + (i * S::TN + j) * kStripFloats, lane);
  lds_ready();
  const Last last = last_of(g, m);
#pragma unroll 1
  for (int b = 0; b < S::TM * S::TN; b++)
    finish<KIND>(g, m, last, i0 + ((wave / S::WN) * S::TM + b / S::TN) * 32, j0 + ((wave % S::WN) * S::TN + b % S::TN) * 32, both, lane,
                 strips + b * kStripFloats);
}

// The slices' sums, added in order; a wave takes 32 x 32 of a tile.
template <int KIND, class S>
__global__ __launch_bounds__(256) void join_kernel(const Group g) {
  constexpr int PER = S::NW * S::TM * S::TN;  // parts of a tile
  __shared__ __attribute__((aligned(16))) float strips[4 * kStripFloats];
  const int lane = threadIdx.x & 63;
  int local;
  const int which = matrix_of(g, (int)blockIdx.x, local);
  const Mat& m = g.m[which];
  const int p = __builtin_amdgcn_readfirstlane(local * 4 + (threadIdx.x >> 6)), tile = p / PER, part = p - tile * PER;
  if (PER % 4 != 0 && tile >= g.tiles[which]) return;  // (whole waves; the barrier counts those that are left)
  const int slices = g.slices[which];
  int i0, j0;
  bool both;
  place<KIND, S>(m, tile, i0, j0, both);
  const int wave = part / (S::TM * S::TN), ij = part - wave * (S::TM * S::TN), i = ij / S::TN, j = ij - i * S::TN;
  const int r0 = i0 + ((wave / S::WN) * S::TM + i) * 32, c0 = j0 + ((wave % S::WN) * S::TN + j) * 32;
  const float4* const from = g.part + m.part + (long long)tile * slices * (S::BM * S::BN / 4) + part * 256 + lane;
  float4 sum[4];
#pragma unroll
  for (int e = 0; e < 4; e++) sum[e] = from[e * 64];
  for (int z = 1; z < slices; z++)
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const float4 v = from[(long long)z * (S::BM * S::BN / 4) + e * 64];
      sum[e].x += v.x; sum[e].y += v.y; sum[e].z += v.z; sum[e].w += v.w;
    }
  v16f s;
#pragma unroll
  for (int e = 0; e < 4; e++) s[4 * e] = sum[e].x, s[4 * e + 1] = sum[e].y, s[4 * e + 2] = sum[e].z, s[4 * e + 3] = sum[e].w;
  float* const strip = strips + (threadIdx.x >> 6) * kStripFloats;
  leave(s, strip, lane);
  lds_ready();
  finish<KIND>(g, m, last_of(g, m), r0, c0, both, lane, strip);
}

// ---- plans --------------------------------------------------------------------------------------
// A matrix's tiles and slices are chosen by its own extents alone, so its
// result does not depend on what else a call holds.
typedef MmaShape<256, 128, 2, 2, 3> Wide;
typedef MmaShape<64, 64, 2, 2, 3> Mid;
// Of small matrices A and A^2 have few tiles and long sums, so each tile is a
// wave's, four times over along k.
template <int KIND>
struct NarrowOf {
  typedef MmaShape<32, 32, 1, 1, KIND == kGram ? 3 : 2, 4> type;
};
enum { kWide, kMid, kNarrow };

int tiles(int n, int b) { return (n + b - 1) / b; }

template <int KIND, class S>
int tiles_of(const Mat& m) {
  const int tm = tiles(m.mp, S::BM);
  if (KIND > kPoly) return tm * tiles(m.np, S::BN);
  const int u = tiles(m.mp, S::BN), q = S::BM / S::BN;
  int n = 0;
  for (int i = 0; i < tm; i++) n += u - i * q;
  return n;
}

// Measured, us a product with its join, at n wide tiles times steps of 32 and t mid tiles:
//             A                        A^2                      B X
//             n     t   wide mid  nar  n     t   wide mid  nar  n     wide  mid
// 256 x 1152  108   10       16.2  9.6     10       8.2  7.0
// 512 x 2048  384   36  25.6 24.4 12.9  96    36  52.0 11.3  9.0  512   33.1  13.4
// 768 x 768   288   78       12.2 14.4  288   78       15.1 12.5
// 1024 x 1024 640  136  26.4 14.9 23.6  640  136  27.9 15.9 19.7  1024  27.6  16.6
// 1536 x 1536 2016 300  32.2      52.0  2016 300  34.8      42.6  3456  39.6  36.4
// 2048 x 4096 9216 528  69.1     184.0  4608 528  48.6      89.7  16384 102.1 147.9
// Wide tiles pay with steps enough over all of them: few leave the chip empty,
// or spend their gain on joining slices; mid tiles with one for every third
// compute unit and more.
struct Plan {
  int size, tiles, slices;
};
template <int KIND>
Plan plan_of(const Mat& m) {
  const int steps = (KIND == kGram ? m.np : m.mp) / 32;
  Plan p{kWide, tiles_of<KIND, Wide>(m), 1};
  if ((long long)p.tiles * steps >= (KIND <= kPoly ? 1000 : 4096)) {
    // one workgroup a compute unit; slices of 16 steps at least
    p.slices = std::max(1, std::min({256 / p.tiles, steps / 16, 32}));
    return p;
  }
  p = Plan{kMid, tiles_of<KIND, Mid>(m), 1};
  if (KIND <= kPoly && p.tiles < 100) {
    p = Plan{kNarrow, tiles_of<KIND, typename NarrowOf<KIND>::type>(m), 1};
    if (KIND == kGram) p.slices = std::max(1, std::min({256 / p.tiles, steps / 48, 32}));
  }
  return p;
}
template <int KIND, class F>
auto with_size(int size, F&& f) {
  if (size == kWide) return f(Wide{});
  if constexpr (KIND <= kPoly)
    if (size == kNarrow) return f(typename NarrowOf<KIND>::type{});
  return f(Mid{});
}
template <int KIND>
long long part_of(const Mat& m) {  // float4 of its slices
  const Plan p = plan_of<KIND>(m);
  const int tile = with_size<KIND>(p.size, [](auto s) { return decltype(s)::BM * decltype(s)::BN; });
  return p.slices == 1 ? 0 : (long long)p.tiles * p.slices * tile / 4;
}
long long part_size(const Mat& m) { return std::max({part_of<kGram>(m), part_of<kPoly>(m), part_of<kApply>(m)}); }

template <int KIND, class S>
hipError_t launch_size(Group& g, int size, hipStream_t st) {
  int total = 0, join = 0, joins[kUpdateGroup];
  for (int i = 0; i < g.count; i++) {
    const Plan p = plan_of<KIND>(g.m[i]);
    const bool in = p.size == size;
    g.start[i] = total;
    g.tiles[i] = p.tiles;
    g.slices[i] = p.slices;
    total += in ? p.tiles * p.slices : 0;
    joins[i] = join;
    join += in && p.slices > 1 ? tiles(p.tiles * S::NW * S::TM * S::TN, 4) : 0;
  }
  if (total == 0) return hipSuccess;
  g.start[g.count] = total;
  hipLaunchKernelGGL((newton_kernel<KIND, S>), dim3((unsigned)total), dim3(S::THREADS), 0, st, g);
  const hipError_t e = launch_check();
  if constexpr (S::BM == Wide::BM || (KIND == kGram && S::BM != Mid::BM)) {  // (the others take no slices)
    if (e != hipSuccess || join == 0) return e;
    std::copy(joins, joins + g.count, g.start);
    g.start[g.count] = join;
    hipLaunchKernelGGL((join_kernel<KIND, S>), dim3((unsigned)join), dim3(256), 0, st, g);
    return launch_check();
  }
  return e;
}

template <int KIND>
hipError_t launch_product(Group& g, hipStream_t st) {
  for (int size = kWide; size <= (KIND <= kPoly ? kNarrow : kMid); size++) {
    const hipError_t e = with_size<KIND>(size, [&](auto s) { return launch_size<KIND, decltype(s)>(g, size, st); });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

Mat make_mat(int rows, int cols) {
  Mat m{};
  m.rows = rows; m.cols = cols;
  m.mp = tiles(std::min(rows, cols), 32) * 32;
  m.np = tiles(std::max(rows, cols), 32) * 32;
  const long long n = (long long)rows * cols;
  m.chunk = (int)std::max(2048LL, ((n + kMaxParts - 1) / kMaxParts + 255) / 256 * 256);
  return m;
}

size_t parts_bytes(int count) { return (size_t)count * kMaxParts * sizeof(double); }

}  // namespace

bool newton_shape_ok(int rows, int cols) {
  const Mat m = make_mat(rows, cols);
  return plane_x(m) < kBeyond && plane_a(m) < kBeyond;
}

size_t newton_workspace_bytes(int count, const int* rows, const int* cols) {
  size_t n = parts_bytes(count);
  for (int i = 0; i < count; i++) {
    const Mat m = make_mat(rows[i], cols[i]);
    n += (size_t)planes_bytes(m) + (size_t)part_size(m) * sizeof(float4);
  }
  return n;
}

hipError_t launch_newton(const UpdateSpec& u, int count, const int* rows, const int* cols, const float* const* grad,
                         float* const* mom, float* const* out, void* ws, hipStream_t st) {
  Group g{};
  g.count = count;
  g.parts = static_cast<double*>(ws);
  g.ws = static_cast<uint8_t*>(ws) + parts_bytes(count);
  g.a = u.a; g.b = u.b; g.c = u.c; g.eps = u.eps;
  g.update = mom != nullptr;
  g.momentum = u.momentum; g.decay = u.decay; g.lr = u.lr; g.nesterov = u.nesterov; g.rate = u.rate;
  long long at = 0, part = 0;
  int norm_groups = 0, init_groups = 0;
  int norm_start[kUpdateGroup], init_start[kUpdateGroup];
  for (int i = 0; i < count; i++) {
    Mat& m = g.m[i] = make_mat(rows[i], cols[i]);
    m.g = grad[i]; m.out = out[i]; m.mom = mom ? mom[i] : nullptr;
    m.scale = u.scale == MQ_SCALE_ASPECT ? sqrtf(std::max(1.0f, (float)rows[i] / (float)cols[i]))
            : u.scale == MQ_SCALE_RMS    ? 0.2f * sqrtf((float)std::max(rows[i], cols[i]))
                                         : 1.0f;
    m.at = at;
    at += planes_bytes(m);
    m.part = part;
    part += part_size(m);
    norm_start[i] = norm_groups;
    norm_groups += (int)(((long long)m.rows * m.cols + m.chunk - 1) / m.chunk);
    init_start[i] = init_groups;
    init_groups += tiles(m.mp, kTile) * tiles(m.np, kTile);
  }
  g.part = reinterpret_cast<float4*>(g.ws + at);
  std::copy(norm_start, norm_start + count, g.start);
  hipLaunchKernelGGL(norm_kernel, dim3((unsigned)norm_groups), dim3(256), 0, st, g);
  hipError_t e = launch_check();
  if (e != hipSuccess) return e;
  std::copy(init_start, init_start + count, g.start);
  hipLaunchKernelGGL(init_kernel, dim3((unsigned)init_groups), dim3(256), 0, st, g);
  if ((e = launch_check()) != hipSuccess) return e;
  for (int s = 0; s < u.steps; s++) {
    if ((e = launch_product<kGram>(g, st)) != hipSuccess) return e;
    if ((e = launch_product<kPoly>(g, st)) != hipSuccess) return e;
    e = s + 1 < u.steps ? launch_product<kApply>(g, st) : launch_product<kLast>(g, st);
    if (e != hipSuccess) return e;
    g.from ^= 1;
  }
  return hipSuccess;
}

}  // namespace mq
