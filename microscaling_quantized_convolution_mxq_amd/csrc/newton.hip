// newton.hip -- the orthogonalised weight update: X0 = U / (|U|_F + eps), then
//   A = X X^T,  B = a I + b A + c A^2,  X <- B X
// for a number of steps, with U the gradient or the momentum that the first
// pass updates. X is m x n with m <= n (the transpose of a tall matrix).
//
// The result has fp32's accuracy: every product's factors are f16 pairs (22
// bits, mma_core.h), summed in fp32 by the f16 matrix units, which at three
// products for one are five times as fast as the fp32 ones. Values are stored
// times a power of two that keeps them within f16's range and their low parts
// above its subnormals: the steps are refused unless |X| and |A| stay below 2
// and |B| below 4 (the polynomial's range, checked on the host), so X and A
// are stored times 2^15 and B times 2^14.
// A and A^2 are symmetric: tiles on and above the diagonal are computed, and
// written on both sides. X is kept in both orientations ([m][n] for A, [n][m]
// for the product with B), since an operand's rows run along k.
// All matrices of a call share every launch (a network's layers are small).
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
  int rows, cols, mp, np;  // mp, np: the smaller and the larger extent, rounded up to 32
  int chunk;               // elements of a partial sum
  float scale;             // factor of the orthogonalised matrix in the weight's update
};

struct Group {
  Mat m[kUpdateGroup];
  int start[kUpdateGroup + 1];  // first workgroup of every matrix
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

// the matrix of workgroup b, and its number within that
__device__ __forceinline__ int matrix_of(const Group& g, int b, int& local) {
  int i = 0;
  while (i + 1 < g.count && b >= g.start[i + 1]) i++;
  local = b - g.start[i];
  return i;
}

__device__ __forceinline__ float direction(const Group& g, const Mat& m, long long i, float mom) {
  return !g.update ? m.g[i] : (g.nesterov ? __builtin_fmaf(g.momentum, mom, m.g[i]) : mom);
}

// Partial sums of squares of U; the momentum is updated on the way.
__global__ __launch_bounds__(256) void norm_kernel(const Group g) {
  __shared__ double red[4];
  int part;
  const int k = matrix_of(g, blockIdx.x, part);
  const Mat& m = g.m[k];
  const long long n = (long long)m.rows * m.cols, i0 = (long long)part * m.chunk, i1 = min(n, i0 + m.chunk);
  double s = 0;
  for (long long i = i0 + threadIdx.x; i < i1; i += 256) {
    float mom = 0;
    if (g.update) {
      mom = __builtin_fmaf(g.momentum, m.mom[i], m.g[i]);
      m.mom[i] = mom;
    }
    const double u = direction(g, m, i, mom);
    s = __builtin_fma(u, u, s);
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
  double s = 0;
  for (int i = threadIdx.x; i < parts; i += 256) s += g.parts[(long long)k * kMaxParts + i];
#pragma unroll
  for (int off = 1; off < 64; off *= 2) s += __shfl_xor(s, off);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  const int nx = (m.np + kTile - 1) / kTile;
  const int i0 = local / nx * kTile, j0 = local % nx * kTile;  // tile of X
  const bool tall = m.rows > m.cols;
  __syncthreads();
  const double inv = (double)kUp / (sqrt((red[0] + red[1]) + (red[2] + red[3])) + (double)g.eps);
  // read along the matrix's own rows
  const int r0 = tall ? j0 : i0, c0 = tall ? i0 : j0;
  for (int t = threadIdx.x; t < kTile * kTile; t += 256) {
    const int r = r0 + t / kTile, c = c0 + t % kTile;
    float v = 0;
    if (r < m.rows && c < m.cols) {
      const long long i = (long long)r * m.cols + c;
      v = (float)((double)direction(g, m, i, g.update ? m.mom[i] : 0.0f) * inv);
    }
    tile[t / kTile][t % kTile] = v;
  }
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

typedef _Float16 half4 __attribute__((ext_vector_type(4)));

// Four values down a column, as neighbours of one row of the transpose.
__device__ __forceinline__ void store_across(uint8_t* p, int ld, int r, int c, const float (&v)[4]) {
  half4 hi, lo;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const Pair x = split(v[e]);
    hi[e] = x.hi;
    lo[e] = x.lo;
  }
  uint8_t* const to = p + at_of(c, r, ld);
  *reinterpret_cast<half4*>(to) = hi;
  *reinterpret_cast<half4*>(to + 64) = lo;
}
__device__ __forceinline__ void store_down(uint8_t* p, int ld, int r, int c, const float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const Pair x = split(v[e]);
    uint8_t* const to = p + at_of(r + e, c, ld);
    *reinterpret_cast<_Float16*>(to) = x.hi;
    *reinterpret_cast<_Float16*>(to + 64) = x.lo;
  }
}

enum { kGram, kPoly, kApply, kLast };

// number of the pair (i, j), i <= j, in rows of the upper triangle of t x t tiles
__device__ __forceinline__ void triangle(int k, int t, int& i, int& j) {
  i = 0;
  while (k >= t - i) {
    k -= t - i;
    i++;
  }
  j = i + k;
}

template <int KIND, class S>
__global__ __launch_bounds__(S::THREADS, 2) void newton_kernel(const Group g) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int local;
  const Mat& m = g.m[matrix_of(g, xcd_tile(blockIdx.x, gridDim.x), local)];
  const int mp = m.mp, np = m.np;
  int ti, tj;
  if (KIND <= kPoly) triangle(local, (mp + S::BM - 1) / S::BM, ti, tj);
  else {
    const int tm = (mp + S::BM - 1) / S::BM;  // neighbours: tiles of one column, which share X's rows
    tj = local / tm;
    ti = local - tj * tm;
  }
  const int i0 = ti * S::BM, j0 = tj * S::BN;
  const uint8_t* const x = x_of(g, m);
  const uint8_t* const left = KIND == kGram ? x : a_of(g, m, KIND == kPoly ? 0 : 1);
  const uint8_t* const right = KIND == kGram ? x : (KIND == kPoly ? left : xt_of(g, m, g.from));
  const int k = KIND == kGram ? np : mp, rows_r = KIND <= kPoly ? mp : np;
  RowLoader<S::LA, S::NW> la;
  RowLoader<S::LB, S::NW> lb;
  la.init(left, (long long)mp * k * 4, i0, mp, k * 4, wave, lane);
  lb.init(right, (long long)rows_r * k * 4, j0, rows_r, k * 4, wave, lane);
  v16f acc[S::TM][S::TN];
  mma_zero<S>(acc);
  mma_loop<Split, S>(lds, la, lb, 0, k / 32, wave, lane, acc);

  if constexpr (KIND <= kPoly) {
    uint8_t* const to = a_of(g, m, KIND == kPoly ? 1 : 0);
    mma_results<S>(acc, wave, lane, [&](int r, int c, const float (&s)[4]) {
      const int row = i0 + r, col = j0 + c;
      if (row >= mp || col >= mp) return;
      float v[4];
      if constexpr (KIND == kGram) {
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = s[e] * (1.0f / kUp);
      } else {
        // b A + c A^2, and a on the diagonal, so that the next product is a whole step (A is symmetric: its row is
        // read along the columns here)
        const uint8_t* const from = left + at_of(col, row, mp);
        const half4 hi = *reinterpret_cast<const half4*>(from), lo = *reinterpret_cast<const half4*>(from + 64);
        const int real = min(m.rows, m.cols);
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float a = (float)hi[e] + (float)lo[e];
          v[e] = __builtin_fmaf(g.b * 0.5f, a, s[e] * (g.c * (0.5f / kUp)));
          if (row + e == col && col < real) v[e] += g.a * (0.5f * kUp);
        }
      }
      store_across(to, mp, row, col, v);
      if (ti != tj) store_down(to, mp, row, col, v);
    });
  } else if constexpr (KIND == kApply) {
    uint8_t* const xo = x_of(g, m);
    uint8_t* const xt = xt_of(g, m, g.from ^ 1);
    mma_results<S>(acc, wave, lane, [&](int r, int c, const float (&s)[4]) {
      const int row = i0 + r, col = j0 + c;
      if (row >= mp || col >= np) return;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] = s[e] * (2.0f / kUp);
      store_across(xt, mp, row, col, v);
      store_down(xo, np, row, col, v);
    });
  } else {
    const bool tall = m.rows > m.cols;
    const float lr = g.rate ? g.lr * *g.rate : g.lr;
    const float keep = __builtin_fmaf(-lr, g.decay, 1.0f), step = -lr * m.scale;
    const int real_m = min(m.rows, m.cols), real_n = max(m.rows, m.cols);
    mma_results<S>(acc, wave, lane, [&](int r, int c, const float (&s)[4]) {
      const int row = i0 + r, col = j0 + c;
      if (col >= real_n) return;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        if (row + e >= real_m) break;
        const long long i = tall ? (long long)col * m.cols + row + e : (long long)(row + e) * m.cols + col;
        const float o = s[e] * (2.0f / kUp / kUp);
        m.out[i] = g.update ? __builtin_fmaf(step, o, m.out[i] * keep) : o;
      }
    });
  }
}

typedef MmaShape<64, 64, 2, 2, 3> Small;
typedef MmaShape<128, 128, 2, 2, 2> Large;

int tiles(int n, int b) { return (n + b - 1) / b; }

template <int KIND, class S>
hipError_t launch_product(Group& g, hipStream_t st) {
  int total = 0;
  for (int i = 0; i < g.count; i++) {
    g.start[i] = total;
    const int tm = tiles(g.m[i].mp, S::BM);
    total += KIND <= kPoly ? tm * (tm + 1) / 2 : tm * tiles(g.m[i].np, S::BN);
  }
  g.start[g.count] = total;
  hipLaunchKernelGGL((newton_kernel<KIND, S>), dim3((unsigned)total), dim3(S::THREADS), 0, st, g);
  return launch_check();
}

template <int KIND>
hipError_t launch_product(Group& g, hipStream_t st) {
  // tiles of 128 x 128 where there are enough of them to fill the chip
  long long large = 0;
  for (int i = 0; i < g.count; i++) {
    const long long tm = tiles(g.m[i].mp, 128);
    large += KIND <= kPoly ? tm * (tm + 1) / 2 : tm * tiles(g.m[i].np, 128);
  }
  return large >= 128 ? launch_product<KIND, Large>(g, st) : launch_product<KIND, Small>(g, st);
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
  for (int i = 0; i < count; i++) n += (size_t)planes_bytes(make_mat(rows[i], cols[i]));
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
  long long at = 0;
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
    norm_start[i] = norm_groups;
    norm_groups += (int)(((long long)m.rows * m.cols + m.chunk - 1) / m.chunk);
    init_start[i] = init_groups;
    init_groups += tiles(m.mp, kTile) * tiles(m.np, kTile);
  }
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
