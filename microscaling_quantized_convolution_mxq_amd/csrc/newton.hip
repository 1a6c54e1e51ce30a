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
#pragma unroll 8
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

// What becomes of four sums down a column, (row .., col) of the product of kind KIND.
struct Last {
  bool tall;
  float keep, step;
  int real_m, real_n;
};
__device__ __forceinline__ Last last_of(const Group& g, const Mat& m) {
  const float lr = g.rate ? g.lr * *g.rate : g.lr;
  return Last{m.rows > m.cols, __builtin_fmaf(-lr, g.decay, 1.0f), -lr * m.scale, min(m.rows, m.cols), max(m.rows, m.cols)};
}
template <int KIND>
__device__ __forceinline__ void finish(const Group& g, const Mat& m, const Last& last, int row, int col, bool both, const float (&s)[4]) {
  const int mp = m.mp, np = m.np;
  if (row >= mp || col >= (KIND <= kPoly ? mp : np)) return;
  float v[4];
  if constexpr (KIND <= kPoly) {
    uint8_t* const to = a_of(g, m, KIND == kPoly ? 1 : 0);
    if constexpr (KIND == kGram) {
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] = s[e] * (1.0f / kUp);
    } else {
      // b A + c A^2, and a on the diagonal, so that the next product is a whole step (A is symmetric: its row is
      // read along the columns here)
      const uint8_t* const from = a_of(g, m, 0) + at_of(col, row, mp);
      const half4 hi = *reinterpret_cast<const half4*>(from), lo = *reinterpret_cast<const half4*>(from + 64);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const float a = (float)hi[e] + (float)lo[e];
        v[e] = __builtin_fmaf(g.b * 0.5f, a, s[e] * (g.c * (0.5f / kUp)));
        if (row + e == col && col < last.real_m) v[e] += g.a * (0.5f * kUp);
      }
    }
    store_across(to, mp, row, col, v);
    if (both) store_down(to, mp, row, col, v);
  } else if constexpr (KIND == kApply) {
#pragma unroll
    for (int e = 0; e < 4; e++) v[e] = s[e] * (2.0f / kUp);
    store_across(xt_of(g, m, g.from ^ 1), mp, row, col, v);
    store_down(x_of(g, m), np, row, col, v);
  } else {
    if (col >= last.real_n) return;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      if (row + e >= last.real_m) break;
      const long long i = last.tall ? (long long)col * m.cols + row + e : (long long)(row + e) * m.cols + col;
      const float o = s[e] * (2.0f / kUp / kUp);
      m.out[i] = g.update ? __builtin_fmaf(last.step, o, m.out[i] * last.keep) : o;
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
  const Last last = last_of(g, m);
  mma_results<S>(acc, wave, lane, [&](int r, int c, const float (&s)[4]) { finish<KIND>(g, m, last, i0 + r, j0 + c, both, s); });
}

// The slices' sums, added in order; a wave takes 32 x 32 of a tile.
template <int KIND, class S>
__global__ __launch_bounds__(256) void join_kernel(const Group g) {
  constexpr int PER = S::NW * S::TM * S::TN;  // parts of a tile
  const int lane = threadIdx.x & 63;
  int local;
  const int which = matrix_of(g, (int)blockIdx.x, local);
  const Mat& m = g.m[which];
  const int p = __builtin_amdgcn_readfirstlane(local * 4 + (threadIdx.x >> 6)), tile = p / PER, part = p - tile * PER;
  const int slices = g.slices[which];
  int i0, j0;
  bool both;
  place<KIND, S>(m, tile, i0, j0, both);
  const int wave = part / (S::TM * S::TN), ij = part - wave * (S::TM * S::TN), i = ij / S::TN, j = ij - i * S::TN;
  const int r0 = i0 + ((wave / S::WN) * S::TM + i) * 32, c0 = j0 + ((wave % S::WN) * S::TN + j) * 32;
  if (r0 >= m.mp || c0 >= (KIND <= kPoly ? m.mp : m.np)) return;  // (whole waves)
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
  const Last last = last_of(g, m);
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const float s[4] = {sum[e].x, sum[e].y, sum[e].z, sum[e].w};
    finish<KIND>(g, m, last, r0 + 8 * e + 4 * (lane >> 5), c0 + (lane & 31), both, s);
  }
}

// ---- plans --------------------------------------------------------------------------------------
// A matrix's tiles and slices are chosen by its own extents alone, so its
// result does not depend on what else a call holds.
typedef MmaShape<64, 64, 2, 2, 3> Small;        // several workgroups a compute unit
typedef MmaShape<64, 64, 2, 2, 4, 2> SmallLong; // for A's few tiles and long sums
typedef MmaShape<256, 128, 2, 2, 3> Wide;

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

struct Plan {
  bool wide;
  int tiles, slices;
};
template <int KIND>
Plan plan_of(const Mat& m) {
  const int steps = (KIND == kGram ? m.np : m.mp) / 32;
  Plan p{};
  p.wide = m.mp >= (KIND == kPoly ? 1536 : 512);
  if (p.wide) {
    // one workgroup a compute unit; slices of 16 steps at least
    p.tiles = tiles_of<KIND, Wide>(m);
    p.slices = std::max(1, std::min({256 / p.tiles, steps / 16, 32}));
  } else {
    p.tiles = KIND == kGram ? tiles_of<KIND, SmallLong>(m) : tiles_of<KIND, Small>(m);
    p.slices = std::max(1, std::min({256 / p.tiles, steps / 48, 32}));
  }
  return p;
}
template <int KIND>
long long part_of(const Mat& m) {  // float4 of its slices
  const Plan p = plan_of<KIND>(m);
  return p.slices == 1 ? 0 : (long long)p.tiles * p.slices * (p.wide ? Wide::BM * Wide::BN : Small::BM * Small::BN) / 4;
}
long long part_size(const Mat& m) { return std::max({part_of<kGram>(m), part_of<kPoly>(m), part_of<kApply>(m)}); }

template <int KIND, class S>
hipError_t launch_class(Group& g, bool wide, hipStream_t st) {
  int total = 0, join = 0, joins[kUpdateGroup];
  for (int i = 0; i < g.count; i++) {
    const Plan p = plan_of<KIND>(g.m[i]);
    const bool in = p.wide == wide;
    g.start[i] = total;
    g.tiles[i] = std::max(1, p.tiles);
    g.slices[i] = p.slices;
    total += in ? p.tiles * p.slices : 0;
    joins[i] = join;
    join += in && p.slices > 1 ? p.tiles * (S::NW * S::TM * S::TN / 4) : 0;
  }
  if (total == 0) return hipSuccess;
  g.start[g.count] = total;
  hipLaunchKernelGGL((newton_kernel<KIND, S>), dim3((unsigned)total), dim3(S::THREADS), 0, st, g);
  const hipError_t e = launch_check();
  if (e != hipSuccess || join == 0) return e;
  std::copy(joins, joins + g.count, g.start);
  g.start[g.count] = join;
  hipLaunchKernelGGL((join_kernel<KIND, S>), dim3((unsigned)join), dim3(256), 0, st, g);
  return launch_check();
}

template <int KIND>
hipError_t launch_product(Group& g, hipStream_t st) {
  const hipError_t e = launch_class<KIND, Wide>(g, true, st);
  if (e != hipSuccess) return e;
  if constexpr (KIND == kGram) return launch_class<KIND, SmallLong>(g, false, st);
  else return launch_class<KIND, Small>(g, false, st);
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
