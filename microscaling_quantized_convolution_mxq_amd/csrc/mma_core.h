// mma_core.h -- the K loop shared by the 16-bit matrix products: the two-level
// products (bf16 operands) and the Newton-Schulz products (fp32 values as two
// f16 planes).
//
// C[i][j] = sum_k A[i][k] B[j][k]. Both operands are rows with k contiguous,
// read in steps of 128 bytes of every row:
//   Bf16:   64 values;
//   Split:  32 values as 32 f16 high parts, then their 32 low parts:
//           a = ah + al with ah = f16(a), al = f16(a - ah), off by at most 2^-22
//           of a, or by 2^-25 where that is more (f16's smallest values are 2^-24
//           apart), a b = ah bh + ah bl + al bh (al bl, below 2^-22 of it, is left out).
// A step of a tile is [row][8] chunks of 16 bytes in LDS, written by loads that
// go to LDS directly. Chunk c of row r is in slot c ^ ((r >> 1) & 7): a row is
// half of the 64 banks, so the sixteen rows that an operand read touches at one
// time lie in sixteen different groups of four banks.
// ST stages form a ring: one barrier a step, after which the stage that was
// read in the step before is filled again.
#pragma once
#include <type_traits>

#include "mx_common.h"

namespace mq {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bhalf8 __attribute__((ext_vector_type(8)));

constexpr int kPiece = 128;         // bytes of a row in a step
constexpr int kBeyond = 0x7fffff00; // an offset past the end of every buffer: such loads write zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mma_rsrc(const void* p, long long bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(bytes < kBeyond ? bytes : kBeyond),
                                           0x00020000);
}

typedef __attribute__((address_space(3))) void* mma_lds_t;
// 16 bytes a lane from voff + soff to lds + 16 * lane
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (mma_lds_t)lds, 16, voff, soff, 0, 0);
}

// Waits until at most N of this wave's loads are under way and its LDS reads
// are done, then for the other waves. (No memory fence: the wait is explicit,
// and the empty asm statements keep LDS accesses on their side.)
template <int N>
__device__ __forceinline__ void stage_ready() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The same for LDS accesses alone: loads stay under way.
__device__ __forceinline__ void lds_ready() {
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A workgroup's tile: BM x BN outputs by WM x WN waves, a ring of ST stages. NG
// groups of waves each take a part of the steps in a ring of their own, and
// group 0 adds their sums: with few tiles, a tile's loads and products come from
// more waves.
template <int BM_, int BN_, int WM_, int WN_, int ST_, int NG_ = 1>
struct MmaShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_, NG = NG_;
  static constexpr int NW = WM * WN, THREADS = 64 * NW * NG;  // NW: waves of a group
  static constexpr int TM = BM / WM / 32, TN = BN / WN / 32;  // a wave's 32 x 32 products
  static constexpr int STAGE = (BM + BN) * kPiece, LDS = ST * STAGE * NG;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;     // loads of a wave and step
  static_assert(LA >= 1 && LB >= 1 && TM >= 1 && TN >= 1, "tile");
  static_assert(NG == 1 || BM * BN * 4 * (NG - 1) <= LDS, "the groups' sums fit the rings");
};

// What a lane loads: load j of wave w covers the eight rows from 8 (w + NW j)
// on, the lane row + lane / 8, and of that the chunk of eight-row block w + NW j;
// with an even number of waves the chunk is the same in all loads.
__device__ __forceinline__ int lane_chunk(int wave, int lane) { return (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7); }
template <int NW>
__device__ __forceinline__ int lane_row(int wave, int lane, int j) {
  return 8 * (wave + NW * j) + (lane >> 3);
}

// Rows of a matrix with k contiguous.
template <int L, int NW>
struct RowLoader {
  __amdgpu_buffer_rsrc_t rsrc;
  int off[L];
  __device__ void init(const void* p, long long bytes, int row0, int rows, int pitch, int wave, int lane) {
    rsrc = mma_rsrc(p, bytes);
#pragma unroll
    for (int j = 0; j < L; j++) {
      const int r = row0 + lane_row<NW>(wave, lane, j);
      off[j] = r < rows ? r * pitch + lane_chunk(wave + NW * j, lane) * 16 : kBeyond;
    }
  }
  __device__ void issue(int step, uint8_t* lds, int wave) const {
#pragma unroll
    for (int j = 0; j < L; j++) load_lds16(rsrc, lds + (wave + NW * j) * 1024, off[j], step * kPiece);
  }
};

struct Bf16 {};
struct Split {};

template <class S>
__device__ __forceinline__ void mma_zero(v16f (&acc)[S::TM][S::TN]) {
#pragma unroll
  for (int i = 0; i < S::TM; i++)
#pragma unroll
    for (int j = 0; j < S::TN; j++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
}
template <class S>
__device__ __forceinline__ void mma_add(v16f (&a)[S::TM][S::TN], const v16f (&b)[S::TM][S::TN]) {
#pragma unroll
  for (int i = 0; i < S::TM; i++)
#pragma unroll
    for (int j = 0; j < S::TN; j++, __builtin_amdgcn_sched_barrier(0)) a[i][j] += b[i][j];
}

// What the products of 16 values of k take: rows of A and of B^T, high (and low) parts.
template <class T, int TM, int TN>
struct Frags {
  static constexpr bool SPLIT = std::is_same<T, Split>::value;
  typedef typename std::conditional<SPLIT, half8, bhalf8>::type vec;
  static constexpr int KK = SPLIT ? 2 : 4;  // of a step
  vec x[TM], y[TN], xl[SPLIT ? TM : 1], yl[SPLIT ? TN : 1];
  __device__ __forceinline__ void read(const uint8_t* ar, const uint8_t* br, int kk, int q, int sw) {
    const int hi = ((2 * kk + q) ^ sw) << 4;
#pragma unroll
    for (int i = 0; i < TM; i++) x[i] = *reinterpret_cast<const vec*>(ar + 32 * i * kPiece + hi);
#pragma unroll
    for (int j = 0; j < TN; j++) y[j] = *reinterpret_cast<const vec*>(br + 32 * j * kPiece + hi);
    if constexpr (SPLIT) {
      const int lo = ((4 + 2 * kk + q) ^ sw) << 4;
#pragma unroll
      for (int i = 0; i < TM; i++) xl[i] = *reinterpret_cast<const vec*>(ar + 32 * i * kPiece + lo);
#pragma unroll
      for (int j = 0; j < TN; j++) yl[j] = *reinterpret_cast<const vec*>(br + 32 * j * kPiece + lo);
    }
  }
  template <int LM, int LN>
  __device__ __forceinline__ void multiply(v16f (&acc)[TM][TN], v16f (&low)[LM][LN]) const {
    if constexpr (SPLIT) {
#pragma unroll
      for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) low[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xl[i], y[j], low[i][j], 0, 0, 0);
#pragma unroll
      for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) low[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[i], yl[j], low[i][j], 0, 0, 0);
#pragma unroll
      for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[i], y[j], acc[i][j], 0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[i], y[j], acc[i][j], 0, 0, 0);
    }
  }
};

// A wave's place: its group, and its number in the group.
template <class S>
struct MmaWave {
  int lane, wave, group;
  __device__ MmaWave() {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lane = threadIdx.x & 63;
    group = S::NG == 1 ? 0 : w / S::NW;
    wave = S::NG == 1 ? w : w - group * S::NW;
  }
  // the group's part [s0, s0 + n) of `steps`
  __device__ int first(int steps) const { return (int)((long long)steps * group / S::NG); }
  __device__ int count(int steps) const { return first_of(steps, group + 1) - first(steps); }
  __device__ static int first_of(int steps, int g) { return (int)((long long)steps * g / S::NG); }
  // the most steps of a group
  __device__ static int most(int steps) { return (steps + S::NG - 1) / S::NG; }
};

// One step's products; acc, and for Split `low`: sums of the products of a high and a low part.
template <class T, int TM, int TN, int LM, int LN>
__device__ __forceinline__ void mma_step(const uint8_t* a, const uint8_t* b, int lane, v16f (&acc)[TM][TN],
                                         v16f (&low)[LM][LN]) {
  const int r = lane & 31, q = lane >> 5, sw = (r >> 1) & 7;
#pragma unroll
  for (int kk = 0; kk < Frags<T, TM, TN>::KK; kk++) {
    Frags<T, TM, TN> f;
    f.read(a + r * kPiece, b + r * kPiece, kk, q, sw);
    f.multiply(acc, low);
  }
}

// The n steps from step0 on of a group's part of a tile; `most`: the most steps
// of any group, which all go through together. Group 0 has the sums. Loaders: issue(step, lds, wave)
// makes L loads of every wave, whatever the step is.
//
// The matrix units align the 16 products of an instruction to the largest of
// them and the accumulator, and drop what lies below 2^-26 of that (measured: 1
// + 16 x 2^-27 stays 1, 1 + 4 x 2^-25 does not). The products with a low part
// are 2^-11 of the others, so they have accumulators of their own, and the two
// are added at the end.
template <class T, class S, class LA, class LB>
__device__ __forceinline__ void mma_loop(uint8_t* ring, LA& la, LB& lb, int step0, int n, int most, const MmaWave<S>& me,
                                         v16f (&acc)[S::TM][S::TN]) {
  const int wave = me.wave, lane = me.lane;
  uint8_t* const lds = ring + me.group * (S::ST * S::STAGE);
  constexpr int ST = S::ST, LPS = S::LA + S::LB;
  const int wm = wave / S::WN, wn = wave % S::WN;
  auto issue = [&](int s, int slot) {
    uint8_t* const to = lds + slot * S::STAGE;
    la.issue(step0 + s, to, wave);
    lb.issue(step0 + s, to + S::BM * kPiece, wave);
  };
#pragma unroll
  for (int s = 0; s < ST - 1; s++)
    if (s < n) issue(s, s);
  int slot = 0, fill = ST - 1;
  constexpr bool LOW = std::is_same<T, Split>::value;
  v16f low[LOW ? S::TM : 1][LOW ? S::TN : 1];
  if constexpr (LOW) mma_zero<S>(low);
  for (int s = 0; s < most; s++) {
    // step s has arrived once only the ST - 2 steps behind it are under way
    if (s + ST - 2 < n) stage_ready<(ST - 2) * LPS>();
    else stage_ready<0>();
    if (s + ST - 1 < n) issue(s + ST - 1, fill);
    const uint8_t* const at = lds + slot * S::STAGE;
    if (S::NG == 1 || s < n) mma_step<T, S::TM, S::TN>(at + wm * S::TM * 32 * kPiece, at + (S::BM + wn * S::TN * 32) * kPiece, lane, acc, low);
    slot = slot + 1 == ST ? 0 : slot + 1;
    fill = fill + 1 == ST ? 0 : fill + 1;
  }
  if constexpr (LOW) mma_add<S>(acc, low);
  if constexpr (S::NG > 1) {
    // the other groups leave their sums in LDS, lane by lane
    float* const sums = reinterpret_cast<float*>(ring);
    constexpr int PER = S::TM * S::TN * 16 * 64, ALL = PER * S::NW;  // floats of a wave and of a group
    stage_ready<0>();
    if (me.group > 0) {
      float* const to = sums + (me.group - 1) * ALL + wave * PER + lane * 4;
#pragma unroll
      for (int i = 0; i < S::TM; i++)
#pragma unroll
        for (int j = 0; j < S::TN; j++)
#pragma unroll
          for (int e = 0; e < 4; e++)
            *reinterpret_cast<float4*>(to + ((i * S::TN + j) * 4 + e) * 256) =
                make_float4(acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]);
    }
    stage_ready<0>();
    if (me.group == 0) {
#pragma unroll
      for (int g = 0; g < S::NG - 1; g++) {
        const float* const from = sums + g * ALL + wave * PER + lane * 4;
#pragma unroll
        for (int i = 0; i < S::TM; i++)
#pragma unroll
          for (int j = 0; j < S::TN; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const float4 v = *reinterpret_cast<const float4*>(from + ((i * S::TN + j) * 4 + e) * 256);
              acc[i][j][4 * e] += v.x;
              acc[i][j][4 * e + 1] += v.y;
              acc[i][j][4 * e + 2] += v.z;
              acc[i][j][4 * e + 3] += v.w;
            }
      }
    }
  }
}

// The same for one wave a SIMD with large tiles of its own (128 x 64 and more),
// which read each operand fewer times.
// With no second wave to fill in, the operands of the next 16 values of k are
// read while the present ones are multiplied, over the barrier too: it stands
// before the last products of a step, and what they read is in registers. n is
// at least 1.
template <class T, class S, class LA, class LB>
__device__ __forceinline__ void mma_loop_wide(uint8_t* lds, LA& la, LB& lb, int step0, int n, const MmaWave<S>& me,
                                              v16f (&acc)[S::TM][S::TN]) {
  constexpr int ST = S::ST, LPS = S::LA + S::LB, KK = Frags<T, S::TM, S::TN>::KK;
  constexpr bool LOW = std::is_same<T, Split>::value;
  static_assert(KK % 2 == 0 && S::NG == 1, "operand buffers alternate");
  const int wave = me.wave, lane = me.lane;
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int r = lane & 31, q = lane >> 5, sw = (r >> 1) & 7;
  const int ao = (wm * S::TM * 32 + r) * kPiece, bo = (S::BM + wn * S::TN * 32 + r) * kPiece;
  v16f low[LOW ? S::TM : 1][LOW ? S::TN : 1];
  if constexpr (LOW) mma_zero<S>(low);
  auto issue = [&](int s, int slot) {
    uint8_t* const to = lds + slot * S::STAGE;
    la.issue(step0 + s, to, wave);
    lb.issue(step0 + s, to + S::BM * kPiece, wave);
  };
  // Loads past the last step fill stages that nothing reads, so every step is the same straight line.
#pragma unroll
  for (int s = 0; s < ST; s++) issue(s, s);
  stage_ready<(ST - 1) * LPS>();
  Frags<T, S::TM, S::TN> f[2];
  f[0].read(lds + ao, lds + bo, 0, q, sw);
  constexpr int NR = (S::TM + S::TN) * (LOW ? 2 : 1), NM = S::TM * S::TN * (LOW ? 3 : 1), REST = NM - NR;
  int slot = 0, s = 0;
  do {
    const uint8_t* const at = lds + slot * S::STAGE;
    const int next = slot + 1 == ST ? 0 : slot + 1;
#pragma unroll
    for (int kk = 0; kk + 1 < KK; kk++) {
      f[(kk + 1) & 1].read(at + ao, at + bo, kk + 1, q, sw);
      f[kk & 1].multiply(acc, low);
#pragma unroll
      for (int k = 0; k < NR; k++) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // a read of LDS,
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
      }
      __builtin_amdgcn_sched_group_barrier(0x008, REST, 0);
    }
    // all of this step is in registers, here and after the barrier everywhere: its stage is filled again
    stage_ready<(ST - 2) * LPS>();
    f[0].read(lds + next * S::STAGE + ao, lds + next * S::STAGE + bo, 0, q, sw);
    issue(s + ST, slot);
    f[(KK - 1) & 1].multiply(acc, low);
#pragma unroll
    for (int k = 0; k < NR; k++) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
#pragma unroll
    for (int k = 0; k < REST; k++) {
      __builtin_amdgcn_sched_group_barrier(0x020, (LPS + REST - 1) / REST, 0);  // loads
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    slot = next;
  } while (++s < n);
  stage_ready<0>();  // (the ring is free, and no load is under way at the end)
  if constexpr (LOW) mma_add<S>(acc, low);
}

// Workgroups go to the eight XCDs in turn; this gives each XCD a contiguous
// range of the n tiles, which share operand rows in its L2.
__device__ __forceinline__ int xcd_tile(int b, int n) {
  const int x = b & 7, i = b >> 3, q = n >> 3, r = n & 7;
  return x * q + min(x, r) + i;
}

}  // namespace mq
