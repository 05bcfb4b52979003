// group_common.h -- parts shared by the kernels of the products grouped by
// expert: the groups' rows, the tile hand-out, operand fragments and the
// layout of a tile in LDS.  Included by group_tile.h and
// group_kernels.h.
#pragma once

#include "gemm_tile.h"
#include "ops_internal.h"

namespace cco {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4_t;
typedef __attribute__((address_space(3))) const u32x4 lds_cu32x4_t;

// Rows [lo, lo + n) of group g that lie inside the row operands.
struct GroupRows {
  int64_t lo;
  int32_t n;
};
__device__ __forceinline__ GroupRows group_rows(const GroupArgs &a, int g) {
  int64_t lo = a.first[g], hi = lo + a.count[g];
  if (lo < 0) lo = 0;
  if (hi > a.rows) hi = a.rows;
  return {lo, hi > lo ? (int32_t)(hi - lo) : 0};
}

// Tiles per group and their prefix over the groups, spread over NT threads:
// thread t holds groups t * PER ...  No workspace and no queue: every
// workgroup computes the prefix for itself (about a microsecond, the counts
// come from L2) and takes every gridDim-th tile, so a call keeps no state.
template <int NT>
struct TileMap {
  static constexpr int PER = (kMaxGroups + NT - 1) / NT;
  int64_t pre[PER];
  int32_t loc[PER];
  int64_t total;

  // units(rows): tiles of a group.  scratch: NT / kWave int64 in LDS.
  template <class F>
  __device__ __forceinline__ void init(const GroupArgs &a, int64_t *scratch, F &&units) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    int64_t sum = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int g = tid * PER + q;
      loc[q] = g < a.groups ? units(group_rows(a, g).n) : 0;
      sum += loc[q];
    }
    int64_t incl = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int64_t up = __shfl_up((long long)incl, d, kWave);
      if (lane >= d) incl += up;
    }
    if (lane == kWave - 1) scratch[wave] = incl;
    __syncthreads();
    int64_t run = incl - sum;
    total = 0;
    for (int w = 0; w < NT / kWave; ++w) {
      const int64_t wt = scratch[w];
      if (w < wave) run += wt;
      total += wt;
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      pre[q] = run;
      run += loc[q];
    }
    __syncthreads();
  }

  // Group and tile-in-group of tile L < total (every thread gets them).
  __device__ __forceinline__ void find(int64_t L, int32_t *scratch, int &g, int &r) const {
    __syncthreads();  // the scratch's last use is over
#pragma unroll
    for (int q = 0; q < PER; ++q)
      if (L >= pre[q] && L < pre[q] + loc[q]) {
        scratch[0] = threadIdx.x * PER + q;
        scratch[1] = (int32_t)(L - pre[q]);
      }
    __syncthreads();
    g = uniform(scratch[0]);
    r = uniform(scratch[1]);
    __syncthreads();
  }
};

// The operands' elements and the sums they give.  8-bit ones stand two to
// each 16 bits of the reduction: the same bytes in the same places.
enum GroupElem { kElemBf16, kElemF16, kElemI8 };
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
template <GroupElem EL>
struct GroupAcc {
  using type = f32x16;
};
template <>
struct GroupAcc<kElemI8> {
  using type = i32x16;
};

// One MFMA, C^T += B A^T: lane l ends up with row l % 32 of the block and
// columns 8 (v / 4) + 4 (l / 32) + v % 4.
template <GroupElem EL>
__device__ __forceinline__ typename GroupAcc<EL>::type group_mfma(
    u32x4 b, u32x4 a, typename GroupAcc<EL>::type c) {
  if constexpr (EL == kElemI8)
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, b),
                                                 __builtin_bit_cast(i32x4, a), c, 0, 0, 0);
  else if constexpr (EL == kElemF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, b),
                                                  __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b),
                                                   __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
}

// An 8-bit product's result in fp32, the same in every kernel.  (Left to
// itself the compiler rounds the last product and the conversion to fp16 at
// once in some of them.)
__device__ __forceinline__ float scaled_sum(float sum, float row, float column) {
  float v = sum * row * column;
  asm("" : "+v"(v));
  return v;
}

template <bool F16>
__device__ __forceinline__ uint16_t to_half_bits(float v) {
  if constexpr (F16)
    return __builtin_bit_cast(uint16_t, (_Float16)v);
  else
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}
// Two values, rounded to nearest even.
template <bool F16>
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  return (uint32_t)to_half_bits<F16>(lo) | ((uint32_t)to_half_bits<F16>(hi) << 16);
}
template <bool F16>
__device__ __forceinline__ float from_half_bits(uint16_t v) {
  if constexpr (F16)
    return (float)__builtin_bit_cast(_Float16, v);
  else
    return (float)__builtin_bit_cast(__bf16, v);
}

// A tile's operand in LDS, unpadded, in 16-byte chunks.
//  k-contiguous operand: [rows][64 k], chunk c of row r at c ^ swz<8>(r)
//    (the 16 rows of a fragment read fall on distinct banks);
//  k-major operand: [64 k][W columns]; a fragment takes 4 k of 32 columns
//    per transposing read, so the four k rows, whose pitch is a multiple of
//    all banks, must not share banks: chunk c of row k at c ^ kswz(k), which
//    moves the rows to distinct 64-byte segments (and distinct 32-byte ones
//    mod 128).
__device__ __forceinline__ int kswz(int k) { return ((k & 1) ? 4 : 0) ^ ((k & 2) ? 10 : 0); }

// ds_read_b64_tr_b16: within 16 lanes, lane s reads 4 columns of k row
// s / 4; lane l gets column l of the 16 at k 0..3 of the 4 rows.
// (The restrict pointer gives the read alias information.  Without any, the
// compiler takes it to depend on every direct load into LDS in flight and
// waits for all of them before each read; the kernels order the two with
// explicit waits.)
__device__ __forceinline__ u32x2 read_tr(lds_s16x4_t *__restrict__ p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}
__device__ __forceinline__ u32x2 lds_read_tr(uint32_t addr) {
  return read_tr((lds_s16x4_t *)(uintptr_t)addr);
}

// Byte offset in LDS of this lane's fragment reads of 32 columns starting at
// column col0 of a k-major tile of W columns, k rows k0 + 0..3 of each lane
// half's eight (k0 16 times the sub-step); the rows 4..7 are 4 W columns on.
template <int W>
__device__ __forceinline__ uint32_t kmajor_offset(int lane, int col0) {
  const int s = lane & 15;
  const int k = (lane >> 5) * 8 + (s >> 2);           // row of the 16
  const int col = col0 + ((lane >> 4) & 1) * 16 + (s & 3) * 4;
  const int chunk = (col >> 3) ^ kswz(k);
  return (uint32_t)(k * W * 2 + chunk * 16 + (col & 7) * 2);
}

}  // namespace
}  // namespace cco
