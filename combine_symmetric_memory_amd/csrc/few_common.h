// few_common.h -- parts shared by the two forms of the layer for a few tokens
// (moe_few.hip, moe_few_shared.hip): the ids and the experts in use, an
// expert's tokens, and one step of a product of weight rows with tokens.
#pragma once

#include <type_traits>

#include "group_common.h"

namespace cco {
namespace {

constexpr int kFewRows = 16;       // weight rows of an MFMA
constexpr int kFewStepBytes = 64;  // bytes of a weight row a step takes

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Global memory.  (Through a pointer that was put together from two scalar
// registers the compiler knows no address space and makes flat loads, which
// LDS reads then wait for.)
typedef __attribute__((address_space(1))) const char GlobalBytes;
typedef u32x4 u32x4_any __attribute__((aligned(1)));
__device__ __forceinline__ GlobalBytes *uniform_bytes(const void *p) {
  return (GlobalBytes *)(uintptr_t)uniform((const char *)p);
}
__device__ __forceinline__ u32x4 load16(GlobalBytes *p) {
  return *(const __attribute__((address_space(1))) u32x4_any *)p;
}
// 16 bytes at p, of which the first `have` exist; the others are zeros.
__device__ __forceinline__ u32x4 load16(GlobalBytes *p, int have) {
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (int i = min(have, 16) - 1; i >= 0; --i) {
    hi = (hi << 8) | (lo >> 56);
    lo = (lo << 8) | (uint8_t)p[i];
  }
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}
// The 16 bytes at `at` of a row of `bytes` out of 16 loaded from there or, so
// as to lie inside the row, from bytes - 16: what is behind the end is zeros.
__device__ __forceinline__ u32x4 end_cut(u32x4 v, int at, int bytes) {
  const int sh = min(max(0, at + 16 - bytes), 16) * 8;  // bits behind the end
  uint64_t lo = v.x | ((uint64_t)v.y << 32), hi = v.z | ((uint64_t)v.w << 32);
  if (sh & 64) {
    lo = hi;
    hi = 0;
  }
  if (sh & 63) {
    lo = (lo >> (sh & 63)) | (hi << (64 - (sh & 63)));
    hi >>= sh & 63;
  }
  if (sh >= 128) lo = hi = 0;
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// The ids and weights of a call in LDS, and the experts in use: `words` of 32
// bits in all.
struct FewIds {
  uint32_t *live;  // [kMaxExperts / 32], a bit an expert
  int32_t *ids;    // [T][K]
  float *w;
  static __host__ __device__ constexpr int words(int pairs) {
    return kMaxExperts / 32 + 2 * pairs;
  }
  __device__ __forceinline__ FewIds(uint32_t *lds, int pairs)
      : live(lds), ids((int32_t *)lds + kMaxExperts / 32), w((float *)ids + pairs) {}
};

template <int THREADS>
__device__ __forceinline__ void few_read_ids(const FewArgs &a, const FewIds &s) {
  for (int i = threadIdx.x; i < kMaxExperts / 32; i += THREADS) s.live[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * a.K; i += THREADS) {
    const int e = a.idx[i];
    s.ids[i] = e;
    s.w[i] = a.w[i];
    if (e >= 0 && e < a.E) atomicOr(&s.live[e / 32], 1u << (e % 32));
  }
  __syncthreads();
}

// The experts in use, in ascending order: how many, and the one of rank a.
struct FewExperts {
  int count;
  int before;  // lane l: experts in use below 32 l
  uint32_t word;
  __device__ __forceinline__ explicit FewExperts(const FewIds &s) {
    const int lane = threadIdx.x % kWave;
    word = lane < kMaxExperts / 32 ? s.live[lane] : 0u;
    const int n = __popc(word);
    int incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up(incl, d, kWave);
      if (lane >= d) incl += up;
    }
    before = incl - n;
    count = uniform(__shfl(incl, kMaxExperts / 32 - 1, kWave));
  }
  __device__ __forceinline__ int at(int rank) const {
    const int lane = threadIdx.x % kWave;
    const uint64_t hit = __ballot(rank >= before && rank < before + __popc(word));
    const int l = __builtin_ctzll(hit);
    uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)word, l);
    for (int k = rank - __builtin_amdgcn_readlane(before, l); k > 0; --k) w &= w - 1;
    return uniform(l * 32 + __builtin_ctz(w));
  }
};

// An expert's tokens, in ascending order.
struct FewTokens {
  int count;
  int pair;  // lane n < count: first pair (token * K + j) of the n-th token ..
  float share;  // .. and the sum of its weights for the expert
  __device__ __forceinline__ void find(const FewArgs &a, const FewIds &s, int e) {
    const int lane = threadIdx.x % kWave;
    int first = -1;
    float sum = 0.0f;
    if (lane < a.T)
      for (int j = a.K - 1; j >= 0; --j)
        if (s.ids[lane * a.K + j] == e) first = lane * a.K + j;
    if (first >= 0)
      for (int p = first; p < (lane + 1) * a.K; ++p)
        if (s.ids[p] == e) sum = p == first ? s.w[p] : sum + s.w[p];
    const uint64_t mask = __ballot(first >= 0), below = (1ull << lane) - 1;
    count = uniform(__popcll(mask));
    // lane t's values go to the lane of its rank, other lanes' behind them
    const int to = first >= 0 ? __popcll(mask & below) : count + __popcll(~mask & below);
    pair = __builtin_amdgcn_ds_permute(to * 4, first);
    share = __builtin_bit_cast(
        float, __builtin_amdgcn_ds_permute(to * 4, __builtin_bit_cast(int, sum)));
  }
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// Two bf16 halves of the top 16 bits of a and b.
__device__ __forceinline__ uint32_t top_halves(float a, float b) {
  return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a),
                               0x07060302u);
}
// Eight 8-bit integers as bf16 or fp16 values, exact in both.
template <bool F16>
__device__ __forceinline__ u32x4 from_i8(uint32_t lo, uint32_t hi) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? lo : hi;
    const int sh = 16 * (i % 2);
    const float a = (float)(int8_t)(w >> sh), b = (float)(int8_t)(w >> (sh + 8));
    if constexpr (F16)
      r[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
    else
      r[i] = top_halves(a, b);
  }
  return r;
}
// Eight fp16 values as the sum of two bf16 ones, exactly: the high one is the
// value to nearest, which leaves at most 2^-8 of it, in three bits.
__device__ __forceinline__ void split_f16(u32x4 v, u32x4 &hi, u32x4 &lo) {
  const f16x8 h = __builtin_bit_cast(f16x8, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = (float)h[2 * i], b = (float)h[2 * i + 1];
    hi[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
    const float ah = __builtin_bit_cast(float, hi[i] << 16);
    const float bh = __builtin_bit_cast(float, hi[i] & 0xffff0000u);
    lo[i] = top_halves(a - ah, b - bh);
  }
}

// acc[n] += one step of a tile of weight rows with column tile n.  EL: the
// weights' elements.  PAIR: the columns are h, in two planes; otherwise x, of
// the weights' type or, with 8-bit weights, fp16 (XF16) or bf16.  A step of
// 8-bit weights takes two 16-byte pieces of a column (and plane).
template <GroupElem EL, bool PAIR, bool XF16, int NT, int NB>
__device__ __forceinline__ void few_multiply(f32x4 (&acc)[NT], u32x4 w,
                                           const u32x4 (&col)[NT][NB]) {
  constexpr bool F = XF16 && !PAIR;
  using V = std::conditional_t<F, f16x8, bf16x8>;
  auto mma = [&](int n, u32x4 x, u32x4 y) __attribute__((always_inline)) {
    acc[n] = mfma16(__builtin_bit_cast(V, x), __builtin_bit_cast(V, y), acc[n]);
  };
  // Weights are converted where they are multiplied.  (Left to itself the
  // compiler takes the loaded vectors apart into bytes and converts them all
  // ahead, which spills.)
  if constexpr (EL == kElemI8 || (EL == kElemF16 && PAIR)) asm volatile("" : "+v"(w));
  if constexpr (EL == kElemI8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 f = from_i8<F>(w[2 * h], w[2 * h + 1]);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < (PAIR ? 2 : 1); ++p) mma(n, f, col[n][p * 2 + h]);
    }
  } else if constexpr (EL == kElemF16 && PAIR) {
    u32x4 hi, lo;
    split_f16(w, hi, lo);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // (the product of the two low parts, 2^-8 of each, is at most 2^-16 of
      // the whole)
      mma(n, hi, col[n][0]);
      mma(n, hi, col[n][1]);
      mma(n, lo, col[n][0]);
    }
  } else {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int p = 0; p < NB; ++p) mma(n, w, col[n][p]);
  }
}

// h as two bf16 values, h = hi + lo to 2^-17 of it.  Where h itself is finite
// and would round to an infinity, bf16's largest value is the high part; an
// infinite or NaN h is whole in it.
__device__ __forceinline__ void few_split(float h, uint16_t &hi, uint16_t &lo) {
  hi = f32_to_bf16_rne(h);
  if (__builtin_fabsf(h) < __builtin_inff() && (hi & 0x7fff) == 0x7f80) --hi;
  const float left = h - from_half_bits<false>(hi);
  lo = __builtin_fabsf(left) < __builtin_inff() ? f32_to_bf16_rne(left) : 0;
}

}  // namespace
}  // namespace cco
