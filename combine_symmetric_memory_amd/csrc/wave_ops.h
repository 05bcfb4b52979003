// wave_ops.h -- reductions over the 64 lanes of a wavefront by data-parallel
// moves: pairs, quads, halves of 16 and 16 lanes, then the four rows of 16
// through scalar registers.  No LDS round trips, a fixed order, and the
// result is wavefront-uniform.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cco {
namespace {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, ((uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32) |
                                        dpp<CTRL>((uint32_t)u));
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int l) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, l);
}
__device__ __forceinline__ float lane_value(float v, int l) {
  return __builtin_bit_cast(float, lane_value(__builtin_bit_cast(uint32_t, v), l));
}
__device__ __forceinline__ uint64_t lane_value(uint64_t v, int l) {
  return ((uint64_t)lane_value((uint32_t)(v >> 32), l) << 32) | lane_value((uint32_t)v, l);
}
__device__ __forceinline__ double lane_value(double v, int l) {
  return __builtin_bit_cast(double, lane_value(__builtin_bit_cast(uint64_t, v), l));
}

template <class T, class Op>
__device__ __forceinline__ T wave_reduce(T v, Op op) {
  v = op(v, dpp<0xB1>(v));   // quad_perm 1 0 3 2
  v = op(v, dpp<0x4E>(v));   // quad_perm 2 3 0 1
  v = op(v, dpp<0x141>(v));  // mirror within 8
  v = op(v, dpp<0x140>(v));  // mirror within 16
  return op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
}
template <class T>
__device__ __forceinline__ T wave_total(T v) {
  return wave_reduce(v, [](T a, T b) { return a + b; });
}
__device__ __forceinline__ float wave_largest(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ uint32_t wave_largest(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint32_t wave_smallest(uint32_t v) {
  return wave_reduce(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

}  // namespace
}  // namespace cco
