// quant.hip -- rows to 8-bit integers with one scale a row, as they are or
// through SwiGLU (include/cco_ops.h):
//
//   v = x[r]  or  silu(x[r][c]) * x[r][cols + c]
//   s = max |v| / 127,  q = rint(127 v / max |v|)
//
// Rounded as the exact quotient is: the product with the inverse of the
// largest value is within 2^-16 of it, and where that lies next to a tie the
// sign of 127 v - (q +- 1/2) max |v| decides, exact in 64 bits.  (Ties are not
// rare in 16-bit rows: half the largest value is one.)
//
// Memory-bound: a row is read once, held in registers while its largest value
// is found, and written.  NT threads a row with NV groups of eight; a row that
// fits no form is read twice.
#include <type_traits>

#include "ops_internal.h"
#include "wave_ops.h"

namespace cco {
namespace {

constexpr int kQuantThreads = 256;

__device__ __forceinline__ float quant_silu(float z) {
  return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// Eight elements from p, whatever its alignment.
template <class T>
__device__ __forceinline__ void load8(float (&v)[8], const T *p) {
  struct {
    T e[8];
  } raw;
  __builtin_memcpy(&raw, p, sizeof(raw));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)raw.e[i];
}

// Values c .. c + 7 of a row (n: how many of them exist, 8 unless SHORT).
template <class T, bool SWIGLU, bool SHORT>
__device__ __forceinline__ void row_values(float (&v)[8], const T *row, int cols, int c, int n) {
  if constexpr (SHORT) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = min(i, n - 1);
      v[i] = (float)row[at];
      if constexpr (SWIGLU) v[i] = quant_silu(v[i]) * (float)row[cols + at];
    }
  } else {
    load8(v, row + c);
    if constexpr (SWIGLU) {
      float u[8];
      load8(u, row + cols + c);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = quant_silu(v[i]) * u[i];
    }
  }
}

__device__ __forceinline__ uint32_t magnitude(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
}

// A row's factors.  As integers magnitudes order like the values, infinities
// and NaN above them.
struct RowScale {
  float top, lift, inv;
  bool ok;
  __device__ __forceinline__ RowScale(uint32_t most) {
    ok = most != 0 && most < 0x7f800000u;
    top = __builtin_bit_cast(float, most);
    // rows far below one are lifted, so that the inverse exists
    lift = top < 0x1p-60f ? 0x1p64f : 1.0f;
    inv = ok ? 127.0f / (top * lift) : 0.0f;
  }
  __device__ __forceinline__ float scale() const {
    return __builtin_bit_cast(uint32_t, top) >= 0x7f800000u ? __builtin_nanf("") : top / 127.0f;
  }
  __device__ __forceinline__ int quant(float v) const {
    if (!ok) return 0;
    const float t = v * lift * inv;
    float k = __builtin_rintf(t);
    if (__builtin_fabsf(t - k) > 0.499f) {
      const double r = 127.0 * (double)v - (double)k * (double)top;
      const double twice = 2.0 * __builtin_fabs(r);
      if (twice > (double)top || (twice == (double)top && ((int)k & 1)))
        k += r < 0.0 ? -1.0f : 1.0f;
    }
    return (int)k;
  }
};

__device__ __forceinline__ void store8(int8_t *q, const float (&v)[8], const RowScale &rs) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[h] |= ((uint32_t)rs.quant(v[4 * h + i]) & 0xffu) << (8 * i);
  }
  __builtin_memcpy(q, w, 8);
}

// The largest magnitude over the NT threads of a row.
template <int NT>
__device__ __forceinline__ uint32_t row_largest(uint32_t m, uint32_t *lds) {
  m = wave_largest(m);
  if constexpr (NT > kWave) {
    __syncthreads();  // the last row's are read
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / kWave; ++w) m = max(m, lds[w]);
  }
  return m;
}

// NV > 0: the row fits NT * NV groups of eight.  A group that would pass the
// row's end starts eight before it: its values are computed and written twice,
// alike.  SHORT (with NV 0): fewer than eight columns, a thread a row.
template <class T, bool SWIGLU, int NT, int NV, bool SHORT>
__global__ __launch_bounds__(kQuantThreads) void quant_kernel(QuantArgs a) {
  __shared__ uint32_t lds[kQuantThreads / kWave];
  constexpr int PER = SHORT ? kQuantThreads : kQuantThreads / NT;  // rows a workgroup
  const int at = SHORT ? 0 : threadIdx.x % NT;
  const int groups = (a.cols + 7) / 8;
  for (int64_t r = (int64_t)blockIdx.x * PER + threadIdx.x / (SHORT ? 1 : NT); r < a.rows;
       r += (int64_t)gridDim.x * PER) {
    const T *row = (const T *)a.x + r * a.ldx;
    int8_t *q = a.q + r * a.ldq;
    float *s = a.s + r * a.lds;
    if constexpr (SHORT) {
      float v[8];
      row_values<T, SWIGLU, true>(v, row, a.cols, 0, a.cols);
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, magnitude(v[i]));
      const RowScale rs(m);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < a.cols) q[i] = (int8_t)rs.quant(v[i]);
      *s = rs.scale();
    } else if constexpr (NV > 0) {
      float v[NV][8];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        row_values<T, SWIGLU, false>(v[j], row, a.cols, min((j * NT + at) * 8, a.cols - 8), 8);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, magnitude(v[j][i]));
      const RowScale rs(row_largest<NT>(m, lds));
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j * NT + at < groups) store8(q + min((j * NT + at) * 8, a.cols - 8), v[j], rs);
      if (at == 0) *s = rs.scale();
    } else {
      uint32_t m = 0;
      for (int g = at; g < groups; g += NT) {
        float v[8];
        row_values<T, SWIGLU, false>(v, row, a.cols, min(g * 8, a.cols - 8), 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, magnitude(v[i]));
      }
      const RowScale rs(row_largest<NT>(m, lds));
      for (int g = at; g < groups; g += NT) {
        float v[8];
        row_values<T, SWIGLU, false>(v, row, a.cols, min(g * 8, a.cols - 8), 8);
        store8(q + min(g * 8, a.cols - 8), v, rs);
      }
      if (at == 0) *s = rs.scale();
    }
  }
}

template <class T, bool SWIGLU, int NT, int NV, bool SHORT = false>
hipError_t launch_form(const QuantArgs &a, hipStream_t st) {
  constexpr int PER = SHORT ? kQuantThreads : kQuantThreads / NT;
  // the rows past the largest grid are taken in a loop
  const int64_t grid = std::min<int64_t>((a.rows + PER - 1) / PER, 1 << 20);
  hipLaunchKernelGGL((quant_kernel<T, SWIGLU, NT, NV, SHORT>), dim3((uint32_t)grid),
                     dim3(kQuantThreads), 0, st, a);
  return hipGetLastError();
}

template <class T, bool SWIGLU>
hipError_t launch_type(const QuantArgs &a, hipStream_t st) {
  if (a.cols < 8) return launch_form<T, SWIGLU, kWave, 0, true>(a, st);
  const int groups = (a.cols + 7) / 8;
  if (groups <= 64) return launch_form<T, SWIGLU, 64, 1>(a, st);
  if (groups <= 128) return launch_form<T, SWIGLU, 64, 2>(a, st);
  if (groups <= 256) return launch_form<T, SWIGLU, 64, 4>(a, st);
  if (groups <= 512) return launch_form<T, SWIGLU, 256, 2>(a, st);
  if (groups <= 1024) return launch_form<T, SWIGLU, 256, 4>(a, st);
  if (groups <= 2048) return launch_form<T, SWIGLU, 256, 8>(a, st);
  return launch_form<T, SWIGLU, 256, 0>(a, st);
}

}  // namespace

hipError_t launch_quant(int dtype, bool swiglu, const QuantArgs &a, hipStream_t st) {
  switch (dtype) {
    case CCO_BF16:
      return swiglu ? launch_type<__bf16, true>(a, st) : launch_type<__bf16, false>(a, st);
    case CCO_F16:
      return swiglu ? launch_type<_Float16, true>(a, st) : launch_type<_Float16, false>(a, st);
    default:
      return swiglu ? launch_type<float, true>(a, st) : launch_type<float, false>(a, st);
  }
}

}  // namespace cco
