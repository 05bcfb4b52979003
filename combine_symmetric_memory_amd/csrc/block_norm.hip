// block_norm.hip -- the norms around a block, fused with its gate and
// residual, and their gradient (include/cco_ops.h).
//
//   z = post ? y ry post : y,          ry = rsqrt(mean y^2 + eps)
//   out = x + scale gate z
//   u = out ro pre,                    ro = rsqrt(mean out^2 + eps)
//
// Gradient, with q = du pre and M = mean(q out):
//   d  = dout + ro q - out ro^3 M                              (dx)
//   dz = scale gate d,   dgate = scale z d (summed over the tokens or a row)
//   dy = post ? ry b - y ry^3 mean(b y) : dz,   b = dz post
//   dpost = sum_t dz y ry,   dpre = sum_t du out ro
// mean(b y) would be a third sum over the row that waits for M; it is linear
// in d, so the row's second sum also carries v . dout, v . q and v . out
// (v = scale gate post y) and mean(b y) follows from them.
//
// Bound by memory: every row is read once and stays in one workgroup's
// registers.  Workgroups walk the rows with the vectors post, gate and pre
// in registers; the gradient's column sums stay in registers too, one
// partial per workgroup, added in workgroup order by a second kernel (no
// atomics).
#include "combine_impl.h"
#include "ops_internal.h"

namespace cco {
namespace {

template <int DT>
struct Elem;
template <>
struct Elem<CCO_BF16> {
  typedef __bf16 T;
};
template <>
struct Elem<CCO_F16> {
  typedef _Float16 T;
};
template <>
struct Elem<CCO_F32> {
  typedef float T;
};

// A thread's share of a row: NV vectors of VW elements.  VW 8: the row is
// whole 16-byte vectors, vector i of thread t is vector i * threads + t;
// VW 1: single elements (any width, any alignment).
template <class T, int VW>
__device__ __forceinline__ void load_vec(const T *p, float *v) {
  if constexpr (VW == 1) {
    v[0] = (float)p[0];
  } else if constexpr (sizeof(T) == 2) {
    typedef T t8 __attribute__((ext_vector_type(8)));
    const t8 q = *(const t8 *)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)q[i];
  } else {
    typedef float f4 __attribute__((ext_vector_type(4)));
    const f4 a = ((const f4 *)p)[0], b = ((const f4 *)p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

template <class T, int VW>
__device__ __forceinline__ void store_vec(T *p, const float *v) {
  if constexpr (VW == 1) {
    p[0] = (T)v[0];
  } else if constexpr (sizeof(T) == 2) {
    typedef T t8 __attribute__((ext_vector_type(8)));
    t8 q;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = (T)v[i];
    *(t8 *)p = q;
  } else {
    typedef float f4 __attribute__((ext_vector_type(4)));
    f4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = v[i];
      b[i] = v[4 + i];
    }
    ((f4 *)p)[0] = a;
    ((f4 *)p)[1] = b;
  }
}

__device__ __forceinline__ int uniform_int(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Sums of N values over the workgroup (every thread gets them, in the same
// order of addition).  `buf` alternates between two halves, so one barrier
// per sum is enough: a half is written again only after the next barrier.
constexpr int kMaxSums = 5;
template <int N>
__device__ __forceinline__ void block_sum(float (&s)[N], float *lds, int &half, int waves) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor(s[i], d, kWave);
  if (waves > 1) {
    float *b = lds + half * (16 * kMaxSums);
    half ^= 1;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) b[wave * kMaxSums + i] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 0.0f;
    for (int w = 0; w < waves; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] += b[w * kMaxSums + i];
  }
}

// Parameter vectors of a thread's elements (1 where absent).
template <class T, int VW, int NV>
__device__ __forceinline__ void load_param(const void *p, int f32, int H, float (&v)[NV * VW]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * blockDim.x + threadIdx.x) * VW;
#pragma unroll
    for (int c = 0; c < VW; ++c) v[i * VW + c] = 1.0f;
    if (p && at < H) {
      // the vectors are aligned to an element only
#pragma unroll
      for (int c = 0; c < VW; ++c)
        v[i * VW + c] = f32 ? ((const float *)p)[at + c] : (float)((const T *)p)[at + c];
    }
  }
}

template <class T, int VW, int NV>
__device__ __forceinline__ void load_row(const T *row, int H, float (&v)[NV * VW]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * blockDim.x + threadIdx.x) * VW;
#pragma unroll
    for (int c = 0; c < VW; ++c) v[i * VW + c] = 0.0f;
    if (row && at < H) load_vec<T, VW>(row + at, v + i * VW);
  }
}

template <class T, int VW, int NV>
__device__ __forceinline__ void store_row(T *row, int H, const float (&v)[NV * VW]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * blockDim.x + threadIdx.x) * VW;
    if (at < H) store_vec<T, VW>(row + at, v + i * VW);
  }
}

__device__ __forceinline__ float rms_inverse(float sum, int H, float eps) {
  return 1.0f / sqrtf(sum / (float)H + eps);
}

// A thread's share of combine's output row of token t, rounded to bf16: the
// sum over the token's K pairs in order, as combine_token forms it.
template <int NV>
__device__ __forceinline__ void combine_row(const CombineView &c, int t, int H,
                                            float (&y)[NV * 8]) {
  const MoeArgs &a = c.moe;
#pragma unroll
  for (int i = 0; i < NV * 8; ++i) y[i] = 0.0f;
  constexpr int B = 8;  // pairs whose rows are in flight together
  for (int j0 = 0; j0 < a.K; j0 += B) {
    u32x4 r[B][NV];
    float w[B];
    bool on[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      w[j] = 0.0f;
      on[j] = false;
      if (j0 + j < a.K) {
        const int64_t f = (int64_t)t * a.K + j0 + j;
        const int e = uniform_int(a.eid[f]), p = uniform_int(a.pos[f]);
        w[j] = c.w[f];
        on[j] = (unsigned)e < (unsigned)a.E && p >= 0 && (int64_t)p < a.cap;
        if (on[j]) {
          const u32x4 *row =
              (const u32x4 *)slot_addr(a, slot_of(a, e), c.win, (uint64_t)p * H * 2);
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int v = i * blockDim.x + threadIdx.x;
            if (v * 8 < H) r[j][i] = __builtin_nontemporal_load(row + v);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (on[j])
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if ((i * blockDim.x + threadIdx.x) * 8 < H)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              y[i * 8 + 2 * q] = __builtin_fmaf(w[j], bf16_lo(r[j][i][q]), y[i * 8 + 2 * q]);
              y[i * 8 + 2 * q + 1] =
                  __builtin_fmaf(w[j], bf16_hi(r[j][i][q]), y[i * 8 + 2 * q + 1]);
            }
  }
#pragma unroll
  for (int i = 0; i < NV * 8; ++i) y[i] = (float)(__bf16)y[i];
}

template <class T, int VW, int NV, bool COMBINE>
__device__ __forceinline__ void norm_rows(const NormArgs &a, const CombineView *cv) {
  constexpr int N = NV * VW;
  __shared__ float lds[2 * 16 * kMaxSums];
  int half = 0;
  const int waves = blockDim.x / kWave, H = a.H;
  float gate[N], post[N], pre[N];
  load_param<T, VW, NV>(a.gate_kind == CCO_GATE_CHANNEL ? a.gate : nullptr, a.w_f32, H, gate);
  load_param<T, VW, NV>(a.post, a.w_f32, H, post);
  load_param<T, VW, NV>(a.pre, a.w_f32, H, pre);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t off = (int64_t)t * H;
    float o[N], y[N];
    load_row<T, VW, NV>((const T *)a.x + off, H, o);
    if (COMBINE || a.y) {
      if constexpr (COMBINE) {
        combine_row<NV>(*cv, t, H, y);
        if (cv->y_out) store_row<T, VW, NV>((T *)cv->y_out + off, H, y);
      } else {
        load_row<T, VW, NV>((const T *)a.y + off, H, y);
      }
      float s = a.scale;
      if (a.gate_kind == CCO_GATE_TOKEN) s *= ((const float *)a.gate)[t];
      float ry[1] = {1.0f};
      if (a.post) {
        ry[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) ry[0] = __builtin_fmaf(y[i], y[i], ry[0]);
        block_sum<1>(ry, lds, half, waves);
        ry[0] = rms_inverse(ry[0], H, a.eps);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = __builtin_fmaf(s * gate[i], y[i] * ry[0] * post[i], o[i]);
      if (a.out) store_row<T, VW, NV>((T *)a.out + off, H, o);
    }
    if (a.u) {
      float ro[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < N; ++i) ro[0] = __builtin_fmaf(o[i], o[i], ro[0]);
      block_sum<1>(ro, lds, half, waves);
      const float r = rms_inverse(ro[0], H, a.eps);
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = o[i] * r * pre[i];
      store_row<T, VW, NV>((T *)a.u + off, H, o);
    }
  }
}

template <class T, int VW, int NV>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
  norm_rows<T, VW, NV, false>(a, nullptr);
}

template <int NV>
__global__ __launch_bounds__(1024) void combine_norm_kernel(CombineView c, NormArgs a) {
  norm_rows<__bf16, 8, NV, true>(a, &c);
}

template <class T, int VW, int NV>
__global__ __launch_bounds__(1024) void norm_grad_kernel(NormArgs a) {
  constexpr int N = NV * VW;
  __shared__ float lds[2 * 16 * kMaxSums];
  int half = 0;
  const int waves = blockDim.x / kWave, H = a.H;
  const float inv_h = 1.0f / (float)H;
  const bool channel = a.gate_kind == CCO_GATE_CHANNEL, token = a.gate_kind == CCO_GATE_TOKEN;
  float gate[N], post[N], pre[N], dgate[N], dpost[N], dpre[N];
  load_param<T, VW, NV>(channel ? a.gate : nullptr, a.w_f32, H, gate);
  load_param<T, VW, NV>(a.post, a.w_f32, H, post);
  load_param<T, VW, NV>(a.pre, a.w_f32, H, pre);
#pragma unroll
  for (int i = 0; i < N; ++i) dgate[i] = dpost[i] = dpre[i] = 0.0f;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t off = (int64_t)t * H;
    float x[N], y[N], d[N], q[N];
    load_row<T, VW, NV>((const T *)a.x + off, H, x);
    load_row<T, VW, NV>(a.y ? (const T *)a.y + off : nullptr, H, y);
    load_row<T, VW, NV>(a.dout ? (const T *)a.dout + off : nullptr, H, d);
    load_row<T, VW, NV>(a.du ? (const T *)a.du + off : nullptr, H, q);
    const float tg = token ? ((const float *)a.gate)[t] : 1.0f;
    float ry = 1.0f;
    if (a.post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] = __builtin_fmaf(y[i], y[i], s[0]);
      block_sum<1>(s, lds, half, waves);
      ry = rms_inverse(s[0], H, a.eps);
    }
    const float st = a.scale * tg;
    // x becomes out; v = scale gate_channel post y
    float s[5] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = __builtin_fmaf(st * gate[i], y[i] * ry * post[i], x[i]);
      const float v = a.scale * gate[i] * post[i] * y[i], qi = q[i] * pre[i];
      s[0] = __builtin_fmaf(x[i], x[i], s[0]);
      s[1] = __builtin_fmaf(qi, x[i], s[1]);
      s[2] = __builtin_fmaf(v, d[i], s[2]);
      s[3] = __builtin_fmaf(v, qi, s[3]);
      s[4] = __builtin_fmaf(v, x[i], s[4]);
    }
    block_sum<5>(s, lds, half, waves);
    const float ro = a.pre ? rms_inverse(s[0], H, a.eps) : 0.0f;
    const float m3 = ro * ro * ro * s[1] * inv_h;                   // ro^3 M
    const float vd = s[2] + ro * s[3] - m3 * s[4];                  // v . d
    if (token && threadIdx.x == 0) a.dgate[t] = vd * ry;
    const float by = a.post ? ry * ry * ry * tg * vd * inv_h : 0.0f;  // ry^3 mean(b y)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dpre[i] = __builtin_fmaf(q[i], x[i] * ro, dpre[i]);
      d[i] += ro * (q[i] * pre[i]) - x[i] * m3;
      const float yr = y[i] * ry;
      const float sd = a.scale * d[i];
      dgate[i] = __builtin_fmaf(sd, yr * post[i], dgate[i]);
      const float dz = sd * tg * gate[i];
      dpost[i] = __builtin_fmaf(dz, yr, dpost[i]);
      q[i] = __builtin_fmaf(-y[i], by, ry * (dz * post[i]));
    }
    store_row<T, VW, NV>((T *)a.dx + off, H, d);
    if (a.dy) store_row<T, VW, NV>((T *)a.dy + off, H, q);
  }
  // this workgroup's column sums: [sum kind][workgroup][H]
  float *part = a.partial + (int64_t)blockIdx.x * H;
  const int64_t kind = (int64_t)gridDim.x * H;
  auto leave = [&](const float (&v)[N]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (i * blockDim.x + threadIdx.x) * VW;
      if (at < H)
#pragma unroll
        for (int c = 0; c < VW; ++c) part[at + c] = v[i * VW + c];
    }
    part += kind;
  };
  if (a.dpost) leave(dpost);
  if (channel) leave(dgate);
  if (a.dpre) leave(dpre);
}

// out[h] = sum over the workgroups of partial[w][h], in fixed order: 16
// chains of every 16th workgroup, then the chains in order.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float *partial, int nwg, int H,
                                                          float *o0, float *o1, float *o2) {
  __shared__ float lds[16][kWave];
  float *outs[3] = {o0, o1, o2};
  const float *part = partial + (int64_t)blockIdx.y * nwg * H;
  const int lane = threadIdx.x % kWave, chain = threadIdx.x / kWave;
  const int h = blockIdx.x * kWave + lane;
  float s = 0.0f;
  if (h < H)
    for (int w = chain; w < nwg; w += 16) s += part[(int64_t)w * H + h];
  lds[chain][lane] = s;
  __syncthreads();
  if (chain == 0 && h < H) {
    for (int c = 1; c < 16; ++c) s += lds[c][lane];
    float *o = blockIdx.y == 0 ? o0 : (blockIdx.y == 1 ? o1 : o2);
    o[h] = s;
  }
}

// Threads per row for n vectors with NV vectors each.
int row_threads(int n, int nv) { return ((n + nv - 1) / nv + kWave - 1) / kWave * kWave; }

bool all_aligned16(std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if ((uintptr_t)p & 15) return false;
  return true;
}

template <class T>
hipError_t launch_norm(const NormArgs &a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  const int H = a.H;
  const int grid = a.T < 2048 ? a.T : 2048;
  const bool vec = H % 8 == 0 && all_aligned16({a.x, a.y, a.out, a.u});
  auto go = [&](auto kernel, int nvec, int nv) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(row_threads(nvec, nv)), 0, st, a);
    return hipGetLastError();
  };
  if (vec) return H <= 8192 ? go(norm_kernel<T, 8, 1>, H / 8, 1) : go(norm_kernel<T, 8, 2>, H / 8, 2);
  if (H <= 1024) return go(norm_kernel<T, 1, 1>, H, 1);
  if (H <= 4096) return go(norm_kernel<T, 1, 4>, H, 4);
  if (H <= 8192) return go(norm_kernel<T, 1, 8>, H, 8);
  return go(norm_kernel<T, 1, 16>, H, 16);
}

template <class T>
hipError_t launch_grad(const NormArgs &a, hipStream_t st) {
  const int H = a.H;
  const int grid = norm_grad_workgroups(a.T);
  const bool vec = H % 8 == 0 && all_aligned16({a.x, a.y, a.dout, a.du, a.dx, a.dy});
  auto go = [&](auto kernel, int nvec, int nv) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(row_threads(nvec, nv)), 0, st, a);
    return hipGetLastError();
  };
  hipError_t err = hipSuccess;
  if (grid > 0) {
    if (vec)
      err = H <= 8192 ? go(norm_grad_kernel<T, 8, 1>, H / 8, 1) : go(norm_grad_kernel<T, 8, 2>, H / 8, 2);
    else if (H <= 1024)
      err = go(norm_grad_kernel<T, 1, 1>, H, 1);
    else if (H <= 4096)
      err = go(norm_grad_kernel<T, 1, 4>, H, 4);
    else if (H <= 8192)
      err = go(norm_grad_kernel<T, 1, 8>, H, 8);
    else
      err = go(norm_grad_kernel<T, 1, 16>, H, 16);
  }
  if (err != hipSuccess) return err;
  float *outs[3];
  int n = 0;
  if (a.dpost) outs[n++] = a.dpost;
  if (a.gate_kind == CCO_GATE_CHANNEL) outs[n++] = a.dgate;
  if (a.dpre) outs[n++] = a.dpre;
  if (n == 0) return hipSuccess;
  for (int i = n; i < 3; ++i) outs[i] = outs[0];
  hipLaunchKernelGGL(column_sum_kernel, dim3((H + kWave - 1) / kWave, n), dim3(1024), 0, st,
                     a.partial, grid, H, outs[0], outs[1], outs[2]);
  return hipGetLastError();
}

}  // namespace

int norm_grad_workgroups(int32_t T) { return T < 256 ? T : 256; }

hipError_t launch_block_norm(int dtype, const NormArgs &a, hipStream_t st) {
  switch (dtype) {
    case CCO_BF16: return launch_norm<__bf16>(a, st);
    case CCO_F16: return launch_norm<_Float16>(a, st);
    default: return launch_norm<float>(a, st);
  }
}

hipError_t launch_block_norm_grad(int dtype, const NormArgs &a, hipStream_t st) {
  switch (dtype) {
    case CCO_BF16: return launch_grad<__bf16>(a, st);
    case CCO_F16: return launch_grad<_Float16>(a, st);
    default: return launch_grad<float>(a, st);
  }
}

hipError_t launch_combine_norm(const CombineView &c, const NormArgs &a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  const int grid = a.T < 2048 ? a.T : 2048, nvec = a.H / 8;
  if (a.H <= 8192)
    hipLaunchKernelGGL((combine_norm_kernel<1>), dim3(grid), dim3(row_threads(nvec, 1)), 0, st, c, a);
  else
    hipLaunchKernelGGL((combine_norm_kernel<2>), dim3(grid), dim3(row_threads(nvec, 2)), 0, st, c, a);
  return hipGetLastError();
}

}  // namespace cco
