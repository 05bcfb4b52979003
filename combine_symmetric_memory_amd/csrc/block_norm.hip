// block_norm.hip -- the norms around a block, fused with its gate and
// residual, and their gradient (include/cco_ops.h).
//
//   z = post ? y ry post : y,          ry = 1 / sqrt(mean y^2 + eps)
//   out = x + scale gate z
//   u = out ro pre,                    ro = 1 / sqrt(mean out^2 + eps)
//
// Gradient, with q = du pre and M = mean(q out ro):
//   d  = dout + ro (q - out ro M)                              (dx)
//   dz = scale gate d,   dgate = scale z d (summed over the tokens or a row)
//   dy = post ? ry (b - y ry mean(b y ry)) : dz,   b = dz post
//   dpost = sum_t dz y ry,   dpre = sum_t du out ro
// mean(b y ry) would be a third sum over the row that waits for M; it is
// linear in d, so the row's second sum also carries v . dout, v . q and
// v . out (v = scale gate post y ry) and mean(b y ry) follows.  With
// C = sum_t scale d y ry (times a token gate), dpost = gate C and a channel's
// dgate = post C: one column sum serves both.
//
// Bound by memory (8192 x 7168 bf16, every operand present, calls back to
// back: 93 us forward, 5.1 TB/s; gradient with its column sums 138 us, 5.1
// TB/s, of which the column sums' kernel is 5 us): every row is read once and
// stays in one workgroup's registers, 16 elements a thread (8 for rows of at
// most 512).  Workgroups walk the rows with the vectors in registers and the
// next row's loads in flight while the present one is summed; as many
// workgroups as the registers let run at once.  The gradient's column sums
// stay in registers too, one partial per workgroup, added in workgroup order
// by a second kernel (no atomics).  Past 8192 columns the gradient's threads
// have half the registers, 264 to 488 bytes of scratch and no row in flight
// ahead (2000 x 16384 bf16: 248 us, 1.6 TB/s; forward 47 us).
#include "combine_impl.h"
#include "ops_internal.h"
#include "wave_ops.h"

namespace cco {
namespace {

// Eight elements as they lie in memory (16-bit types 16 bytes, fp32 32).
// Rows and vectors may be aligned to an element only: the loads are
// unaligned 16-byte ones, which cost nothing where the address is aligned.
template <class T>
struct Raw8 {
  T v[8];
};

// The elements n, n + 1, ... of r, zeros behind (n uniform over the row's
// last vector; 0..7).
template <class T>
__device__ __forceinline__ Raw8<T> drop_first(Raw8<T> r, int n) {
#pragma unroll
  for (int step = 4; step > 0; step /= 2)
    if (n & step) {
#pragma unroll
      for (int c = 0; c < 8; ++c) r.v[c] = c + step < 8 ? r.v[c + step] : (T)0.0f;
    }
  return r;
}

// How a row of H ends: in whole vectors of eight, inside one, or before the
// first one is full.  A property of the kernel, so that no branch stands
// around a load (the compiler would wait for the load where it ends).
enum RowEnd { kWhole, kInside, kShort };
inline RowEnd row_end(int H) { return H % 8 == 0 ? kWhole : (H > 8 ? kInside : kShort); }

// Elements [at, at + 8) of a row of H.  Past H - 8 the row's last eight are
// loaded instead; cut8, which waits for the load, moves those down that
// belong to the vector and puts zeros behind the row's end.
template <RowEnd END, class T>
__device__ __forceinline__ Raw8<T> load8(const T *row, int at, int H) {
  Raw8<T> r;
  if constexpr (END == kShort) {
#pragma unroll
    for (int c = 0; c < 8; ++c) r.v[c] = row[min(at + c, H - 1)];
  } else {
    __builtin_memcpy(&r, row + min(at, H - 8), sizeof(r));
  }
  return r;
}
template <RowEnd END, class T>
__device__ __forceinline__ Raw8<T> cut8(Raw8<T> r, int at, int H) {
  if constexpr (END == kInside) {
    const Raw8<T> tail = drop_first(r, 8 - H % 8);
#pragma unroll
    for (int c = 0; c < 8; ++c) r.v[c] = at + 8 > H ? tail.v[c] : r.v[c];
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) r.v[c] = (END == kShort ? at + c : at) < H ? r.v[c] : (T)0.0f;
  return r;
}

template <RowEnd END, class T>
__device__ __forceinline__ void store8(T *row, int at, int H, const float *v) {
  Raw8<T> r;
#pragma unroll
  for (int c = 0; c < 8; ++c) r.v[c] = (T)v[c];
  if (END == kWhole ? at < H : at + 8 <= H) {
    __builtin_memcpy(row + at, &r, sizeof(r));
  } else if (END != kWhole) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (at + c < H) row[at + c] = r.v[c];
  }
}

// A thread's share of a row: NV vectors, vector i at (i * threads + t) * 8.
template <RowEnd END, class T, int NV>
struct RowRaw {
  Raw8<T> v[NV];
  __device__ __forceinline__ void load(const T *row, int H) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = load8<END>(row, (i * blockDim.x + threadIdx.x) * 8, H);
  }
  __device__ __forceinline__ void get(int H, float (&f)[NV * 8]) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Raw8<T> r = cut8<END>(v[i], (i * blockDim.x + threadIdx.x) * 8, H);
#pragma unroll
      for (int c = 0; c < 8; ++c) f[i * 8 + c] = (float)r.v[c];
    }
  }
};

template <RowEnd END, class T, int NV>
__device__ __forceinline__ void store_row(T *row, int H, const float (&v)[NV * 8]) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
    store8<END>(row, (i * blockDim.x + threadIdx.x) * 8, H, v + i * 8);
}

// A parameter vector's elements of this thread (1 where absent).
template <RowEnd END, class T, int NV>
__device__ __forceinline__ void load_param(const void *p, int f32, int H, float (&v)[NV * 8]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * blockDim.x + threadIdx.x) * 8;
    if (!p) {
#pragma unroll
      for (int c = 0; c < 8; ++c) v[i * 8 + c] = 1.0f;
    } else if (f32) {
      const Raw8<float> r = cut8<END>(load8<END>((const float *)p, at, H), at, H);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[i * 8 + c] = r.v[c];
    } else {
      const Raw8<T> r = cut8<END>(load8<END>((const T *)p, at, H), at, H);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[i * 8 + c] = (float)r.v[c];
    }
  }
}

// gate * post of this thread's elements.
template <RowEnd END, class T, int NV>
__device__ __forceinline__ void load_gate_post(const NormArgs &a, float (&v)[NV * 8]) {
  float g[NV * 8];
  load_param<END, T, NV>(a.post, a.w_f32, a.H, v);
  load_param<END, T, NV>(a.gate_kind == CCO_GATE_CHANNEL ? a.gate : nullptr, a.w_f32, a.H, g);
#pragma unroll
  for (int i = 0; i < NV * 8; ++i) v[i] *= g[i];
}

// Sums of N values over the workgroup (every thread gets them, in one order
// of addition).  `half` alternates between two halves of the scratch, so one
// barrier per sum is enough: a half is written again only after the next
// barrier.
constexpr int kMaxSums = 8, kMaxWaves = 16;
template <int N>
__device__ __forceinline__ void block_sum(float (&s)[N], float *lds, int &half, int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = wave_total(s[i]);
  if (waves > 1) {
    float *b = lds + half * (kMaxWaves * kMaxSums);
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

__device__ __forceinline__ float rms_inverse(float sum, int H, float eps) {
  return 1.0f / sqrtf(sum / (float)H + eps);
}

// The row this workgroup takes after row t, or t again behind the last (its
// elements are then loaded and not used: no branch around the loads).
__device__ __forceinline__ int64_t next_row(int64_t t, int T) {
  return t + gridDim.x < T ? t + gridDim.x : t;
}

__device__ __forceinline__ int uniform_int(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A thread's share of combine's output row of token t, rounded to bf16: the
// sum over the token's K pairs in order, as combine_token forms it.  (H is a
// multiple of 8 and the windows are aligned.)  Bound by latency: a pair's id
// and position are loads as well, and loads complete in order, so those of
// the next pair wait for this pair's rows, K round trips a token.  Measured
// with 7168 columns and 8 pairs, against the two launches it replaces: 256
// tokens 12 and 17 us, 512 tokens 25 and 22 us, 8192 tokens 323 and 274 us.
template <int NV>
__device__ __forceinline__ void combine_row(const CombineView &c, int64_t t, int H,
                                            RowRaw<kWhole, __bf16, NV> &out) {
  const MoeArgs &a = c.moe;
  float y[NV * 8];
#pragma unroll
  for (int i = 0; i < NV * 8; ++i) y[i] = 0.0f;
  constexpr int B = 8;  // pairs summed together
  for (int j0 = 0; j0 < a.K; j0 += B) {
    u32x4 r[B][NV];
    float w[B];
    bool on[B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      w[j] = 0.0f;
      on[j] = false;
      if (j0 + j < a.K) {
        const int64_t f = t * a.K + j0 + j;
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
  for (int i = 0; i < NV * 8; ++i) out.v[i / 8].v[i % 8] = (__bf16)y[i];
}

template <RowEnd END, class T, int NV, bool COMBINE>
__device__ __forceinline__ void norm_rows(const NormArgs &a, const CombineView *cv) {
  constexpr int N = NV * 8;
  __shared__ float lds[2 * kMaxWaves * kMaxSums];
  int half = 0;
  const int waves = blockDim.x / kWave, H = a.H;
  const bool has_y = COMBINE || a.y;
  // an absent y is read as x and not used: no branch around the loads
  const T *yrow = (const T *)(a.y ? a.y : a.x);
  RowRaw<END, T, NV> rx, ry;
  const bool token = a.gate_kind == CCO_GATE_TOKEN;
  float tgate = 1.0f;  // the token's gate; first of the loads, which return in order
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    if (token) tgate = ((const float *)a.gate)[t];
    rx.load((const T *)a.x + t * H, H);
    if constexpr (!COMBINE) ry.load(yrow + t * H, H);
    __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the row's work
  };
  int64_t t = blockIdx.x;
  fetch(t);
  float gp[N], pre[N];
  load_gate_post<END, T, NV>(a, gp);
  load_param<END, T, NV>(a.pre, a.w_f32, H, pre);
  for (; t < a.T; t += gridDim.x) {
    const int64_t off = t * H;
    float o[N], y[N];
    if constexpr (COMBINE) {
      combine_row<NV>(*cv, t, H, ry);
      if (cv->y_out) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int at = (i * blockDim.x + threadIdx.x) * 8;
          if (at < H) *(Raw8<T> *)((T *)cv->y_out + off + at) = ry.v[i];
        }
      }
    }
    rx.get(H, o);
    if (has_y) ry.get(H, y);
    float s = a.scale * tgate;
    fetch(next_row(t, a.T));
    if (has_y) {
      if (a.post) {
        float sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < N; ++i) sum[0] = __builtin_fmaf(y[i], y[i], sum[0]);
        block_sum<1>(sum, lds, half, waves);
        s *= rms_inverse(sum[0], H, a.eps);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = __builtin_fmaf(s * gp[i], y[i], o[i]);
      if (a.out) store_row<END, T, NV>((T *)a.out + off, H, o);
    }
    if (a.u) {
      float sum[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < N; ++i) sum[0] = __builtin_fmaf(o[i], o[i], sum[0]);
      block_sum<1>(sum, lds, half, waves);
      const float r = rms_inverse(sum[0], H, a.eps);
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = o[i] * r * pre[i];
      store_row<END, T, NV>((T *)a.u + off, H, o);
    }
  }
}

template <RowEnd END, class T, int NV, int MAXT>
__global__ __launch_bounds__(MAXT) void norm_kernel(NormArgs a) {
  norm_rows<END, T, NV, false>(a, nullptr);
}

template <int NV, int MAXT>
__global__ __launch_bounds__(MAXT) void combine_norm_kernel(CombineView c, NormArgs a) {
  norm_rows<kWhole, __bf16, NV, true>(a, &c);
}

// KEEP: the vectors stay in registers and the next row is fetched ahead;
// otherwise (rows of more than 512 threads, whose register budget is half)
// both are read when they are needed.
template <RowEnd END, class T, int NV, int MAXT, bool KEEP>
__global__ __launch_bounds__(MAXT) void norm_grad_kernel(NormArgs a) {
  constexpr int N = NV * 8;
  __shared__ float lds[2 * kMaxWaves * kMaxSums];
  int half = 0;
  const int waves = blockDim.x / kWave, H = a.H;
  const float inv_h = 1.0f / (float)H;
  const bool token = a.gate_kind == CCO_GATE_TOKEN;
  // an absent y, dout or du is read as x and then taken as zeros: no branch
  // around the loads
  const T *yrow = (const T *)(a.y ? a.y : a.x), *drow = (const T *)(a.dout ? a.dout : a.x),
          *qrow = (const T *)(a.du ? a.du : a.x);
  RowRaw<END, T, NV> rx, ry, rd, rq;
  float tgate = 1.0f;  // the token's gate; first of the loads, which return in order
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    const int64_t off = t * H;
    if (token) tgate = ((const float *)a.gate)[t];
    ry.load(yrow + off, H);
    rx.load((const T *)a.x + off, H);
    rd.load(drow + off, H);
    rq.load(qrow + off, H);
    __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the row's work
  };
  int64_t t = blockIdx.x;
  if (KEEP) fetch(t);
  float gp[N], pre[N], csum[N], dpre[N];
  if (KEEP) {
    load_gate_post<END, T, NV>(a, gp);
    load_param<END, T, NV>(a.pre, a.w_f32, H, pre);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) csum[i] = dpre[i] = 0.0f;
  for (; t < a.T; t += gridDim.x) {
    const int64_t off = t * H;
    float x[N], y[N], d[N], q[N];
    if (!KEEP) {
      fetch(t);
      load_gate_post<END, T, NV>(a, gp);
      load_param<END, T, NV>(a.pre, a.w_f32, H, pre);
    }
    rx.get(H, x);
    ry.get(H, y);
    rd.get(H, d);
    rq.get(H, q);
    auto absent = [&](float (&v)[N]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.0f;
    };
    if (!a.y) absent(y);
    if (!a.dout) absent(d);
    if (!a.du) absent(q);
    const float tg = tgate;
    if (KEEP) fetch(next_row(t, a.T));
    float ry1 = 1.0f;
    if (a.post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] = __builtin_fmaf(y[i], y[i], s[0]);
      block_sum<1>(s, lds, half, waves);
      ry1 = rms_inverse(s[0], H, a.eps);
    }
    const float st = a.scale * tg;
    // y becomes y ry.  With pre x becomes out and then out ro;
    // v = gate_channel post y ry.  A norm that is not there leaves its row
    // out of the sums and products: an infinity in it would come back as
    // 0 * inf.  ry and ro meet the rows they normalise before anything else:
    // their squares and cubes leave the range of fp32 long before the rows'
    // sums of squares do.
    float vd;  // scale v . d, d with what comes through the norm of out
    if (a.post) {
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] *= ry1;
    }
    if (a.pre) {
      float s[5] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float v = gp[i] * y[i], qi = q[i] * pre[i];
        x[i] = __builtin_fmaf(st, v, x[i]);
        s[0] = __builtin_fmaf(x[i], x[i], s[0]);
        s[1] = __builtin_fmaf(qi, x[i], s[1]);
        s[2] = __builtin_fmaf(v, d[i], s[2]);
        s[3] = __builtin_fmaf(v, qi, s[3]);
        s[4] = __builtin_fmaf(v, x[i], s[4]);
      }
      block_sum<5>(s, lds, half, waves);
      const float ro = rms_inverse(s[0], H, a.eps);
      const float m = ro * s[1] * inv_h;  // ro M
      vd = a.scale * (s[2] + ro * (s[3] - ro * s[4] * m));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xn = x[i] * ro;
        dpre[i] = __builtin_fmaf(q[i], xn, dpre[i]);
        d[i] = __builtin_fmaf(ro, __builtin_fmaf(-xn, m, q[i] * pre[i]), d[i]);
      }
    } else {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] = __builtin_fmaf(gp[i] * y[i], d[i], s[0]);
      block_sum<1>(s, lds, half, waves);
      vd = a.scale * s[0];
    }
    if (token && threadIdx.x == 0) a.dgate[t] = vd;
    const float by = tg * vd * inv_h;  // mean(b y ry)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float sd = st * d[i];
      csum[i] = __builtin_fmaf(sd, y[i], csum[i]);
      q[i] = sd * gp[i];
      if (a.post) q[i] = ry1 * __builtin_fmaf(-y[i], by, q[i]);
    }
    store_row<END, T, NV>((T *)a.dx + off, H, d);
    if (a.dy) store_row<END, T, NV>((T *)a.dy + off, H, q);
  }
  // this workgroup's column sums: [sum][workgroup][H]
  float *part = a.partial + (int64_t)blockIdx.x * H;
  if (a.dpost || a.gate_kind == CCO_GATE_CHANNEL) {
    store_row<END, float, NV>(part, H, csum);
    part += (int64_t)gridDim.x * H;
  }
  if (a.dpre) store_row<END, float, NV>(part, H, dpre);
}

// Columns of the partial sums, added in fixed order: 16 chains of every 16th
// workgroup, then the chains in order.  Block y 0 is C (where it exists),
// the other dpre.
__global__ __launch_bounds__(1024) void column_sum_kernel(NormArgs a, int nwg) {
  __shared__ float lds[16][kWave];
  const bool has_c = a.dpost || a.gate_kind == CCO_GATE_CHANNEL;
  const float *part = a.partial + (int64_t)blockIdx.y * nwg * a.H;
  const int lane = threadIdx.x % kWave, chain = threadIdx.x / kWave;
  const int h = blockIdx.x * kWave + lane;
  float s = 0.0f;
  if (h < a.H) {
    // eight loads in flight a chain: one after the other each would wait
    // out a round trip
    int w = chain;
    for (; w + 7 * 16 < nwg; w += 8 * 16) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = part[(int64_t)(w + i * 16) * a.H + h];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; w < nwg; w += 16) s += part[(int64_t)w * a.H + h];
  }
  lds[chain][lane] = s;
  __syncthreads();
  if (chain != 0 || h >= a.H) return;
  for (int c = 1; c < 16; ++c) s += lds[c][lane];
  if (!has_c || blockIdx.y == 1) {
    a.dpre[h] = s;
    return;
  }
  auto param = [&](const void *p) -> float {
    if (!p) return 1.0f;
    return a.w_f32 ? ((const float *)p)[h] : (a.w_f16 ? (float)((const _Float16 *)p)[h]
                                                      : (float)((const __bf16 *)p)[h]);
  };
  const bool channel = a.gate_kind == CCO_GATE_CHANNEL;
  if (a.dpost) a.dpost[h] = s * param(channel ? a.gate : nullptr);
  if (channel) a.dgate[h] = s * param(a.post);
}

// Vectors per thread and threads per row.
struct RowShape {
  int nv, threads;
};
RowShape row_shape(int H) {
  const int nv = H <= 512 ? 1 : 2;
  const int n = (H + 7) / 8;
  return {nv, ((n + nv - 1) / nv + kWave - 1) / kWave * kWave};
}
// Workgroups that fill the chip with `per_cu` threads a CU.
int row_grid(int64_t T, int threads, int per_cu) {
  return (int)std::min<int64_t>(T, (int64_t)kNumCus * std::max(1, per_cu / threads));
}

template <RowEnd END, class T>
hipError_t launch_norm_as(const NormArgs &a, hipStream_t st) {
  const RowShape rs = row_shape(a.H);
  const dim3 grid(row_grid(a.T, rs.threads, 1024)), block(rs.threads);
  if (rs.nv == 1)
    hipLaunchKernelGGL((norm_kernel<END, T, 1, 512>), grid, block, 0, st, a);
  else if constexpr (END != kShort) {
    if (rs.threads <= 512)
      hipLaunchKernelGGL((norm_kernel<END, T, 2, 512>), grid, block, 0, st, a);
    else
      hipLaunchKernelGGL((norm_kernel<END, T, 2, 1024>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

template <class T>
hipError_t launch_norm(const NormArgs &a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  switch (row_end(a.H)) {
    case kWhole: return launch_norm_as<kWhole, T>(a, st);
    case kInside: return launch_norm_as<kInside, T>(a, st);
    default: return launch_norm_as<kShort, T>(a, st);
  }
}

template <RowEnd END, class T>
hipError_t launch_grad_as(const NormArgs &a, int nwg, hipStream_t st) {
  const RowShape rs = row_shape(a.H);
  const dim3 grid(nwg), block(rs.threads);
  if (rs.nv == 1)
    hipLaunchKernelGGL((norm_grad_kernel<END, T, 1, 512, true>), grid, block, 0, st, a);
  else if constexpr (END != kShort) {
    if (rs.threads <= 512)
      hipLaunchKernelGGL((norm_grad_kernel<END, T, 2, 512, true>), grid, block, 0, st, a);
    else
      hipLaunchKernelGGL((norm_grad_kernel<END, T, 2, 1024, false>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

template <class T>
hipError_t launch_grad(const NormArgs &a, hipStream_t st) {
  const int nwg = norm_grad_workgroups(a.H, a.T);
  if (nwg > 0) {
    hipError_t err;
    switch (row_end(a.H)) {
      case kWhole: err = launch_grad_as<kWhole, T>(a, nwg, st); break;
      case kInside: err = launch_grad_as<kInside, T>(a, nwg, st); break;
      default: err = launch_grad_as<kShort, T>(a, nwg, st);
    }
    if (err != hipSuccess) return err;
  }
  const int sums = (a.dpost || a.gate_kind == CCO_GATE_CHANNEL) + (a.dpre != nullptr);
  if (sums == 0) return hipSuccess;
  hipLaunchKernelGGL(column_sum_kernel, dim3((a.H + kWave - 1) / kWave, sums), dim3(1024), 0, st,
                     a, nwg);
  return hipGetLastError();
}

}  // namespace

int norm_grad_workgroups(int32_t H, int32_t T) {
  return row_grid(T, row_shape(H).threads, 512);
}

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
  const RowShape rs = row_shape(a.H);
  const dim3 grid(row_grid(a.T, rs.threads, 1024)), block(rs.threads);
  if (rs.nv == 1)
    hipLaunchKernelGGL((combine_norm_kernel<1, 512>), grid, block, 0, st, c, a);
  else if (rs.threads <= 512)
    hipLaunchKernelGGL((combine_norm_kernel<2, 512>), grid, block, 0, st, c, a);
  else
    hipLaunchKernelGGL((combine_norm_kernel<2, 1024>), grid, block, 0, st, c, a);
  return hipGetLastError();
}

}  // namespace cco
