// route.hip -- choice of experts from router logits, their weights, and the
// weights' gradient (include/cco_ops.h).
//
// One wavefront per token; lane l holds logits l, l + 64, ...  The K largest
// choice values are taken one after the other: each lane keeps its best
// remaining candidate, the wavefront's largest is found by a reduction over
// the lanes and removed.  Choice values are compared as integers that order
// like the floating-point numbers (sign bit flipped, negative numbers
// inverted), with the lower id first among equals.  Sums of scores with a
// bias are formed in 64 bits, so that values next to a border do not change
// places by rounding.
#include "ops_internal.h"

namespace cco {
namespace {

constexpr int kRouteWaves = 4;

template <int DT>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
  if constexpr (DT == CCO_BF16) return (float)((const __bf16 *)p)[i];
  if constexpr (DT == CCO_F16) return (float)((const _Float16 *)p)[i];
  return ((const float *)p)[i];
}
template <int DT>
__device__ __forceinline__ void store_logit(void *p, int64_t i, float v) {
  if constexpr (DT == CCO_BF16)
    ((__bf16 *)p)[i] = (__bf16)v;
  else if constexpr (DT == CCO_F16)
    ((_Float16 *)p)[i] = (_Float16)v;
  else
    ((float *)p)[i] = v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, kWave));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

// Integers that order like the numbers; NaN like -inf, and -0 like +0; 0 is
// below all.
__device__ __forceinline__ uint64_t order_key(double v) {
  if (!(v == v)) v = -__builtin_inf();
  v += 0.0;
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return (b >> 63) ? ~b : (b | (1ull << 63));
}

// exp(l - m) with m the largest: 0 for masked logits even if all are.
__device__ __forceinline__ float exp_below(float l, float m) {
  return l == -__builtin_inff() ? 0.0f : expf(l - m);
}

// The largest (key, lowest id) over the wavefront.
__device__ __forceinline__ void wave_best(uint64_t &key, int &id) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const uint64_t k2 = __shfl_xor((unsigned long long)key, d, kWave);
    const int i2 = __shfl_xor(id, d, kWave);
    if (k2 > key || (k2 == key && i2 < id)) {
      key = k2;
      id = i2;
    }
  }
}

// Which experts' groups stay: bit g of the result.  c: choice values of the
// token in LDS (NaN not present).
__device__ __forceinline__ uint64_t kept_groups(const double *c, int E, int groups, int kept,
                                                int lane) {
  const int per = E / groups;
  int lanes = 1;  // lanes per group: the largest power of two that fits
  while (lanes * 2 * groups <= kWave) lanes *= 2;
  const int g = lane / lanes, s = lane % lanes;
  const double low = -__builtin_inf();
  double one = low, two = low;
  if (g < groups)
    for (int i = s; i < per; i += lanes) {
      const double v = c[g * per + i];
      if (v > one) {
        two = one;
        one = v;
      } else if (v > two) {
        two = v;
      }
    }
  for (int d = 1; d < lanes; d <<= 1) {
    const double o1 = __shfl_xor(one, d, kWave), o2 = __shfl_xor(two, d, kWave);
    two = fmax(fmin(one, o1), fmax(two, o2));
    one = fmax(one, o1);
  }
  const double score = two == low ? one : one + two;  // masked experts do not count
  const uint64_t key = order_key(score);
  int rank = 0;
  for (int h = 0; h < groups; ++h) {
    const uint64_t other = __shfl((unsigned long long)key, h * lanes, kWave);
    rank += other > key || (other == key && h < g);
  }
  // lane g * lanes speaks for group g
  const uint64_t votes = __ballot(g < groups && rank < kept);
  uint64_t mask = 0;
  for (int h = 0; h < groups; ++h) mask |= ((votes >> (h * lanes)) & 1ull) << h;
  return mask;
}

template <int DT, int EPL>
__global__ __launch_bounds__(kRouteWaves *kWave) void route_kernel(RouteArgs a) {
  extern __shared__ double choice[];  // [waves][E], with groups only
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int t = blockIdx.x * kRouteWaves + wave;
  if (t >= a.T) return;
  const int E = a.E;
  const int64_t row = (int64_t)t * a.ld;
  const float low = -__builtin_inff();
  float l[EPL];
  float m = low;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + i * kWave;
    l[i] = e < E ? load_logit<DT>(a.logits, row + e) : low;
    m = fmaxf(m, l[i]);
  }
  m = wave_max(m);
  uint64_t key[EPL];
  const bool scored = a.bias || a.groups > 1;
  if (scored) {
    double c[EPL];
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const double d = (double)l[i];
      if (a.score == CCO_SCORE_SOFTMAX) {
        c[i] = l[i] == m ? 1.0 : (l[i] > low ? exp(d - (double)m) : 0.0);
        sum += l[i] > low ? c[i] : 0.0;
      } else {
        c[i] = 1.0 / (1.0 + exp(-d));
      }
    }
    if (a.score == CCO_SCORE_SOFTMAX) sum = wave_sum(sum);
    double *cw = choice + wave * E;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + i * kWave;
      if (a.score == CCO_SCORE_SOFTMAX) c[i] /= sum;
      if (a.bias && e < E) c[i] += (double)a.bias[e];
      if (!(l[i] > low) || !(c[i] == c[i])) c[i] = -__builtin_inf();
      key[i] = e < E ? order_key(c[i]) : 0;
      if (a.groups > 1 && e < E) cw[e] = c[i];
    }
    if (a.groups > 1) {
      // the wavefront's own values: no barrier needed, its LDS accesses are
      // in order
      __builtin_amdgcn_wave_barrier();
      __threadfence_block();
      const uint64_t mask = kept_groups(cw, E, a.groups, a.kept, lane);
      const int per = E / a.groups;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + i * kWave;
        if (e < E && !((mask >> (e / per)) & 1)) key[i] = 0;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      key[i] = lane + i * kWave < E ? order_key((double)l[i]) : 0;
  }
  // K rounds; lane j keeps the id of round j
  int mine = 0;
  for (int j = 0; j < a.K; ++j) {
    uint64_t best = 0;
    int id = 1 << 30;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] > best) {
        best = key[i];
        id = lane + i * kWave;
      }
    wave_best(best, id);
    if (lane == j) mine = id;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + i * kWave == id) key[i] = 0;
  }
  // weights, lane j for round j
  const bool on = lane < a.K;
  const float lc = on ? load_logit<DT>(a.logits, row + mine) : low;
  float w;
  if (a.renorm) {
    const float mc = wave_max(lc);
    float s;
    if (a.score == CCO_SCORE_SOFTMAX) {
      s = exp_below(lc, mc);
    } else {
      // sigmoid scores, all divided by exp(min(mc, 0)), so that a row of
      // very low logits keeps its proportions
      const float down = fminf(mc, 0.0f);
      s = lc > 0.0f ? expf(-down) / (1.0f + expf(-lc)) : exp_below(lc, down) / (1.0f + expf(lc));
    }
    if (!on) s = 0.0f;
    const float total = wave_sum(s);
    w = total == 0.0f ? 0.0f : s / total;
  } else if (a.score == CCO_SCORE_SOFTMAX) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += exp_below(l[i], m);
    sum = wave_sum(sum);
    w = sum == 0.0f ? 0.0f : exp_below(lc, m) / sum;
  } else {
    w = lc > 0.0f ? 1.0f / (1.0f + expf(-lc)) : expf(lc) / (1.0f + expf(lc));
  }
  if (on) {
    a.idx[(int64_t)t * a.K + lane] = mine;
    a.w[(int64_t)t * a.K + lane] = w * a.scale;
  }
}

// Gradient: lane j < K holds the chosen id j, its score s and the
// derivative ds to it; part_j = ds_j d s_j / d l is added to the logits that
// id j names.
//   renorm    ds_j = scale (dw_j - sum_i dw_i q_i) / total, q = s / total
//   sigmoid   part_j = ds_j s_j (1 - s_j)
//   softmax   part_j = ds_j s_j, and without renorm - p_e sum_j part_j for
//             every e (with renorm the sum is zero: the softmax's own
//             normalisation cancels)
template <int DT, int EPL>
__global__ __launch_bounds__(kRouteWaves *kWave) void route_grad_kernel(RouteArgs a) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int t = blockIdx.x * kRouteWaves + wave;
  if (t >= a.T) return;
  const int E = a.E;
  const int64_t row = (int64_t)t * a.ld, drow = (int64_t)t * a.lddl;
  const float low = -__builtin_inff();
  int id = -1;
  float dw = 0.0f, lc = low;
  if (lane < a.K) {
    id = a.idx[(int64_t)t * a.K + lane];
    if ((unsigned)id < (unsigned)E) {
      dw = a.dw[(int64_t)t * a.K + lane];
      lc = load_logit<DT>(a.logits, row + id);
    } else {
      id = -1;
    }
  }
  const bool on = id >= 0;
  float p[EPL];
  float part, down_all = 0.0f;
  if (a.score == CCO_SCORE_SOFTMAX && !a.renorm) {
    float m = low;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + i * kWave;
      p[i] = e < E ? load_logit<DT>(a.logits, row + e) : low;
      m = fmaxf(m, p[i]);
    }
    m = wave_max(m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = exp_below(p[i], m);
      sum += p[i];
    }
    sum = wave_sum(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] *= inv;
    part = on ? a.scale * dw * (exp_below(lc, m) * inv) : 0.0f;
    down_all = wave_sum(part);
  } else if (a.renorm) {
    const float mc = wave_max(lc);
    float s, other = 1.0f;  // other: 1 - score (sigmoid)
    if (a.score == CCO_SCORE_SOFTMAX) {
      s = exp_below(lc, mc);
    } else {
      const float down = fminf(mc, 0.0f);
      s = lc > 0.0f ? expf(-down) / (1.0f + expf(-lc)) : exp_below(lc, down) / (1.0f + expf(lc));
      other = lc > 0.0f ? expf(-lc) / (1.0f + expf(-lc)) : 1.0f / (1.0f + expf(lc));
    }
    if (!on) s = 0.0f;
    const float total = wave_sum(s);
    const float q = total == 0.0f ? 0.0f : s / total;
    const float mean = wave_sum(on ? dw * q : 0.0f);
    part = on ? a.scale * (dw - mean) * q * other : 0.0f;
  } else {
    const float s = lc > 0.0f ? 1.0f / (1.0f + expf(-lc)) : expf(lc) / (1.0f + expf(lc));
    const float other = lc > 0.0f ? expf(-lc) / (1.0f + expf(-lc)) : 1.0f / (1.0f + expf(lc));
    part = on ? a.scale * dw * s * other : 0.0f;
  }
  float g[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    g[i] = (a.score == CCO_SCORE_SOFTMAX && !a.renorm) ? -p[i] * down_all : 0.0f;
  for (int j = 0; j < a.K; ++j) {
    const int ej = __shfl(id, j, kWave);
    const float pj = __shfl(part, j, kWave);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + i * kWave == ej) g[i] += pj;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + i * kWave;
    if (e < E) store_logit<DT>(a.dlogits, drow + e, g[i]);
  }
}

template <int DT, int EPL>
hipError_t launch_route_as(bool grad, const RouteArgs &a, hipStream_t st) {
  const dim3 grid((uint32_t)(((int64_t)a.T + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * kWave);
  if (grad)
    hipLaunchKernelGGL((route_grad_kernel<DT, EPL>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((route_kernel<DT, EPL>), grid, block,
                       a.groups > 1 ? (size_t)kRouteWaves * a.E * sizeof(double) : 0, st, a);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_route_dt(bool grad, const RouteArgs &a, hipStream_t st) {
  const int per_lane = (a.E + kWave - 1) / kWave;
  if (per_lane <= 1) return launch_route_as<DT, 1>(grad, a, st);
  if (per_lane <= 2) return launch_route_as<DT, 2>(grad, a, st);
  if (per_lane <= 4) return launch_route_as<DT, 4>(grad, a, st);
  if (per_lane <= 8) return launch_route_as<DT, 8>(grad, a, st);
  return launch_route_as<DT, 16>(grad, a, st);
}

hipError_t launch_route_any(bool grad, const RouteArgs &a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  switch (a.dtype) {
    case CCO_BF16: return launch_route_dt<CCO_BF16>(grad, a, st);
    case CCO_F16: return launch_route_dt<CCO_F16>(grad, a, st);
    default: return launch_route_dt<CCO_F32>(grad, a, st);
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, hipStream_t st) { return launch_route_any(false, a, st); }
hipError_t launch_route_grad(const RouteArgs &a, hipStream_t st) { return launch_route_any(true, a, st); }

}  // namespace cco
