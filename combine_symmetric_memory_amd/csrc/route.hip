// route.hip -- choice of experts from router logits, their weights, and the
// weights' gradient (include/cco_ops.h).
//
// One wavefront per token; lane l holds logits l, l + 64, ...  The K largest
// choice values are taken one after the other: each lane offers its best
// remaining candidate, the wavefront's largest is found by a reduction over
// the lanes (data-parallel moves, no LDS) and removed.  Choice values are
// compared as integers that order like the floating-point numbers (sign bit
// flipped, negative numbers inverted), with the lower id first among equals.
// Choice by scores with a bias or groups is formed in 64 bits, so that
// values next to a border do not change places by rounding.
//
// Latency and issue bound, not memory: 16384 tokens of 256 fp32 logits, top
// 8, take 15.2 us for 18 MB (the gradient 12.9 us for 35 MB); 256 tokens
// with 8 groups 8.5 us, of which the launch itself is about 4.  (Reductions
// through LDS permutes took 37 and 12.2 us.)
#include "ops_internal.h"
#include "wave_ops.h"

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

// Integers that order like the numbers; NaN like -inf, and -0 like +0; 0 is
// below all.
__device__ __forceinline__ uint64_t order_key(double v) {
  if (!(v == v)) v = -__builtin_inf();
  v += 0.0;
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return (b >> 63) ? ~b : (b | (1ull << 63));
}

__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v == v)) v = -__builtin_inff();
  v += 0.0f;
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  return (b >> 31) ? ~b : (b | (1u << 31));
}

__device__ __forceinline__ int uniform_wave() {
  return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
}

// exp(l - m) with m the largest: 0 for masked logits even if all are.
__device__ __forceinline__ float exp_below(float l, float m) {
  return l == -__builtin_inff() ? 0.0f : expf(l - m);
}

// The lane-wise best candidates' best: the largest (hi, lo), the lowest id
// among equals.  Most rounds end after the first reduction.
template <bool WIDE>
__device__ __forceinline__ int wave_best(uint32_t hi, uint32_t lo, int id) {
  const uint32_t top = wave_largest(hi);
  uint64_t tied = __ballot(hi == top);
  if (WIDE && (tied & (tied - 1))) {
    const uint32_t low = hi == top ? lo : 0u;
    const uint32_t best = wave_largest(low);
    tied = __ballot(hi == top && lo == best);
  }
  if (tied & (tied - 1)) {
    const bool in = (tied >> (threadIdx.x % kWave)) & 1;
    return (int)wave_smallest(in ? (uint32_t)id : 0xFFFFFFFFu);
  }
  return (int)lane_value((uint32_t)id, __builtin_ctzll(tied));
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
    const uint64_t other = lane_value(key, h * lanes);
    rank += other > key || (other == key && h < g);
  }
  // lane g * lanes speaks for group g
  const uint64_t votes = __ballot(g < groups && rank < kept);
  uint64_t mask = 0;
  for (int h = 0; h < groups; ++h) mask |= ((votes >> (h * lanes)) & 1ull) << h;
  return mask;
}

// SCORED: the choice goes by scores (a bias or groups), in 64 bits; otherwise
// by the logits' own order, 32 bits.
template <int DT, int EPL, bool SCORED>
__global__ __launch_bounds__(kRouteWaves *kWave) void route_kernel(RouteArgs a) {
  extern __shared__ double choice[];  // [waves][E], with groups only
  const int wave = uniform_wave(), lane = threadIdx.x % kWave;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / kWave) + wave;
  if (t >= a.T) return;
  const int E = a.E;
  const int64_t row = t * a.ld;
  const float low = -__builtin_inff();
  float l[EPL];
  float m = low;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + i * kWave;
    l[i] = e < E ? load_logit<DT>(a.logits, row + e) : low;
    m = fmaxf(m, l[i]);
  }
  m = wave_largest(m);
  uint32_t hi[EPL], lo[SCORED ? EPL : 1];
  if constexpr (SCORED) {
    uint64_t key[EPL];
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
    if (a.score == CCO_SCORE_SOFTMAX) sum = wave_total(sum);
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
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      hi[i] = (uint32_t)(key[i] >> 32);
      lo[i] = (uint32_t)key[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) hi[i] = lane + i * kWave < E ? order_key(l[i]) : 0;
  }
  // K rounds; lane j keeps the id of round j
  int mine = 0;
  for (int j = 0; j < a.K; ++j) {
    uint32_t bh = hi[0], bl = SCORED ? lo[0] : 0;
    int id = lane;
#pragma unroll
    for (int i = 1; i < EPL; ++i)
      if (hi[i] > bh || (SCORED && hi[i] == bh && lo[SCORED ? i : 0] > bl)) {
        bh = hi[i];
        if (SCORED) bl = lo[SCORED ? i : 0];
        id = lane + i * kWave;
      }
    id = wave_best<SCORED>(bh, bl, id);
    if (lane == j) mine = id;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + i * kWave == id) {
        hi[i] = 0;
        if (SCORED) lo[SCORED ? i : 0] = 0;
      }
  }
  // weights, lane j for round j
  const bool on = lane < a.K;
  const float lc = on ? load_logit<DT>(a.logits, row + mine) : low;
  float w;
  if (a.renorm) {
    const float mc = wave_largest(lc);
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
    const float total = wave_total(s);
    w = total == 0.0f ? 0.0f : s / total;
  } else if (a.score == CCO_SCORE_SOFTMAX) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += exp_below(l[i], m);
    sum = wave_total(sum);
    w = sum == 0.0f ? 0.0f : exp_below(lc, m) / sum;
  } else {
    w = lc > 0.0f ? 1.0f / (1.0f + expf(-lc)) : expf(lc) / (1.0f + expf(lc));
  }
  if (on) {
    a.idx[t * a.K + lane] = mine;
    a.w[t * a.K + lane] = w * a.scale;
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
  const int wave = uniform_wave(), lane = threadIdx.x % kWave;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / kWave) + wave;
  if (t >= a.T) return;
  const int E = a.E;
  const int64_t row = t * a.ld, drow = t * a.lddl;
  const float low = -__builtin_inff();
  int id = -1;
  float dw = 0.0f, lc = low;
  if (lane < a.K) {
    id = a.idx[t * a.K + lane];
    if ((unsigned)id < (unsigned)E) {
      dw = a.dw[t * a.K + lane];
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
    m = wave_largest(m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = exp_below(p[i], m);
      sum += p[i];
    }
    sum = wave_total(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] *= inv;
    part = on ? a.scale * dw * (exp_below(lc, m) * inv) : 0.0f;
    down_all = wave_total(part);
  } else if (a.renorm) {
    const float mc = wave_largest(lc);
    float s, other = 1.0f;  // other: 1 - score (sigmoid)
    if (a.score == CCO_SCORE_SOFTMAX) {
      s = exp_below(lc, mc);
    } else {
      const float down = fminf(mc, 0.0f);
      s = lc > 0.0f ? expf(-down) / (1.0f + expf(-lc)) : exp_below(lc, down) / (1.0f + expf(lc));
      other = lc > 0.0f ? expf(-lc) / (1.0f + expf(-lc)) : 1.0f / (1.0f + expf(lc));
    }
    if (!on) s = 0.0f;
    const float total = wave_total(s);
    const float q = total == 0.0f ? 0.0f : s / total;
    const float mean = wave_total(on ? dw * q : 0.0f);
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
    const int ej = (int)lane_value((uint32_t)id, j);
    const float pj = lane_value(part, j);
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

// Tokens of one launch: with 64 lanes a token, 2^26 of them would need a
// grid of 2^32 threads, which does not run as such.
constexpr int32_t kLaunchTokens = 1 << 24;

template <int DT, int EPL>
hipError_t launch_route_as(bool grad, const RouteArgs &all, hipStream_t st) {
  RouteArgs a = all;
  if (a.T > kLaunchTokens) {
    const int64_t size = DT == CCO_F32 ? 4 : 2;
    for (int64_t t = 0; t < all.T; t += kLaunchTokens) {
      a.T = (int32_t)std::min<int64_t>(kLaunchTokens, all.T - t);
      a.logits = (const char *)all.logits + t * all.ld * size;
      a.idx = all.idx + t * all.K;
      if (grad) {
        a.dw = all.dw + t * all.K;
        a.dlogits = (char *)all.dlogits + t * all.lddl * size;
      } else {
        a.w = all.w + t * all.K;
      }
      const hipError_t err = launch_route_as<DT, EPL>(grad, a, st);
      if (err != hipSuccess) return err;
    }
    return hipSuccess;
  }
  // few tokens: a workgroup each, so that they spread over the CUs
  const int waves = a.T < 4096 ? 1 : kRouteWaves;
  const dim3 grid((uint32_t)(((int64_t)a.T + waves - 1) / waves)), block(waves * kWave);
  if (grad)
    hipLaunchKernelGGL((route_grad_kernel<DT, EPL>), grid, block, 0, st, a);
  else if (a.bias || a.groups > 1)
    hipLaunchKernelGGL((route_kernel<DT, EPL, true>), grid, block,
                       a.groups > 1 ? (size_t)waves * a.E * sizeof(double) : 0, st, a);
  else
    hipLaunchKernelGGL((route_kernel<DT, EPL, false>), grid, block, 0, st, a);
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

hipError_t launch_route(const RouteArgs &a, hipStream_t st) {
  return launch_route_any(false, a, st);
}
hipError_t launch_route_grad(const RouteArgs &a, hipStream_t st) {
  return launch_route_any(true, a, st);
}

}  // namespace cco
