// moe_few.hip -- a whole mixture-of-experts layer for a few tokens in two
// launches (include/cco_ops.h):
//
//   h[t, e] = silu(Wg_e x[t]) * (Wu_e x[t])
//   out[t]  = sum_e share[t][e] W2_e h[t, e]
//
// Bound by the weights of the experts that some token has, each read once.
// Nothing is planned beforehand: every workgroup finds the experts in use and
// their tokens from the ids (a bit set of experts; the tokens of an expert are
// one ballot, so there are at most 64).
//
// Weight rows are the M side of 16x16x32 MFMAs, tokens the N side: a lane
// loads 16 bytes of a weight row straight into registers, 64 bytes of 16 rows
// a load, and its expert's tokens' rows come from the caches.  The columns of
// a tile that no token fills repeat the first token's; nothing reads them.
//
// h is held in 32 bits and handed on as two bf16 values, h = hi + lo to 2^-17
// of it: the matrix cores have the time, since a compute unit gets about nine
// bytes of weights a cycle, and only the output is rounded.  16-bit floating
// weights of the second product are split the same way, exactly (fp16's
// eleven bits into two bf16 values), so that h may exceed fp16's range.
// 8-bit weights are exact in bf16 and fp16 and meet their scales in the sums.
#include <type_traits>

#include "group_common.h"

namespace cco {
namespace {

constexpr int kFewWaves = 8, kFewThreads = kFewWaves * kWave;
constexpr int kFewRows = 16;      // weight rows of a tile
constexpr int kFewStepBytes = 64; // bytes of a weight row a step takes

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 16 bytes at p, of which the first `have` exist; the others are zeros.
__device__ __forceinline__ u32x4 load16(const char *p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ u32x4 load16(const char *p, int have) {
  if (have >= 16) return load16(p);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < have) v[i / 4] |= (uint32_t)(uint8_t)p[i] << (8 * (i % 4));
  return v;
}

// The ids of a call in LDS and the experts in use.
struct FewIds {
  uint32_t live[kMaxExperts / 32];
  int32_t ids[kFewMaxTokens * kMaxTopk];
};

__device__ __forceinline__ void few_read_ids(const FewArgs &a, FewIds &s) {
  for (int i = threadIdx.x; i < kMaxExperts / 32; i += kFewThreads) s.live[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * a.K; i += kFewThreads) {
    const int e = a.idx[i];
    s.ids[i] = e;
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
  template <bool SHARE>
  __device__ __forceinline__ void find(const FewArgs &a, const FewIds &s, int e) {
    const int lane = threadIdx.x % kWave;
    int first = -1;
    float sum = 0.0f;
    if (lane < a.T)
      for (int j = a.K - 1; j >= 0; --j)
        if (s.ids[lane * a.K + j] == e) first = lane * a.K + j;
    if constexpr (SHARE) {
      if (first >= 0)
        for (int p = first; p < (lane + 1) * a.K; ++p)
          if (s.ids[p] == e) sum = p == first ? a.w[p] : sum + a.w[p];
    }
    const uint64_t mask = __ballot(first >= 0), below = (1ull << lane) - 1;
    count = uniform(__popcll(mask));
    // lane t's values go to the lane of its rank, other lanes' behind them
    const int to = first >= 0 ? __popcll(mask & below) : count + __popcll(~mask & below);
    pair = __builtin_amdgcn_ds_permute(to * 4, first);
    if constexpr (SHARE)
      share = __builtin_bit_cast(
          float, __builtin_amdgcn_ds_permute(to * 4, __builtin_bit_cast(int, sum)));
  }
};

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
// Eight fp16 values as the sum of two bf16 ones.
__device__ __forceinline__ void split_f16(u32x4 v, u32x4 &hi, u32x4 &lo) {
  const f16x8 h = __builtin_bit_cast(f16x8, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = (float)h[2 * i], b = (float)h[2 * i + 1];
    hi[i] = top_halves(a, b);
    const float ah = __builtin_bit_cast(float, hi[i] << 16);
    const float bh = __builtin_bit_cast(float, hi[i] & 0xffff0000u);
    lo[i] = top_halves(a - ah, b - bh);
  }
}

// The product of MT tiles of weight rows with NT tiles of columns, over a
// range of steps of the reduction.  EL: the weights' elements.  PAIR: the
// columns are h, in two planes; otherwise x, of the weights' type or, with
// 8-bit weights, fp16 (XF16) or bf16.
//
// U steps are loaded together.  The weights' loads run a chunk ahead; the
// columns', which the caches hold, are issued before them and waited for
// alone, so that their registers are needed once.
template <GroupElem EL, bool PAIR, bool XF16, int MT, int NT>
struct FewStream {
  static constexpr int HALVES = EL == kElemI8 ? 2 : 1;  // 16-byte pieces of a column a step
  static constexpr int NB = (PAIR ? 2 : 1) * HALVES;
  static constexpr int U = NT * NB + 2 * MT <= 6 ? 4 : 2;
  template <int N>
  struct Rows {
    u32x4 v[N][MT];
  };
  template <int N>
  struct Columns {
    u32x4 v[N][NT][NB];
  };
  const char *a[MT];  // uniform: the tiles' matrices
  uint32_t arow[MT];  // this lane's byte offset: its row, and its piece of a step
  const char *b;      // uniform: x, or the high plane of h
  uint32_t brow[NT];
  uint64_t plane;     // bytes between the planes of h
  int abytes;         // bytes of a weight row
  int bbytes;         // bytes of a column that may be read
  f32x4 acc[MT][NT];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[i][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // Steps s .. s + N - 1, all inside the rows.
  template <int N>
  __device__ __forceinline__ void load_rows(Rows<N> &r, int s) const {
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        r.v[u][i] = load16(a[i] + (s * kFewStepBytes + arow[i]) + u * kFewStepBytes);
  }
  template <int N>
  __device__ __forceinline__ void load_columns(Columns<N> &c, int s) const {
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < NB; ++h)
          c.v[u][n][h] = load16(b + (h / HALVES) * plane +
                                (s * (kFewStepBytes * HALVES) + brow[n]) +
                                (u * kFewStepBytes * HALVES + (h % HALVES) * 16));
  }
  // Step s, in which rows end.
  __device__ __forceinline__ void load_end(Rows<1> &r, Columns<1> &c, int s) const {
    const int piece = (threadIdx.x % kWave) / 16;
    const int at = s * kFewStepBytes + piece * 16;
#pragma unroll
    for (int i = 0; i < MT; ++i)
      r.v[0][i] = load16(a[i] + s * kFewStepBytes + arow[i], abytes - at);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < NB; ++h)
        c.v[0][n][h] = load16(b + (h / HALVES) * plane + s * (kFewStepBytes * HALVES) + brow[n] +
                                  (h % HALVES) * 16,
                              bbytes - at * HALVES - (h % HALVES) * 16);
  }
  template <int N>
  __device__ __forceinline__ void multiply(const Rows<N> &r, const Columns<N> &c) {
    constexpr bool F = XF16 && !PAIR;
    using V = std::conditional_t<F, f16x8, bf16x8>;
    auto mma = [&](int i, int n, u32x4 x, u32x4 y) __attribute__((always_inline)) {
      acc[i][n] = mfma16(__builtin_bit_cast(V, x), __builtin_bit_cast(V, y), acc[i][n]);
    };
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const u32x4 w = r.v[u][i];
        if constexpr (EL == kElemI8) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4 f = from_i8<F>(w[2 * h], w[2 * h + 1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int p = 0; p < (PAIR ? 2 : 1); ++p) mma(i, n, f, c.v[u][n][p * 2 + h]);
          }
        } else if constexpr (EL == kElemF16 && PAIR) {
          u32x4 hi, lo;
          split_f16(w, hi, lo);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            // (the product of the two low parts is 2^-16 of the whole)
            mma(i, n, hi, c.v[u][n][0]);
            mma(i, n, hi, c.v[u][n][1]);
            mma(i, n, lo, c.v[u][n][0]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < NB; ++p) mma(i, n, w, c.v[u][n][p]);
        }
      }
  }
  // Steps [from, to).
  __device__ __forceinline__ void run(int from, int to) {
    const int inside = min(to, min(abytes / kFewStepBytes, bbytes / (kFewStepBytes * HALVES)));
    int s = from;
    if (s + U <= inside) {
      Rows<U> r[2];
      load_rows<U>(r[0], s);
      auto chunk = [&](Rows<U> &now, Rows<U> &next) __attribute__((always_inline)) {
        Columns<U> c;
        load_columns<U>(c, s);
        // (past the last chunk: the last one again)
        load_rows<U>(next, s + 2 * U <= inside ? s + U : s);
        __builtin_amdgcn_sched_barrier(0);
        multiply<U>(now, c);
        s += U;
      };
      while (s + 2 * U <= inside) {
        chunk(r[0], r[1]);
        chunk(r[1], r[0]);
      }
      if (s + U <= inside) chunk(r[0], r[1]);
    }
#pragma unroll 1
    for (; s < to; ++s) {
      Rows<1> r;
      Columns<1> c;
      if (s < inside) {
        load_rows<1>(r, s);
        load_columns<1>(c, s);
      } else {
        load_end(r, c, s);
      }
      multiply<1>(r, c);
    }
  }
};

// Wavefronts share a reduction in pieces of kFewPiece steps (a multiple of
// every U), so that only a row's end is left over.
constexpr int kFewPiece = 4;
constexpr int few_steps(int bytes) { return (bytes + kFewStepBytes - 1) / kFewStepBytes; }
constexpr int few_pieces(int bytes) { return (few_steps(bytes) + kFewPiece - 1) / kFewPiece; }

// ---------------------------------------------------------- gate and up --
// A workgroup takes tiles of 16 gate rows and their 16 up rows of an expert;
// its wavefronts split the reduction and add their sums up in LDS, in order.
template <GroupElem EL, bool XF16, int NT>
__device__ __forceinline__ void few_up_tile(const FewArgs &a, const FewTokens &tk, int e, int it,
                                            int base, f32x4 (*red)[2][kWave]) {
  constexpr int ES = EL == kElemI8 ? 1 : 2;
  const int lane = threadIdx.x % kWave, wave = uniform((int)threadIdx.x / kWave);
  const int piece = lane / 16, col = lane % 16;
  FewStream<EL, false, XF16, 2, NT> st;
  st.abytes = a.H * ES;
  st.bbytes = a.H * 2;
  const int row = min(col, a.I - 1 - it * kFewRows);  // the last one where there are fewer
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    st.a[i] = uniform(a.w13 + (((int64_t)e * 2 + i) * a.I + it * kFewRows) * st.abytes);
    st.arow[i] = (uint32_t)row * st.abytes + piece * 16;
  }
  st.b = a.x;
  st.plane = 0;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int want = base + n * 16 + col;
    const int pair = __shfl(tk.pair, want < tk.count ? want : base, kWave);
    st.brow[n] = (uint32_t)(pair / a.K) * st.bbytes + piece * 16 * st.HALVES;
  }
  st.clear();
  const int pieces = few_pieces(st.abytes);
  st.run(pieces * wave / kFewWaves * kFewPiece,
         min(pieces * (wave + 1) / kFewWaves * kFewPiece, few_steps(st.abytes)));

#pragma unroll
  for (int n = 0; n < NT; ++n) {
    red[wave][0][lane] = st.acc[0][n];
    red[wave][1][lane] = st.acc[1][n];
    __syncthreads();
    if (wave == 0) {
      f32x4 g = red[0][0][lane], u = red[0][1][lane];
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) {
        g += red[w][0][lane];
        u += red[w][1][lane];
      }
      // this lane: rows 4 piece .. of the tile, token `want`
      const int want = base + n * 16 + col, i0 = it * kFewRows + piece * 4;
      const int pair = __shfl(tk.pair, want < tk.count ? want : base, kWave);
      uint16_t hi[4], lo[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float h = 0.0f;
        if (i0 + v < a.I) {
          float gv = g[v], uv = u[v];
          if constexpr (EL == kElemI8) {
            gv *= a.s13[(int64_t)e * 2 * a.I + i0 + v];
            uv *= a.s13[((int64_t)e * 2 + 1) * a.I + i0 + v];
          }
          h = silu(gv) * uv;
        }
        hi[v] = f32_to_bf16_rne(h);
        const float left = h - from_half_bits<false>(hi[v]);
        // (an infinite or NaN h is whole in its high part)
        lo[v] = left == left ? f32_to_bf16_rne(left) : 0;
      }
      if (want < tk.count) {
        uint16_t *out = a.h + (int64_t)pair * a.Ipad + i0;
        __builtin_memcpy(out, hi, 8);
        __builtin_memcpy(out + a.plane, lo, 8);
        // the padding behind the last tile
        if ((it + 1) * kFewRows >= a.I)
          for (int c = (it + 1) * kFewRows + piece * 4; c < a.Ipad; c += 16) {
            __builtin_memset(a.h + (int64_t)pair * a.Ipad + c, 0, 8);
            __builtin_memset(a.h + a.plane + (int64_t)pair * a.Ipad + c, 0, 8);
          }
      }
    }
    __syncthreads();
  }
}

template <GroupElem EL, bool XF16>
__global__ __launch_bounds__(kFewThreads, 4) void few_up_kernel(FewArgs a) {
  __shared__ FewIds s;
  __shared__ f32x4 red[kFewWaves][2][kWave];
  few_read_ids(a, s);
  const FewExperts ex(s);
  const int tiles = (a.I + kFewRows - 1) / kFewRows;
  for (int L = blockIdx.x; L < ex.count * tiles; L += gridDim.x) {
    const int rank = L / tiles, e = ex.at(rank);
    FewTokens tk;
    tk.template find<false>(a, s, e);
    for (int base = 0; base < tk.count; base += 32) {
      if (tk.count - base <= 16)
        few_up_tile<EL, XF16, 1>(a, tk, e, L - rank * tiles, base, red);
      else
        few_up_tile<EL, XF16, 2>(a, tk, e, L - rank * tiles, base, red);
    }
  }
}

// ----------------------------------------------------------------- down --
// A workgroup owns 16 output columns of all tokens.  Its wavefronts split the
// reduction over all experts in use, end to end, into equal ranges; each keeps
// its own sums of the tokens in LDS, and they are added up in order.
template <GroupElem EL, int NT>
__device__ __forceinline__ void few_down_part(const FewArgs &a, const FewTokens &tk, int e, int n0,
                                              int base, int from, int to, float *mine) {
  constexpr int ES = EL == kElemI8 ? 1 : 2;
  const int lane = threadIdx.x % kWave, piece = lane / 16, col = lane % 16;
  FewStream<EL, true, false, 1, NT> st;
  st.abytes = a.I * ES;
  st.bbytes = a.Ipad * 2;
  st.a[0] = uniform(a.w2 + ((int64_t)e * a.H + n0) * st.abytes);
  st.arow[0] = (uint32_t)min(col, a.H - 1 - n0) * st.abytes + piece * 16;
  st.b = (const char *)a.h;
  st.plane = a.plane * 2;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int want = base + n * 16 + col;
    const int pair = __shfl(tk.pair, want < tk.count ? want : base, kWave);
    st.brow[n] = (uint32_t)pair * st.bbytes + piece * 16 * st.HALVES;
  }
  st.clear();
  st.run(from, to);
  f32x4 sc = {1.0f, 1.0f, 1.0f, 1.0f};
  if constexpr (EL == kElemI8) {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      sc[v] = a.s2[(int64_t)e * a.H + min(n0 + piece * 4 + v, a.H - 1)];
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int want = base + n * 16 + col;
    const int at = want < tk.count ? want : base;
    const float share = __shfl(tk.share, at, kWave);
    const int t = __shfl(tk.pair, at, kWave) / a.K;
    if (want < tk.count) {
      f32x4 *sum = (f32x4 *)(mine + t * kFewRows + piece * 4);
      *sum += st.acc[0][n] * sc * share;
    }
  }
}

template <GroupElem EL, bool XF16>
__global__ __launch_bounds__(kFewThreads, 4) void few_down_kernel(FewArgs a) {
  __shared__ FewIds s;
  __shared__ __align__(16) float sums[kFewWaves][kFewMaxTokens * kFewRows];
  const int wave = uniform((int)threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int n0 = blockIdx.x * kFewRows;
  for (int i = lane; i < a.T * kFewRows; i += kWave) sums[wave][i] = 0.0f;
  few_read_ids(a, s);
  const FewExperts ex(s);
  constexpr int ES = EL == kElemI8 ? 1 : 2;
  const int steps = few_steps(a.I * ES), pieces = few_pieces(a.I * ES);
  const int64_t all = (int64_t)ex.count * pieces;
  const int64_t from = all * wave / kFewWaves, to = all * (wave + 1) / kFewWaves;
  for (int64_t c = from; c < to;) {
    const int rank = (int)(c / pieces), at = (int)(c - (int64_t)rank * pieces);
    const int n = (int)min((int64_t)(pieces - at), to - c);
    const int k0 = at * kFewPiece, k1 = min((at + n) * kFewPiece, steps);
    const int e = ex.at(rank);
    FewTokens tk;
    tk.template find<true>(a, s, e);
    for (int base = 0; base < tk.count; base += 32) {
      if (tk.count - base <= 16)
        few_down_part<EL, 1>(a, tk, e, n0, base, k0, k1, sums[wave]);
      else
        few_down_part<EL, 2>(a, tk, e, n0, base, k0, k1, sums[wave]);
    }
    c += n;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * kFewRows; i += kFewThreads) {
    const int t = i / kFewRows, n = n0 + i % kFewRows;
    float v = sums[0][i];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += sums[w][i];
    if (n < a.H) ((uint16_t *)a.out)[(int64_t)t * a.H + n] = to_half_bits<XF16>(v);
  }
}

template <GroupElem EL, bool XF16>
hipError_t launch_few(const FewArgs &a, hipStream_t st) {
  const int64_t pairs = (int64_t)a.T * a.K;
  const int64_t tiles = std::min<int64_t>(pairs, a.E) * ((a.I + kFewRows - 1) / kFewRows);
  const int64_t grid = std::min<int64_t>(tiles, 2 * kNumCus);
  hipLaunchKernelGGL((few_up_kernel<EL, XF16>), dim3((uint32_t)grid), dim3(kFewThreads), 0, st, a);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL((few_down_kernel<EL, XF16>), dim3((uint32_t)((a.H + kFewRows - 1) / kFewRows)),
                     dim3(kFewThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_few(bool f16, bool i8, const FewArgs &a, hipStream_t st) {
  if (i8) return f16 ? launch_few<kElemI8, true>(a, st) : launch_few<kElemI8, false>(a, st);
  return f16 ? launch_few<kElemF16, true>(a, st) : launch_few<kElemBf16, false>(a, st);
}

}  // namespace cco
