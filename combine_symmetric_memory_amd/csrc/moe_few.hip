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

constexpr int kFewRows = 16;       // weight rows of an MFMA
constexpr int kFewStepBytes = 64;  // bytes of a weight row a step takes

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ u32x4 load16(const char *p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
// 16 bytes at p, of which the first `have` exist; the others are zeros.
__device__ __forceinline__ u32x4 load16(const char *p, int have) {
  if (have >= 16) return load16(p);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < have) v[i / 4] |= (uint32_t)(uint8_t)p[i] << (8 * (i % 4));
  return v;
}

// Tiles of 16 tokens multiplied at once.  (With four the 8-bit forms spill; an
// expert of more than 32 tokens has its weights read again, from the caches.)
constexpr int kFewColumns = 2;

// The ids and weights of a call in LDS, and the experts in use.
struct FewIds {
  uint32_t live[kMaxExperts / 32];
  int32_t ids[kFewMaxTokens * kMaxTopk];
  float w[kFewMaxTokens * kMaxTopk];
};

template <int THREADS>
__device__ __forceinline__ void few_read_ids(const FewArgs &a, FewIds &s) {
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

// The product of MT tiles of weight rows with the columns of an expert's
// tokens.  EL: the weights' elements.  PAIR: the columns are h, in two planes;
// otherwise x, of the weights' type or, with 8-bit weights, fp16 (XF16) or
// bf16.
//
// The reduction goes by chunks of U steps.  The weights of the next chunk, be
// it the same expert's or the next one's, are in flight while a chunk is
// multiplied; its columns, which the caches hold, are issued before them and
// waited for alone, UB steps at a time, so that they take few registers.  What
// a row has behind its last whole chunk goes step by step.
template <GroupElem EL, bool PAIR, bool XF16, int MT>
struct FewStream {
  static constexpr int HALVES = EL == kElemI8 ? 2 : 1;  // 16-byte pieces of a column a step
  static constexpr int NB = (PAIR ? 2 : 1) * HALVES;
  static constexpr int U = PAIR && EL == kElemI8 ? 4 : 8 / MT;
  template <int NT>
  static constexpr int UB = NT * NB >= 16 ? 1 : (16 / (NT * NB) < U ? 16 / (NT * NB) : U);
  struct Rows {
    u32x4 v[U][MT];
  };
  struct Tiles {
    const char *a[MT];  // uniform: first rows of the tiles
  };
  uint32_t arow[MT];  // this lane's row in the tiles and its piece of a step, in bytes
  int piece;          // which 16 bytes of a step are this lane's
  int abytes;         // bytes of a weight row
  const char *b;      // uniform: x, or the high plane of h
  uint64_t plane;     // bytes between the planes of h
  int bbytes;         // bytes of a column that may be read

  // Chunks of a row, the last one's end included, and those that are whole.
  __device__ __forceinline__ int chunks() const {
    return (abytes + U * kFewStepBytes - 1) / (U * kFewStepBytes);
  }
  __device__ __forceinline__ int whole() const { return abytes / (U * kFewStepBytes); }

  __device__ __forceinline__ void load_rows(Rows &r, const Tiles &t, int c) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        r.v[u][i] = load16(t.a[i] + (arow[i] + c * U * kFewStepBytes) + u * kFewStepBytes);
  }
  // acc += the product over the whole chunk c, whose rows are `now`; with
  // `ahead` the rows of chunk nc of tiles nt are put in flight into `next`.
  template <int NT>
  __device__ __forceinline__ void chunk(f32x4 (&acc)[MT][NT], const Rows &now, int c,
                                        const uint32_t (&brow)[NT], Rows &next, bool ahead,
                                        const Tiles &nt, int nc) const {
    constexpr int G = UB<NT>;
#pragma unroll
    for (int u0 = 0; u0 < U; u0 += G) {
      u32x4 col[G][NT][NB];
      const int s = (c * U + u0) * kFewStepBytes * HALVES;
#pragma unroll
      for (int u = 0; u < G; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < NB; ++h)
            col[u][n][h] = load16(b + (h / HALVES) * plane + (brow[n] + s) +
                                  (u * kFewStepBytes * HALVES + (h % HALVES) * 16));
      if (u0 + G >= U && ahead) load_rows(next, nt, nc);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < G; ++u)
#pragma unroll
        for (int i = 0; i < MT; ++i) multiply<NT>(acc[i], now.v[u0 + u][i], col[u]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // acc += the product over step s, in or behind which rows end.
  template <int NT>
  __device__ __forceinline__ void step(f32x4 (&acc)[MT][NT], const Tiles &t, int s,
                                       const uint32_t (&brow)[NT]) const {
    u32x4 col[NT][NB], w[MT];
    const int at = s * kFewStepBytes + piece * 16;
#pragma unroll
    for (int i = 0; i < MT; ++i)
      w[i] = load16(t.a[i] + arow[i] + s * kFewStepBytes, abytes - at);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < NB; ++h) {
        const int in = (h % HALVES) * 16;
        col[n][h] = load16(b + (h / HALVES) * plane + brow[n] + s * kFewStepBytes * HALVES + in,
                           bbytes - at * HALVES - in);
      }
#pragma unroll
    for (int i = 0; i < MT; ++i) multiply<NT>(acc[i], w[i], col);
  }
  template <int NT>
  static __device__ __forceinline__ void multiply(f32x4 (&acc)[NT], u32x4 w,
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
        // (the product of the two low parts is 2^-16 of the whole)
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
  // Chunks [from, to) of tiles t.  The rows of a range's first whole chunk are
  // in flight into r0 when it begins; with `more` those of chunk nc of tiles
  // nt are when it ends (if that chunk is whole).
  template <int NT>
  __device__ __forceinline__ void run(f32x4 (&acc)[MT][NT], Rows &r0, Rows &r1, const Tiles &t,
                                      int from, int to, const uint32_t (&brow)[NT], bool more,
                                      const Tiles &nt, int nc) const {
    const int in = min(to, whole());
    more = more && nc < whole();
    int c = from;
#pragma unroll 1
    for (; c + 2 <= in; c += 2) {
      chunk<NT>(acc, r0, c, brow, r1, true, t, c + 1);
      const bool last = c + 2 >= in;
      // the next range's where this one ends
      Tiles n;
#pragma unroll
      for (int i = 0; i < MT; ++i) n.a[i] = last ? nt.a[i] : t.a[i];
      chunk<NT>(acc, r1, c + 1, brow, r0, !last || more, n, last ? nc : c + 2);
    }
    if (c < in) chunk<NT>(acc, r0, c, brow, r1, false, t, c);
    // (an even range's are on their way)
    if ((c < in || from >= in) && more) load_rows(r0, nt, nc);
    if (to > in) {
      const int end = (abytes + kFewStepBytes - 1) / kFewStepBytes;
#pragma unroll 1
      for (int s = in * U; s < end; ++s) step<NT>(acc, t, s, brow);
    }
  }
};

// ---------------------------------------------------------- gate and up --
// A workgroup takes tiles of 16 gate rows and their 16 up rows of an expert;
// its wavefronts split the reduction and add their sums up in LDS, in order.
// The sums of two tiles have room there, so one barrier a tile is enough: the
// wavefront that adds a tile up does so while the others go on.
constexpr int kUpWaves = 4, kUpThreads = kUpWaves * kWave;
struct UpSums {
  f32x4 v[2][kUpWaves][kFewColumns][2][kWave];
};

template <GroupElem EL, bool XF16>
struct FewUp {
  using Stream = FewStream<EL, false, XF16, 2>;
  static constexpr int ES = EL == kElemI8 ? 1 : 2;

  __device__ static __forceinline__ typename Stream::Tiles tiles_of(const FewArgs &a, int e,
                                                                    int it) {
    typename Stream::Tiles t;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      t.a[i] = uniform(a.w13 + (((int64_t)e * 2 + i) * a.I + first_row(a, it)) * (a.H * ES));
    return t;
  }
  // The last tile lies back so that it is whole (its first rows are computed
  // twice, alike); only experts of fewer than 16 rows have tiles that are not.
  __device__ static __forceinline__ int first_row(const FewArgs &a, int it) {
    return max(0, min(it * kFewRows, a.I - kFewRows));
  }

  // Tile `it` of expert e for its tokens base .. base + 16 NT - 1.
  template <int NT>
  __device__ static __forceinline__ void tile(const FewArgs &a, Stream &st,
                                              typename Stream::Rows &r0, typename Stream::Rows &r1,
                                              const FewTokens &tk, int e, int it, int base,
                                              const typename Stream::Tiles &now, int from, int to,
                                              bool more, const typename Stream::Tiles &nt,
                                              UpSums &sums, int turn) {
    const int lane = threadIdx.x % kWave, wave = uniform((int)threadIdx.x / kWave);
    const int col = lane % 16, piece = lane / 16;
    uint32_t brow[NT];
    f32x4 acc[2][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int want = base + n * 16 + col;
      const int pair = __shfl(tk.pair, want < tk.count ? want : base, kWave);
      brow[n] = (uint32_t)(pair / a.K) * st.bbytes + piece * 16 * st.HALVES;
      acc[0][n] = acc[1][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    st.template run<NT>(acc, r0, r1, now, from, to, brow, more, nt, from);
    auto &red = sums.v[turn & 1];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      red[wave][n][0][lane] = acc[0][n];
      red[wave][n][1][lane] = acc[1][n];
    }
    __syncthreads();
#pragma unroll 1
    for (int n = 0; n < NT; ++n) {
      if ((turn + n) % kUpWaves != wave) continue;
      f32x4 g = red[0][n][0][lane], u = red[0][n][1][lane];
#pragma unroll
      for (int w = 1; w < kUpWaves; ++w) {
        g += red[w][n][0][lane];
        u += red[w][n][1][lane];
      }
      // this lane: rows 4 piece .. of the tile, token `want`
      const int want = base + n * 16 + col, i0 = first_row(a, it) + piece * 4;
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
        uint16_t *row = a.h + (int64_t)pair * a.Ipad;
        if (i0 + 4 <= a.I) {
          __builtin_memcpy(row + i0, hi, 8);
          __builtin_memcpy(row + a.plane + i0, lo, 8);
        } else {
          for (int v = 0; v < a.I - i0; ++v) {
            row[i0 + v] = hi[v];
            row[a.plane + i0 + v] = lo[v];
          }
        }
        // the padding behind the last tile
        if ((it + 1) * kFewRows >= a.I)
          for (int c = a.I + piece; c < a.Ipad; c += 4) row[c] = row[a.plane + c] = 0;
      }
    }
  }
};

template <GroupElem EL, bool XF16>
__global__ __launch_bounds__(kUpThreads, 2) void few_up_kernel(FewArgs a) {
  __shared__ FewIds s;
  __shared__ UpSums sums;
  using Up = FewUp<EL, XF16>;
  using Stream = typename Up::Stream;
  few_read_ids<kUpThreads>(a, s);
  const FewExperts ex(s);
  const int lane = threadIdx.x % kWave, wave = uniform((int)threadIdx.x / kWave);
  const int tiles = (a.I + kFewRows - 1) / kFewRows, all = ex.count * tiles;
  Stream st;
  st.abytes = a.H * Up::ES;
  st.bbytes = a.H * 2;
  st.b = a.x;
  st.plane = 0;
  st.piece = lane / 16;
  st.arow[0] = st.arow[1] =
      (uint32_t)min(lane % 16, a.I - 1) * (uint32_t)st.abytes + st.piece * 16;
  const int chunks = st.chunks();
  const int from = chunks * wave / kUpWaves, to = chunks * (wave + 1) / kUpWaves;
  int L = blockIdx.x;
  if (L >= all) return;
  int e = ex.at(L / tiles), it = L % tiles;
  typename Stream::Tiles now = Up::tiles_of(a, e, it);
  typename Stream::Rows r0, r1;
  int turn = 0;
  if (from < min(to, st.whole())) st.load_rows(r0, now, from);
  for (; L < all; L += gridDim.x) {
    FewTokens tk;
    tk.find(a, s, e);
    const bool more = L + (int)gridDim.x < all;
    const int ne = more ? ex.at((L + gridDim.x) / tiles) : e;
    const int nit = more ? (L + gridDim.x) % tiles : it;
    typename Stream::Tiles nt = Up::tiles_of(a, ne, nit);
    for (int base = 0; base < tk.count; base += 16 * kFewColumns) {
      const bool again = base + 16 * kFewColumns < tk.count;
      const typename Stream::Tiles then = again ? now : nt;
      if (tk.count - base <= 16)
        Up::template tile<1>(a, st, r0, r1, tk, e, it, base, now, from, to, more || again, then,
                             sums, turn);
      else
        Up::template tile<2>(a, st, r0, r1, tk, e, it, base, now, from, to, more || again, then,
                             sums, turn);
      ++turn;
    }
    now = nt;
    e = ne;
    it = nit;
  }
}

// ----------------------------------------------------------------- down --
// A workgroup owns a.cols output columns of all tokens, 16 or 32 at most.  Its
// wavefronts split the reduction over all experts in use, end to end, into
// equal ranges; each keeps its own sums of the tokens in LDS, and they are
// added up in order.
template <GroupElem EL, int MT>
struct FewDown {
  using Stream = FewStream<EL, true, false, MT>;
  static constexpr int ES = EL == kElemI8 ? 1 : 2;
  static constexpr int SUMS = MT * kFewRows;  // sums of a token

  __device__ static __forceinline__ typename Stream::Tiles tiles_of(const FewArgs &a, int e,
                                                                    int n0) {
    typename Stream::Tiles t;
#pragma unroll
    for (int i = 0; i < MT; ++i) t.a[i] = uniform(a.w2 + ((int64_t)e * a.H + n0) * (a.I * ES));
    return t;
  }

  template <int NT>
  __device__ static __forceinline__ void part(const FewArgs &a, Stream &st,
                                              typename Stream::Rows &r0, typename Stream::Rows &r1,
                                              const FewTokens &tk, int e, int n0, int base,
                                              const typename Stream::Tiles &now, int from, int to,
                                              bool more, const typename Stream::Tiles &nt, int nc,
                                              float *mine) {
    const int lane = threadIdx.x % kWave, piece = lane / 16, col = lane % 16;
    f32x4 sc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        sc[i][v] = EL == kElemI8 ? a.s2[(int64_t)e * a.H +
                                        min(n0 + i * kFewRows + piece * 4 + v, a.H - 1)]
                                 : 1.0f;
    uint32_t brow[NT];
    f32x4 acc[MT][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int want = base + n * 16 + col;
      brow[n] = (uint32_t)__shfl(tk.pair, want < tk.count ? want : base, kWave) * st.bbytes +
                piece * 16 * st.HALVES;
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    st.template run<NT>(acc, r0, r1, now, from, to, brow, more, nt, nc);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int want = base + n * 16 + col, at = want < tk.count ? want : base;
      const float share = __shfl(tk.share, at, kWave);
      const int t = __shfl(tk.pair, at, kWave) / a.K;
      if (want < tk.count)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          f32x4 *sum = (f32x4 *)(mine + t * SUMS + i * kFewRows + piece * 4);
          *sum += acc[i][n] * sc[i] * share;
        }
    }
  }
};

template <GroupElem EL, bool XF16, int MT, int WAVES>
__global__ __launch_bounds__(WAVES *kWave, WAVES <= 8 ? 2 : WAVES / 4) void few_down_kernel(
    FewArgs a) {
  using Down = FewDown<EL, MT>;
  using Stream = typename Down::Stream;
  constexpr int SUMS = Down::SUMS;
  __shared__ FewIds s;
  extern __shared__ __align__(16) float sums[];  // [WAVES][T][SUMS]
  const int wave = uniform((int)threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int n0 = blockIdx.x * a.cols;
  float *mine = sums + wave * a.T * SUMS;
  for (int i = lane; i < a.T * SUMS; i += kWave) mine[i] = 0.0f;
  few_read_ids<WAVES * kWave>(a, s);
  const FewExperts ex(s);
  Stream st;
  st.abytes = a.I * Down::ES;
  st.bbytes = a.Ipad * 2;
  st.b = (const char *)a.h;
  st.plane = a.plane * 2;
  st.piece = lane / 16;
  // rows past the workgroup's last repeat it
#pragma unroll
  for (int i = 0; i < MT; ++i)
    st.arow[i] = (uint32_t)min(min(i * kFewRows + lane % 16, a.cols - 1), a.H - 1 - n0) *
                     (uint32_t)st.abytes +
                 st.piece * 16;
  const int chunks = st.chunks();
  const int64_t all = (int64_t)ex.count * chunks;
  const int64_t from = all * wave / WAVES, to = all * (wave + 1) / WAVES;
  if (from < to) {
    int rank = (int)(from / chunks), at = (int)(from - (int64_t)rank * chunks);
    int e = ex.at(rank);
    typename Stream::Tiles now = Down::tiles_of(a, e, n0);
    typename Stream::Rows r0, r1;
    if (at < st.whole()) st.load_rows(r0, now, at);
    for (int64_t c = from; c < to;) {
      const int n = (int)min((int64_t)(chunks - at), to - c);
      const bool more = c + n < to;
      const int ne = more ? ex.at(rank + 1) : e;
      typename Stream::Tiles nt = Down::tiles_of(a, ne, n0);
      FewTokens tk;
      tk.find(a, s, e);
      for (int base = 0; base < tk.count; base += 16 * kFewColumns) {
        const bool again = base + 16 * kFewColumns < tk.count;
        const typename Stream::Tiles then = again ? now : nt;
        const int tc = again ? at : 0;
        if (tk.count - base <= 16)
          Down::template part<1>(a, st, r0, r1, tk, e, n0, base, now, at, at + n, more || again,
                                 then, tc, mine);
        else
          Down::template part<2>(a, st, r0, r1, tk, e, n0, base, now, at, at + n, more || again,
                                 then, tc, mine);
      }
      c += n;
      ++rank;
      at = 0;
      e = ne;
      now = nt;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * SUMS; i += WAVES * kWave) {
    const int t = i / SUMS, n = i % SUMS;
    float v = sums[i];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += sums[w * a.T * SUMS + i];
    if (n < a.cols && n0 + n < a.H)
      ((uint16_t *)a.out)[(int64_t)t * a.H + n0 + n] = to_half_bits<XF16>(v);
  }
}

template <GroupElem EL, bool XF16, int MT, int WAVES>
hipError_t launch_down(const FewArgs &a, hipStream_t st) {
  const int lds = WAVES * a.T * MT * kFewRows * (int)sizeof(float);
  hipLaunchKernelGGL((few_down_kernel<EL, XF16, MT, WAVES>),
                     dim3((uint32_t)((a.H + a.cols - 1) / a.cols)), dim3(WAVES * kWave), lds, st, a);
  return hipGetLastError();
}

template <GroupElem EL, bool XF16>
hipError_t launch_few(FewArgs a, hipStream_t st) {
  const int64_t pairs = (int64_t)a.T * a.K;
  const int64_t tiles = std::min<int64_t>(pairs, a.E) * ((a.I + kFewRows - 1) / kFewRows);
  const int64_t grid = std::min<int64_t>(tiles, 2 * kNumCus);
  hipLaunchKernelGGL((few_up_kernel<EL, XF16>), dim3((uint32_t)grid), dim3(kUpThreads), 0, st, a);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  // one workgroup on every CU, or whole rounds of them
  const int rounds = (a.H + 32 * kNumCus - 1) / (32 * kNumCus);
  a.cols = std::max(kFewRows, (a.H + rounds * kNumCus - 1) / (rounds * kNumCus));
  return a.cols > kFewRows ? launch_down<EL, XF16, 2, 8>(a, st)
                           : launch_down<EL, XF16, 1, 8>(a, st);
}

}  // namespace

hipError_t launch_moe_few(bool f16, bool i8, const FewArgs &a, hipStream_t st) {
  if (i8) return f16 ? launch_few<kElemI8, true>(a, st) : launch_few<kElemI8, false>(a, st);
  return f16 ? launch_few<kElemF16, true>(a, st) : launch_few<kElemBf16, false>(a, st);
}

}  // namespace cco
