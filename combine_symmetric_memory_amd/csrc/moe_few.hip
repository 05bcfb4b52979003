// moe_few.hip -- a whole mixture-of-experts layer for a few tokens in two or
// three launches (include/cco_ops.h):
//
//   h[t, e] = silu(Wg_e x[t]) * (Wu_e x[t])
//   out[t]  = sum_e share[t][e] W2_e h[t, e]
//
// Bound by the weights of the experts that some token has, each read once, and
// again, mostly from the caches, for every further 32 tokens of an expert.
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
//
// What carries the stream is that a wavefront asks for the next 8 KiB of
// weights before it multiplies a chunk, over the ends of tiles and experts too,
// with eight wavefronts a CU that need 256 registers a lane for it: 16
// wavefronts of 128 registers, which spill, took 1.25 to 1.4 times as long,
// chunks of 16 KiB 1.1 to 1.4 times.  The weights do not stay in flight
// throughout: by a chunk's last product the compiler's waits for its columns
// are for everything (it counts the paths of a row's middle and of its end as
// one), a tile or an expert begins with rows moved between registers behind
// such a wait, the scales of 8-bit gate and up weights are read behind the next
// tile's rows, and the kernels that spill (8-bit weights: gate and up split over
// wavefronts, 84 bytes a lane, down with two tiles of rows, 44; fp16: the
// latter, 20) reload between tiles and experts.  The CU's other wavefronts
// cover that.
// Of the experts in use, one token of 256 of 7168 x 2048, top-8, bf16: gate and
// up 5.9 TB/s, down 5.4; 16 tokens with 8-bit weights 5.5 and, in the form with
// shared rows, 4.6.
#include "few_common.h"

namespace cco {
namespace {

// Tiles of 16 tokens multiplied at once.  (With four the 8-bit forms spill; an
// expert of more than 32 tokens has its weights read again, from the caches.)
constexpr int kFewColumns = 2;

// The product of MT tiles of weight rows with the columns of an expert's
// tokens.  EL: the weights' elements.  PAIR: the columns are h, in two planes;
// otherwise x, of the weights' type or, with 8-bit weights, fp16 (XF16) or
// bf16.
//
// The reduction goes by chunks of U steps.  The weights of the next chunk, be
// it the same expert's or the next one's, are asked for before a chunk is
// multiplied, behind its columns, which the caches hold and which come UB steps
// at a time, so that they take few registers.
//
// Weight rows of fewer than 16 bytes are read byte by byte: in the down product
// (PAIR) by kernels of their own (TINY), since beside the other loads that path
// cost its kernels 12 to 68 bytes of scratch a lane (4 tokens, 8 experts of
// 256 x 512, fp16: 8.9 us, without 6.6; one token of 256 of 7168 x 2048 in all
// 135 and 130), in the gate and up product beside them, which took the same
// change badly (64 tokens, 8 experts of 4096 x 14336, in all 613 and 625).
template <GroupElem EL, bool PAIR, bool XF16, int MT, bool TINY>
struct FewStream {
  static_assert(PAIR || !TINY, "");
  static constexpr int HALVES = EL == kElemI8 ? 2 : 1;  // 16-byte pieces of a column a step
  static constexpr int NB = (PAIR ? 2 : 1) * HALVES;
  static constexpr int U = TINY ? 1 : PAIR && EL == kElemI8 ? 4 : 8 / MT;
  // pieces of columns in registers at once; conversions need some themselves
  static constexpr int kColumnPieces = EL == kElemI8 ? 8 : 16;
  template <int NT>
  static constexpr int UB = kColumnPieces / (NT * NB) < U ? kColumnPieces / (NT * NB) : U;
  struct Rows {
    u32x4 v[U][MT];
  };
  struct Tiles {
    GlobalBytes *a[MT];  // uniform: first rows of the tiles
  };
  uint32_t arow[MT];  // this lane's row in the tiles and its piece of a step, in bytes
  int piece;          // which 16 bytes of a step are this lane's
  int abytes;         // bytes of a weight row
  GlobalBytes *b;     // uniform: x, or h
  int bbytes;         // bytes of a column that may be read

  // Chunks of a row, the last one's end included.
  __device__ __forceinline__ int chunks() const {
    return (abytes + U * kFewStepBytes - 1) / (U * kFewStepBytes);
  }
  // Whether rows end inside chunk c.
  __device__ __forceinline__ bool ends(int c) const {
    return (c + 1) * U * kFewStepBytes > abytes;
  }

  __device__ __forceinline__ void load_rows(Rows &r, const Tiles &t, int c) const {
    if constexpr (TINY) {  // all of the row is in the first piece
#pragma unroll
      for (int i = 0; i < MT; ++i)
        r.v[0][i] = load16(t.a[i] + (arow[i] - piece * 16), piece == 0 ? abytes : 0);
      return;
    }
    if (!ends(c)) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          r.v[u][i] = load16(t.a[i] + (arow[i] + c * U * kFewStepBytes) + u * kFewStepBytes);
      return;
    }
    if (!PAIR && abytes < 16) {  // all of the row is in the first piece
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          r.v[u][i] = u == 0 ? load16(t.a[i] + (arow[i] - piece * 16), piece == 0 ? abytes : 0)
                             : u32x4{0, 0, 0, 0};
      return;
    }
    // pieces that would pass the row's end take its last 16 bytes
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        r.v[u][i] = load16(t.a[i] + (arow[i] - piece * 16 +
                                     (uint32_t)min((c * U + u) * kFewStepBytes + piece * 16,
                                                   abytes - 16)));
    // (keeps the compiler from one set of loads for both cases, at addresses
    // of 64 bits each)
    asm volatile("" ::: "memory");
  }
  // What lies behind the row's end in its last chunk becomes zeros.
  __device__ __forceinline__ void cut_rows(Rows &r, int c) const {
    if (TINY || (!PAIR && abytes < 16)) return;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        r.v[u][i] = end_cut(r.v[u][i], (c * U + u) * kFewStepBytes + piece * 16, abytes);
        asm volatile("" : "+v"(r.v[u][i]));  // one after the other, in few registers
      }
  }
  // acc += the product over chunk c, whose rows are `now`; with `ahead` the
  // rows of chunk nc of tiles nt are put in flight into `next`.
  template <int NT>
  __device__ __forceinline__ void chunk(f32x4 (&acc)[MT][NT], Rows &now, int c,
                                        const uint32_t (&brow)[NT], Rows &next, bool ahead,
                                        const Tiles &nt, int nc) const {
    constexpr int G = UB<NT>;
    const bool end = ends(c);
#pragma unroll
    for (int u0 = 0; u0 < U; u0 += G) {
      u32x4 col[G][NT][NB];
      const int s = (c * U + u0) * kFewStepBytes * HALVES;
      if (PAIR || !end) {
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < NB; ++h)
              col[u][n][h] = load16(b + (h / HALVES) * bbytes + (brow[n] + s) +
                                    (u * kFewStepBytes * HALVES + (h % HALVES) * 16));
      } else {
        // x ends with the row (h is padded with zeros to whole chunks)
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < NB; ++h) {
              const int in = piece * 16 * HALVES;
              const int at = s + u * kFewStepBytes * HALVES + in + h * 16;
              const uint32_t row = brow[n] - in;
              if (abytes >= 16)
                col[u][n][h] = end_cut(load16(b + (row + (uint32_t)min(at, bbytes - 16))), at, bbytes);
              else  // (all of it is in the first piece, 32 bytes with 8-bit weights)
                col[u][n][h] = u0 + u == 0
                                   ? load16(b + (row + h * 16), piece == 0 ? bbytes - h * 16 : 0)
                                   : u32x4{0, 0, 0, 0};
              asm volatile("" : "+v"(col[u][n][h]));
            }
      }
      if (end && u0 == 0) cut_rows(now, c);
      if (u0 + G >= U && ahead) load_rows(next, nt, nc);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < G; ++u)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          few_multiply<EL, PAIR, XF16, NT, NB>(acc[i], now.v[u0 + u][i], col[u]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // Chunks [from, to) of tiles t.  The rows of the first are in flight into r0
  // when the range begins; with `more` those of chunk nc of tiles nt are when
  // it ends, into r0 again or, behind an odd number of chunks, into r1.
  template <int NT>
  __device__ __forceinline__ void run(f32x4 (&acc)[MT][NT], Rows &r0, Rows &r1, const Tiles &t,
                                      int from, int to, const uint32_t (&brow)[NT], bool more,
                                      const Tiles &nt, int nc) const {
    int c = from;
#pragma unroll 1
    for (; c + 2 <= to; c += 2) {
      chunk<NT>(acc, r0, c, brow, r1, true, t, c + 1);
      const bool last = c + 2 >= to;
      // the next range's where this one ends
      Tiles n;
#pragma unroll
      for (int i = 0; i < MT; ++i) n.a[i] = last ? nt.a[i] : t.a[i];
      chunk<NT>(acc, r1, c + 1, brow, r0, !last || more, n, last ? nc : c + 2);
    }
    if (c < to) chunk<NT>(acc, r0, c, brow, r1, more, nt, nc);
  }
};

// ---------------------------------------------------------- gate and up --
// Tiles of 16 gate rows and their 16 up rows of an expert.  With PARTS a
// workgroup's wavefronts split the reduction of a tile and add their sums up in
// LDS, in order; the sums of two tiles have room there, so one barrier a tile
// is enough: the wavefront that adds a tile up does so while the others go on.
// Otherwise (PARTS 1) each wavefront takes tiles of its own.
constexpr int kUpWaves = 4, kUpThreads = kUpWaves * kWave;
struct UpSums {
  f32x4 v[2][kUpWaves][kFewColumns][2][kWave];
};

template <GroupElem EL, bool XF16, int PARTS>
struct FewUp {
  using Stream = FewStream<EL, false, XF16, 2, false>;
  static constexpr int ES = EL == kElemI8 ? 1 : 2;

  __device__ static __forceinline__ typename Stream::Tiles tiles_of(const FewArgs &a, int e,
                                                                    int it) {
    typename Stream::Tiles t;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      t.a[i] = uniform_bytes(a.w13 + (((int64_t)e * 2 + i) * a.I + first_row(a, it)) * (a.H * ES));
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
    if constexpr (PARTS > 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        red[wave][n][0][lane] = acc[0][n];
        red[wave][n][1][lane] = acc[1][n];
      }
      __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 g = acc[0][n], u = acc[1][n];
      if constexpr (PARTS > 1) {
        if ((turn + n) % PARTS != wave) continue;
        g = red[0][n][0][lane];
        u = red[0][n][1][lane];
#pragma unroll
        for (int w = 1; w < PARTS; ++w) {
          g += red[w][n][0][lane];
          u += red[w][n][1][lane];
        }
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
        few_split(h, hi[v], lo[v]);
      }
      if (want < tk.count) {
        uint16_t *row = a.h + (int64_t)pair * 2 * a.Ipad;
        if (i0 + 4 <= a.I) {
          __builtin_memcpy(row + i0, hi, 8);
          __builtin_memcpy(row + a.Ipad + i0, lo, 8);
        } else {
          for (int v = 0; v < a.I - i0; ++v) {
            row[i0 + v] = hi[v];
            row[a.Ipad + i0 + v] = lo[v];
          }
        }
        // the padding behind the last tile
        if ((it + 1) * kFewRows >= a.I)
          for (int c = a.I + piece; c < a.Ipad; c += 4) row[c] = row[a.Ipad + c] = 0;
      }
    }
  }
};

template <GroupElem EL, bool XF16, int PARTS>
__global__ __launch_bounds__(kUpThreads, 2) void few_up_kernel(FewArgs a) {
  __shared__ uint32_t id_words[FewIds::words(kFewMaxTokens * kMaxTopk)];
  __shared__ UpSums sums;
  const FewIds s(id_words, a.T * a.K);
  using Up = FewUp<EL, XF16, PARTS>;
  using Stream = typename Up::Stream;
  few_read_ids<kUpThreads>(a, s);
  const FewExperts ex(s);
  const int lane = threadIdx.x % kWave, wave = uniform((int)threadIdx.x / kWave);
  const int tiles = (a.I + kFewRows - 1) / kFewRows, all = ex.count * tiles;
  Stream st;
  st.abytes = a.H * Up::ES;
  st.bbytes = a.H * 2;
  st.b = (GlobalBytes *)a.x;
  st.piece = lane / 16;
  st.arow[0] = st.arow[1] =
      (uint32_t)min(lane % 16, a.I - 1) * (uint32_t)st.abytes + st.piece * 16;
  const int chunks = st.chunks();
  const int from = PARTS > 1 ? chunks * wave / PARTS : 0;
  const int to = PARTS > 1 ? chunks * (wave + 1) / PARTS : chunks;
  int L = PARTS > 1 ? blockIdx.x : blockIdx.x * kUpWaves + wave;
  const int step = PARTS > 1 ? gridDim.x : gridDim.x * kUpWaves;
  if (L >= all) return;
  int e = ex.at(L / tiles), it = L % tiles;
  typename Stream::Tiles now = Up::tiles_of(a, e, it);
  typename Stream::Rows r0, r1;
  int turn = 0;
  bool flip = false;
  if (from < to) st.load_rows(r0, now, from);
  for (; L < all; L += step) {
    FewTokens tk;
    tk.find(a, s, e);
    const bool more = L + step < all;
    const int ne = more ? ex.at((L + step) / tiles) : e;
    const int nit = more ? (L + step) % tiles : it;
    typename Stream::Tiles nt = Up::tiles_of(a, ne, nit);
    for (int base = 0; base < tk.count; base += 16 * kFewColumns) {
      const bool again = base + 16 * kFewColumns < tk.count;
      const typename Stream::Tiles then = again ? now : nt;
      auto columns = [&](auto nt_c, typename Stream::Rows &x, typename Stream::Rows &y)
                         __attribute__((always_inline)) {
        Up::template tile<decltype(nt_c)::value>(a, st, x, y, tk, e, it, base, now, from, to,
                                                 more || again, then, sums, turn);
      };
      auto tile = [&](typename Stream::Rows &x, typename Stream::Rows &y)
                      __attribute__((always_inline)) {
        if (tk.count - base <= 16)
          columns(std::integral_constant<int, 1>{}, x, y);
        else
          columns(std::integral_constant<int, 2>{}, x, y);
      };
      if (!flip)
        tile(r0, r1);
      else
        tile(r1, r0);
      flip ^= (to - from) % 2 != 0;
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
template <GroupElem EL, int MT, bool TINY>
struct FewDown {
  using Stream = FewStream<EL, true, false, MT, TINY>;
  static constexpr int ES = EL == kElemI8 ? 1 : 2;
  static constexpr int SUMS = MT * kFewRows;  // sums of a token

  __device__ static __forceinline__ typename Stream::Tiles tiles_of(const FewArgs &a, int e,
                                                                    int n0) {
    typename Stream::Tiles t;
#pragma unroll
    for (int i = 0; i < MT; ++i) t.a[i] = uniform_bytes(a.w2 + ((int64_t)e * a.H + n0) * (a.I * ES));
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
      brow[n] = (uint32_t)__shfl(tk.pair, want < tk.count ? want : base, kWave) * 2 * st.bbytes +
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

constexpr int kDownWaves = 8, kDownThreads = kDownWaves * kWave;

template <GroupElem EL, bool XF16, int MT, bool TINY>
__device__ __forceinline__ void few_down(const FewArgs &a) {
  using Down = FewDown<EL, MT, TINY>;
  using Stream = typename Down::Stream;
  constexpr int SUMS = Down::SUMS;
  __shared__ uint32_t id_words[FewIds::words(kFewMaxTokens * kMaxTopk)];
  const FewIds s(id_words, a.T * a.K);
  extern __shared__ __align__(16) float sums[];  // [kDownWaves][T][SUMS]
  const int wave = uniform((int)threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int n0 = blockIdx.x * a.cols;
  float *mine = sums + wave * a.T * SUMS;
  for (int i = lane; i < a.T * SUMS; i += kWave) mine[i] = 0.0f;
  few_read_ids<kDownThreads>(a, s);
  const FewExperts ex(s);
  Stream st;
  st.abytes = a.I * Down::ES;
  st.bbytes = a.Ipad * 2;
  st.b = (GlobalBytes *)a.h;
  st.piece = lane / 16;
  // rows past the workgroup's last repeat it
#pragma unroll
  for (int i = 0; i < MT; ++i)
    st.arow[i] = (uint32_t)min(min(i * kFewRows + lane % 16, a.cols - 1), a.H - 1 - n0) *
                     (uint32_t)st.abytes +
                 st.piece * 16;
  const int chunks = st.chunks();
  const int64_t all = (int64_t)ex.count * chunks;
  const int64_t from = all * wave / kDownWaves, to = all * (wave + 1) / kDownWaves;
  if (from < to) {
    int rank = (int)(from / chunks), at = (int)(from - (int64_t)rank * chunks);
    int e = ex.at(rank);
    typename Stream::Tiles now = Down::tiles_of(a, e, n0);
    typename Stream::Rows r0, r1;
    st.load_rows(r0, now, at);
    bool flip = false;
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
        auto part = [&](typename Stream::Rows &x, typename Stream::Rows &y)
                        __attribute__((always_inline)) {
          if (tk.count - base <= 16)
            Down::template part<1>(a, st, x, y, tk, e, n0, base, now, at, at + n, more || again,
                                   then, tc, mine);
          else
            Down::template part<2>(a, st, x, y, tk, e, n0, base, now, at, at + n, more || again,
                                   then, tc, mine);
        };
        if (!flip)
          part(r0, r1);
        else
          part(r1, r0);
        flip ^= n % 2 != 0;
      }
      c += n;
      ++rank;
      at = 0;
      e = ne;
      now = nt;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * SUMS; i += kDownThreads) {
    const int t = i / SUMS, n = i % SUMS;
    float v = sums[i];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) v += sums[w * a.T * SUMS + i];
    if (n < a.cols && n0 + n < a.H)
      ((uint16_t *)a.out)[(int64_t)t * a.H + n0 + n] = to_half_bits<XF16>(v);
  }
}

template <GroupElem EL, bool XF16, int MT>
__global__ __launch_bounds__(kDownThreads, 2) void few_down_kernel(FewArgs a) {
  few_down<EL, XF16, MT, false>(a);
}
template <GroupElem EL, bool XF16>
__global__ __launch_bounds__(kDownThreads, 2) void few_tiny_down_kernel(FewArgs a) {
  few_down<EL, XF16, 1, true>(a);
}

hipError_t launch_down(void (*kernel)(FewArgs), const FewArgs &a, int sums, hipStream_t st) {
  const int lds = kDownWaves * a.T * sums * (int)sizeof(float);
  hipLaunchKernelGGL(kernel, dim3((uint32_t)((a.H + a.cols - 1) / a.cols)), dim3(kDownThreads),
                     lds, st, a);
  return hipGetLastError();
}

// Whether a wavefront takes whole tiles instead of a part of the reduction of
// each: where there are tiles for all of them, and rows of few chunks, of which
// a part is soon over, or of 8-bit weights.  Parts and whole, in us: 37 experts
// of 1001 x 1419, 8-bit weights, 69 and 62; 256 of 7168 x 2048, 8-bit weights,
// 16 tokens 700 and 640; 64 of 256 x 2048, bf16, 47 and 37, of 1024 x 2048 94
// and 93, but of 2048 x 2048 169 and 197.
template <GroupElem EL>
bool few_whole_tiles(const FewArgs &a, int64_t tiles) {
  return tiles >= 2 * kNumCus * kUpWaves && (EL == kElemI8 || a.H * 2 <= 2048);
}

template <GroupElem EL, bool XF16>
hipError_t launch_few(FewArgs a, hipStream_t st) {
  const int64_t pairs = (int64_t)a.T * a.K;
  const int64_t tiles = std::min<int64_t>(pairs, a.E) * ((a.I + kFewRows - 1) / kFewRows);
  if (few_whole_tiles<EL>(a, tiles)) {
    const int64_t grid = std::min<int64_t>((tiles + kUpWaves - 1) / kUpWaves, 2 * kNumCus);
    hipLaunchKernelGGL((few_up_kernel<EL, XF16, 1>), dim3((uint32_t)grid), dim3(kUpThreads), 0, st,
                       a);
  } else {
    const int64_t grid = std::min<int64_t>(tiles, 2 * kNumCus);
    hipLaunchKernelGGL((few_up_kernel<EL, XF16, kUpWaves>), dim3((uint32_t)grid),
                       dim3(kUpThreads), 0, st, a);
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  if (a.parts > 0) return launch_few_shared(XF16, EL == kElemI8, a, st);
  if (a.I * (EL == kElemI8 ? 1 : 2) < 16) {
    a.cols = kFewRows;
    return launch_down(few_tiny_down_kernel<EL, XF16>, a, kFewRows, st);
  }
  // one workgroup on every CU, or whole rounds of them
  const int rounds = (a.H + 32 * kNumCus - 1) / (32 * kNumCus);
  a.cols = std::max(kFewRows, (a.H + rounds * kNumCus - 1) / (rounds * kNumCus));
  return a.cols > kFewRows ? launch_down(few_down_kernel<EL, XF16, 2>, a, 2 * kFewRows, st)
                           : launch_down(few_down_kernel<EL, XF16, 1>, a, kFewRows, st);
}

}  // namespace

hipError_t launch_moe_few(bool f16, bool i8, const FewArgs &a, hipStream_t st) {
  if (i8) return f16 ? launch_few<kElemI8, true>(a, st) : launch_few<kElemI8, false>(a, st);
  return f16 ? launch_few<kElemF16, true>(a, st) : launch_few<kElemBf16, false>(a, st);
}

}  // namespace cco
