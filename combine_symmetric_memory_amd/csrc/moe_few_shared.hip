// moe_few_shared.hip -- the down product of the layer for a few tokens, in the
// form that shares the tokens' rows (moe_few.hip has the mathematics, the gate
// and up product, and the other form).
//
// The four wavefronts of a workgroup take 16 output columns each over the same
// stretch of the reduction and share its tokens' rows of h in LDS, which
// direct loads fill a chunk ahead; a chunk's weights are asked for a chunk
// ahead too, and the barrier between chunks waits for both.  (At a segment's
// end rows move between registers behind such a wait, and 8-bit weights' scales
// are read behind the next segment's rows.)  Each wavefront for itself, as in
// the other form, loads one to four times the weights' bytes of h over its
// compute unit's load path, whatever the number of tokens (the columns that
// none fills included).  A workgroup takes one part of the reduction over all experts in use; the
// parts' sums, a few MB, are added up by another launch.
//
// Measured (down product alone): 8 experts of 4096 x 14336, 16 tokens each:
// 3.5 TB/s of weights, the other form 2.7; 2 tokens each 4.6 and 3.9.
#include "few_common.h"

namespace cco {
namespace {

constexpr int kWaves = 4, kThreads = kWaves * kWave;
constexpr int kFewBlock = kWaves * kFewRows;  // output columns of a workgroup

typedef __attribute__((address_space(3))) const u32x4 lds_piece_t;

// A stretch of the reduction of one expert: its first weight row for this
// workgroup, and its tokens [first, first + columns).
struct Segment {
  GlobalBytes *rows;
  FewTokens tk;
  int e, first, columns;
};

template <GroupElem EL>
struct SharedStream {
  static constexpr int HALVES = EL == kElemI8 ? 2 : 1;  // 16-byte pieces of a plane a step
  static constexpr int NB = 2 * HALVES;
  static constexpr int U = EL == kElemI8 ? 4 : 8;  // steps of a chunk
  static constexpr int CHUNK = U * kFewStepBytes;  // its bytes of a weight row
  static constexpr int PB = CHUNK * HALVES;        // ... of a column's plane
  static constexpr int ROW = PB * 2;               // ... of a column in LDS
  static_assert(ROW == 1024, "a direct load a column");
  struct Rows {
    u32x4 v[U];
  };
  uint32_t arow;     // this lane's row and its piece of a step, in bytes
  int abytes;        // bytes of a weight row
  const char *cols;  // h
  int bbytes;        // bytes of a plane, whole chunks
  char *slots;       // two of `columns` rows of ROW bytes
  int slot_bytes;

  __device__ __forceinline__ int chunks() const { return (abytes + CHUNK - 1) / CHUNK; }

  __device__ __forceinline__ void load_rows(Rows &r, GlobalBytes *at, int c) const {
    if ((c + 1) * CHUNK <= abytes) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        r.v[u] = load16(at + (arow + c * CHUNK) + u * kFewStepBytes);
      return;
    }
    // the row's end: pieces that would pass it take its last 16 bytes
    const int piece = (threadIdx.x % kWave) / 16 * 16;
#pragma unroll
    for (int u = 0; u < U; ++u)
      r.v[u] = load16(at + (arow - piece + (uint32_t)min(c * CHUNK + u * kFewStepBytes + piece,
                                                         abytes - 16)));
    // (keeps the compiler from one set of loads for both cases, at addresses
    // of 64 bits each)
    asm volatile("" ::: "memory");
  }
  // What lies behind the row's end in its last chunk becomes zeros.
  __device__ __forceinline__ void cut_rows(Rows &r, int c) const {
    const int piece = (threadIdx.x % kWave) / 16 * 16;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r.v[u] = end_cut(r.v[u], c * CHUNK + u * kFewStepBytes + piece, abytes);
      asm volatile("" : "+v"(r.v[u]));  // one after the other, in few registers
    }
  }

  // Chunk c of the segment's columns into the slot, each wavefront its share
  // of the loads.  Piece g of 16 bytes of a plane lies at g ^ (column % 8), so
  // that the 16 columns of a fragment read fall on distinct banks.
  __device__ __forceinline__ void load_columns(int slot, const Segment &s, int c) const {
    const int wave = uniform((int)threadIdx.x / kWave), lane = threadIdx.x % kWave;
#pragma unroll 1
    for (int n = wave; n < s.columns; n += kWaves) {
      const int pair = uniform(__shfl(s.tk.pair, s.first + n, kWave));
      const int p = lane * 16 / PB, g = (lane * 16 % PB / 16) ^ (n % 8);
      buffer_load_lds_16(byte_range_rsrc(cols + (int64_t)pair * 2 * bbytes, 2 * (uint32_t)bbytes),
                         (uint32_t)(p * bbytes + c * PB + g * 16), 0,
                         slots + slot * slot_bytes + n * ROW);
    }
  }

  // acc += the product over chunk c, whose rows are r and whose columns are in
  // the slot.
  template <int NT>
  __device__ __forceinline__ void multiply(f32x4 (&acc)[NT], Rows &r, int c, int slot,
                                           int columns) const {
    const int lane = threadIdx.x % kWave, piece = lane / 16;
    if ((c + 1) * CHUNK > abytes) cut_rows(r, c);
    uint32_t at[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = min(n * 16 + lane % 16, columns - 1);
      at[n] = lds_addr(slots) + slot * slot_bytes + col * ROW +
              (((piece * HALVES) ^ (col % 8)) * 16);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      u32x4 col[NT][NB];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int p = b / HALVES, h = b % HALVES;
          // piece u 4 HALVES + piece HALVES + h, its low three bits swizzled
          const uint32_t flip = HALVES == 2 ? (h ? 16 : 0) : (u % 2 ? 64 : 0);
          const int line = HALVES == 2 ? u * 128 : u / 2 * 128;
          col[n][b] = *(lds_piece_t *)(uintptr_t)((at[n] ^ flip) + p * PB + line);
        }
      few_multiply<EL, true, false, NT, NB>(acc, r.v[u], col);
    }
  }

  // Everything in flight has landed, for all wavefronts, and the other slot is
  // read out.
  static __device__ __forceinline__ void sync() {
    wait_vmcnt<0>();
    wait_lgkmcnt<0>();
    asm volatile("" ::: "memory");
    stage_barrier();
    asm volatile("" ::: "memory");
  }

  // Chunks [from, to) of segment s, the first of which is in flight: its rows
  // into r0, its columns into the slot.  With `more` the same then holds of
  // chunk nfrom of segment next.
  template <int NT>
  __device__ __forceinline__ void run(f32x4 (&acc)[NT], Rows &r0, Rows &r1, int &slot,
                                      const Segment &s, int from, int to, bool more,
                                      const Segment &next, int nfrom) const {
    int c = from;
#pragma unroll 1
    for (; c + 2 <= to; c += 2) {
      sync();
      load_columns(slot ^ 1, s, c + 1);
      load_rows(r1, s.rows, c + 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply<NT>(acc, r0, c, slot, s.columns);
      sync();
      if (c + 2 < to) {
        load_columns(slot, s, c + 2);
        load_rows(r0, s.rows, c + 2);
      } else if (more) {
        load_columns(slot, next, nfrom);
        load_rows(r0, next.rows, nfrom);
      }
      __builtin_amdgcn_sched_barrier(0);
      multiply<NT>(acc, r1, c + 1, slot ^ 1, s.columns);
    }
    if (c < to) {
      // an odd one: its registers are free only behind it
      sync();
      if (more) load_columns(slot ^ 1, next, nfrom);
      __builtin_amdgcn_sched_barrier(0);
      multiply<NT>(acc, r0, c, slot, s.columns);
      if (more) load_rows(r0, next.rows, nfrom);
      slot ^= 1;
    }
  }
};

// The next columns of the same expert, if it has more than fit one segment.
__device__ __forceinline__ bool more_tokens(Segment &s, int columns) {
  const int first = s.first + s.columns;
  if (first >= s.tk.count) return false;
  s.first = first;
  s.columns = min(columns, s.tk.count - first);
  return true;
}
__device__ __forceinline__ void tokens_of(const FewArgs &a, const FewIds &ids, Segment &s,
                                          int columns) {
  s.tk.find(a, ids, s.e);
  s.first = 0;
  s.columns = min(columns, s.tk.count);
}

// ----------------------------------------------------------------- down --
// A workgroup owns 64 output columns of all tokens, 16 a wavefront, over one
// part of the reduction over all experts in use, end to end.  Each wavefront
// keeps its sums in LDS.  With several parts they go to the workspace, where
// another launch adds them up, in order.
template <GroupElem EL>
struct SharedDown {
  using Stream = SharedStream<EL>;
  static constexpr int ES = EL == kElemI8 ? 1 : 2;

  template <int NT>
  __device__ static __forceinline__ void segment(const FewArgs &a, const Stream &st,
                                                 typename Stream::Rows &r0,
                                                 typename Stream::Rows &r1, int &slot,
                                                 const Segment &s, int n0, int from, int to,
                                                 bool more, const Segment &next, int nfrom,
                                                 float *mine) {
    const int lane = threadIdx.x % kWave, piece = lane / 16;
    f32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    st.template run<NT>(acc, r0, r1, slot, s, from, to, more, next, nfrom);
    f32x4 sc = {1.0f, 1.0f, 1.0f, 1.0f};
    if constexpr (EL == kElemI8)
      __builtin_memcpy(&sc, a.s2 + (int64_t)s.e * a.H + n0 + piece * 4, 16);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = n * 16 + lane % 16, at = s.first + min(col, s.columns - 1);
      const float share = __shfl(s.tk.share, at, kWave);
      const int t = __shfl(s.tk.pair, at, kWave) / a.K;
      if (col < s.columns) {
        f32x4 *sum = (f32x4 *)(mine + t * kFewRows + piece * 4);
        *sum += acc[n] * sc * share;
      }
    }
  }
};

template <GroupElem EL, bool XF16>
__global__ __launch_bounds__(kThreads, 2) void few_shared_down_kernel(FewArgs a, int columns) {
  using Down = SharedDown<EL>;
  using Stream = typename Down::Stream;
  extern __shared__ __align__(1024) char smem[];
  const int lane = threadIdx.x % kWave, wave = uniform((int)threadIdx.x / kWave);
  const int blocks = (a.H + kFewBlock - 1) / kFewBlock;
  const int part = blockIdx.x / blocks, block = blockIdx.x - part * blocks;
  // this wavefront's columns are own .. own + 15; the last ones' products
  // lie back so that they are whole
  const int own = block * kFewBlock + wave * kFewRows, n0 = min(own, a.H - kFewRows);
  Stream st;
  st.slots = smem;
  st.slot_bytes = columns * Stream::ROW;
  st.abytes = a.I * Down::ES;
  st.arow = (uint32_t)(lane % 16) * (uint32_t)st.abytes + lane / 16 * 16;
  st.cols = (const char *)a.h;
  st.bbytes = a.Ipad * 2;
  uint32_t *const words = (uint32_t *)(smem + 2 * st.slot_bytes);
  const FewIds ids(words, a.T * a.K);
  float *const mine =
      (float *)(words + (FewIds::words(a.T * a.K) + 3) / 4 * 4) + wave * a.T * kFewRows;
  for (int i = lane; i < a.T * kFewRows; i += kWave) mine[i] = 0.0f;
  few_read_ids<kThreads>(a, ids);
  const FewExperts ex(ids);
  const int chunks = st.chunks();
  const int64_t all = (int64_t)ex.count * chunks;
  const int64_t from = all * part / a.parts, to = all * (part + 1) / a.parts;
  if (from < to) {
    int rank = (int)(from / chunks), at = (int)(from - (int64_t)rank * chunks);
    auto segment_at = [&](Segment &s, int r) __attribute__((always_inline)) {
      s.e = ex.at(r);
      s.rows = uniform_bytes(a.w2 + ((int64_t)s.e * a.H + n0) * (int64_t)st.abytes);
      tokens_of(a, ids, s, columns);
    };
    Segment s;
    segment_at(s, rank);
    typename Stream::Rows r0, r1;
    int slot = 0;
    st.load_columns(slot, s, at);
    st.load_rows(r0, s.rows, at);
    int64_t c = from;
    for (;;) {
      const int n = (int)min((int64_t)(chunks - at), to - c);
      Segment next = s;
      bool more = more_tokens(next, columns);
      const bool again = more;
      if (!again) {
        more = c + n < to;
        if (more) segment_at(next, rank + 1);
      }
      const int nat = again ? at : 0;
      if (s.columns <= 16)
        Down::template segment<1>(a, st, r0, r1, slot, s, n0, at, at + n, more, next, nat, mine);
      else
        Down::template segment<2>(a, st, r0, r1, slot, s, n0, at, at + n, more, next, nat, mine);
      if (!more) break;
      if (!again) {
        c += n;
        ++rank;
        at = 0;
      }
      s = next;
    }
  }
  for (int i = lane; i < a.T * kFewRows; i += kWave) {
    const int t = i / kFewRows, n = n0 + i % kFewRows;
    if (n < own) continue;  // another wavefront's
    if (a.parts == 1)
      ((uint16_t *)a.out)[(int64_t)t * a.H + n] = to_half_bits<XF16>(mine[i]);
    else
      a.partial[((int64_t)part * a.T + t) * a.H + n] = mine[i];
  }
}

// out = the parts' sums, in order; one element a thread.
template <bool XF16>
__global__ __launch_bounds__(256) void few_join_kernel(FewArgs a) {
  const int64_t all = (int64_t)a.T * a.H;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    float v = 0.0f;
#pragma unroll 8
    for (int k = 0; k < a.parts; ++k) v += a.partial[k * all + i];
    ((uint16_t *)a.out)[i] = to_half_bits<XF16>(v);
  }
}

template <GroupElem EL, bool XF16>
hipError_t launch_shared(const FewArgs &a, hipStream_t st) {
  const int columns = a.T <= 16 || (int64_t)a.T * a.K <= 8 * (int64_t)a.E ? 16 : 32;
  using Stream = typename SharedDown<EL>::Stream;
  const int blocks = (a.H + kFewBlock - 1) / kFewBlock;
  const int lds = 2 * columns * Stream::ROW + 4 * ((FewIds::words(a.T * a.K) + 3) / 4 * 4) +
                  kWaves * a.T * kFewRows * 4;
  hipLaunchKernelGGL((few_shared_down_kernel<EL, XF16>), dim3((uint32_t)(blocks * a.parts)),
                     dim3(kThreads), lds, st, a, columns);
  const hipError_t down = hipGetLastError();
  if (down != hipSuccess || a.parts == 1) return down;
  const int64_t grid = std::min<int64_t>(((int64_t)a.T * a.H + 255) / 256, 8 * kNumCus);
  hipLaunchKernelGGL((few_join_kernel<XF16>), dim3((uint32_t)grid), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

// Both forms of the whole layer, in us (this one second).  64 experts of
// 2048 x 1024, top-8, 1 token 27 and 26, 2 tokens 46 and 40, 8 tokens 132 and
// 106; 8 experts of 4096 x 14336, top-2, 8 tokens 543 and 520; 8 of
// 1024 x 1024, top-2: 1 and 4 tokens 16 and 19 (the launch that joins the
// parts), 16 and 64 tokens 26 and 22, 37 and 28.  One token with 16-bit weights:
// the other form's workgroups need no join and, where 16 columns each do not
// cover H, are one on every CU; 256 experts of H x 2048, top-8, bf16: H 2048 47
// and 39, 4096 80 and 77, 5120 94 and 97, 7168 129 and 133 (fp16 134 and 144).
// The rule goes by H alone: longer rows and more than one round of that form's
// workgroups are for this one (8 of 5120 x 14336 160 and 156, 128 of
// 10240 x 2048 185 and 179).  With 8-bit weights H 2048 40 and 35, 4160 57 and
// 53, 7168 89 and 91, 10240 132 and 120.
int few_parts(bool i8, int32_t T, int32_t K, int32_t E, int32_t H, int32_t I) {
  const int64_t row = (int64_t)I * (i8 ? 1 : 2);
  // what the kernel assumes: whole wavefronts of columns, rows of 16 bytes
  if (H < kFewRows || row < 16) return 0;
  const int64_t experts = std::min<int64_t>((int64_t)T * K, E);
  const bool little = experts * H * row < (24 << 20) && (int64_t)T * K < 2 * (int64_t)E;
  if (little || (T == 1 && !i8 && H > 16 * kNumCus)) return 0;
  const int64_t blocks = (H + kFewBlock - 1) / kFewBlock;
  const int64_t chunk = SharedDown<kElemI8>::Stream::CHUNK * (i8 ? 1 : 2);
  const int64_t chunks = experts * ((row + chunk - 1) / chunk);
  // two workgroups a CU, parts of four chunks at least.  (With 32 columns a
  // segment the LDS of 60 tokens of two experts each, or 51 of eight, leaves
  // room for one a CU, and the grid runs as two rounds: 3.3 TB/s of weights at
  // 64 tokens of 8 experts of 4096 x 14336, 4.6 at 16 tokens of 256.)
  const int64_t want = (2 * kNumCus + blocks / 2) / blocks;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, chunks / 4), 32));
}

hipError_t launch_few_shared(bool f16, bool i8, const FewArgs &a, hipStream_t st) {
  if (i8) return f16 ? launch_shared<kElemI8, true>(a, st) : launch_shared<kElemI8, false>(a, st);
  return f16 ? launch_shared<kElemF16, true>(a, st) : launch_shared<kElemBf16, false>(a, st);
}

}  // namespace cco
