// group_kernels.h -- matrix products over rows grouped by expert, with their
// gradients (include/cco_ops.h):
//
//   product  y[r]  = x[r] W_g^T             rows ragged, both operands k-contiguous
//   dx       dx[r] = dy[r] W_g              rows ragged, W_g k-major (k here: n)
//   dw       dW_g  = sum_r dy[r]^T x[r]     reduction ragged, both k-major
//
// Included by group_product.hip, group_dx.hip and group_dw.hip, one direction
// each (they compile side by side).
//
// Rows of whole 16 bytes take the fast kernel (group_tile.h: 256 x 256 tiles
// fed by direct loads into LDS).
//
// The general kernel, for all others: 128 x 128 tiles on four wavefronts, each 64 x 64 as
// 2 x 2 blocks of 32x32x16 MFMAs with fp32 sums; reduction steps of 64
// through two LDS buffers, the next step's operands in registers while the
// present one is multiplied.  Every global access is checked against its
// matrix, so any size, row distance and alignment is right.
#pragma once

#include "group_tile.h"

namespace cco {
namespace {

constexpr int kGenTile = 128, kGenThreads = 256, kGenStep = 64;
constexpr int kGenOperand = kGenTile * kGenStep * 2;  // bytes of one operand's step

// One operand of the tile: a matrix [nr][nc] (a group's part), and where the
// tile sits in it.  KC: rows row0.. are tile rows, columns are the
// reduction.  Otherwise rows are the reduction and columns col0.. the tile's.
// Rows may have any alignment: the loads are unaligned 16-byte ones, always
// inside the matrix and without a branch around them (the compiler would
// wait for a load where its branch ends): the row is clamped to the last
// one and the column to the row's last eight; `put`, which runs once the
// loads are in, moves down what a chunk at the row's end has, and puts zeros
// outside.  SHORT: rows of fewer than eight, element by element.
// 8-bit elements (I8; KC only) come sixteen to a chunk and 128 to a step.
template <bool KC, bool SHORT, bool I8>
struct GenOperand {
  static_assert(KC || !I8, "8-bit operands are k-contiguous");
  static constexpr int EB = I8 ? 1 : 2, CE = 16 / EB;  // bytes an element, elements a chunk
  static constexpr int STEP = kGenStep * 2 / EB;
  const char *base;
  int64_t ld, nr;
  int32_t nc;
  int64_t row0;
  int32_t col0;
  u32x4 stage[4];

  // row (in the step or tile) and first column of this thread's chunk q
  __device__ __forceinline__ int chunk_row(int q) const {
    return (q * kGenThreads + (int)threadIdx.x) / (KC ? 8 : 16);
  }
  __device__ __forceinline__ int chunk_col(int q, int64_t k0) const {
    const int c = (q * kGenThreads + (int)threadIdx.x) % (KC ? 8 : 16) * CE;
    return KC ? (int)k0 + c : col0 + c;
  }

  __device__ __forceinline__ void fetch(int64_t k0) {
    const int64_t first = KC ? row0 : k0;  // uniform: the rows' base
    const char *rows = base + first * ld * EB;
    const int last = (int)min((int64_t)(kGenTile - 1), nr - 1 - first);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t row = (uint32_t)min(chunk_row(q), last) * (uint32_t)ld;
      const int c = chunk_col(q, k0);
      if constexpr (SHORT && I8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            v |= (uint32_t)(uint8_t)rows[row + (uint32_t)min(c + 4 * i + b, nc - 1)] << (8 * b);
          stage[q][i] = v;
        }
      } else if constexpr (SHORT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint16_t lo, hi;
          __builtin_memcpy(&lo, rows + (row + (uint32_t)min(c + 2 * i, nc - 1)) * 2, 2);
          __builtin_memcpy(&hi, rows + (row + (uint32_t)min(c + 2 * i + 1, nc - 1)) * 2, 2);
          stage[q][i] = (uint32_t)lo | ((uint32_t)hi << 16);
        }
      } else {
        __builtin_memcpy(&stage[q], rows + (row + (uint32_t)min(c, nc - CE)) * EB, 16);
      }
    }
  }
  // The chunk as it belongs in LDS: elements past the row's end and rows past
  // the last are zeros.
  __device__ __forceinline__ u32x4 cut(u32x4 v, int64_t row, int c) const {
    uint64_t lo = v.x | ((uint64_t)v.y << 32), hi = v.z | ((uint64_t)v.w << 32);
    if constexpr (SHORT) {
      // keep the nc - c elements that exist
      const int keep = max(0, min(CE, nc - c)) * (8 * EB);
      lo = keep >= 64 ? lo : lo & ((1ull << keep) - 1);
      hi = keep >= 128 ? hi : (keep <= 64 ? 0 : hi & ((1ull << (keep - 64)) - 1));
    } else if (c + CE > nc) {
      // loaded from nc - CE: the first CE - nc % CE elements are before it
      const int sh = (CE - nc % CE) * (8 * EB);
      lo = sh >= 64 ? hi >> (sh - 64) : (lo >> sh) | (hi << (64 - sh));
      hi = sh >= 64 ? 0 : hi >> sh;
    }
    if (row >= nr || c >= nc) lo = hi = 0;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
  __device__ __forceinline__ void put(char *lds, int64_t k0) const {
    // only steps and tiles at the matrix' edges need cutting
    const bool edge = (KC ? row0 + kGenTile : k0 + STEP) > nr ||
                      (KC ? k0 + STEP : (int64_t)col0 + kGenTile) > nc || SHORT;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = q * kGenThreads + threadIdx.x;
      const u32x4 v = edge ? cut(stage[q], (KC ? row0 : k0) + chunk_row(q), chunk_col(q, k0))
                           : stage[q];
      const int at = KC ? (i / 8) * 128 + ((i % 8) ^ swz<8>(i / 8)) * 16
                        : (i / 16) * 256 + ((i % 16) ^ kswz(i / 16)) * 16;
      *(u32x4 *)(lds + at) = v;
    }
  }
  // fragment of the 32 tile rows / columns from `at`, sub-step sk
  __device__ __forceinline__ u32x4 frag(const char *lds, int at, int sk) const {
    const int lane = threadIdx.x % kWave;
    const uint32_t b = lds_addr(lds);
    if (KC) {
      const int row = at + (lane & 31), c = sk * 2 + (lane >> 5);
      return *(lds_cu32x4_t *)(uintptr_t)(b + row * 128 + ((c ^ swz<8>(row)) * 16));
    }
    const uint32_t p = b + kmajor_offset<kGenTile>(lane, at) + sk * 16 * 256;
    const u32x2 lo = lds_read_tr(p), hi = lds_read_tr(p + 4 * 256);
    return u32x4{lo.x, lo.y, hi.x, hi.y};
  }
};

// (EL, F16 and OUT32 as in run_group_tile)
template <int OP, GroupElem EL, bool F16, bool OUT32, bool SHORT>
__global__ __launch_bounds__(kGenThreads) void group_general_kernel(GroupArgs a) {
  constexpr bool I8 = EL == kElemI8;
  __shared__ __align__(16) char lds[2][2][kGenOperand];
  static_assert(sizeof(lds) == kGenTile * kGenTile * 4, "the LDS holds one tile's results");
  constexpr bool AKC = OP != kGroupDw, BKC = OP == kGroupProduct;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int wm = wave / 2, wn = wave % 2;
  // output columns, and (dw) output rows
  const int ncol = OP == kGroupProduct ? a.n : a.k;
  const int ct = (ncol + kGenTile - 1) / kGenTile;
  TileMap<kGenThreads> map;
  map.init(a, (int64_t *)&lds[0][0][0], [&](int rows) {
    return OP == kGroupDw ? ct * ((a.n + kGenTile - 1) / kGenTile)
                          : (rows + kGenTile - 1) / kGenTile * ct;
  });
  for (int64_t L = blockIdx.x; L < map.total; L += gridDim.x) {
    int g, r;
    map.find(L, (int32_t *)&lds[0][0][0], g, r);
    const GroupRows gr = group_rows(a, g);
    const int row0 = r / ct * kGenTile, col0 = r % ct * kGenTile;
    const int64_t welems = (int64_t)a.n * a.k;
    GenOperand<AKC, SHORT, I8> oa;
    GenOperand<BKC, SHORT, I8> ob;
    constexpr int EB = oa.EB, STEP = oa.STEP;
    int64_t kdim;       // reduction length
    int32_t out_rows;   // rows of this group's output
    oa.base = a.a + gr.lo * a.lda * EB;
    oa.ld = a.lda;
    oa.nr = gr.n;
    oa.nc = OP == kGroupProduct ? a.k : a.n;
    oa.row0 = oa.col0 = row0;
    if (OP == kGroupDw) {
      kdim = gr.n;
      out_rows = a.n;
      ob.base = a.b + gr.lo * a.ldb * 2;
      ob.nr = gr.n;
    } else {
      kdim = oa.nc;
      out_rows = gr.n;
      ob.base = a.b + (int64_t)g * welems * EB;
      ob.nr = a.n;
    }
    ob.ld = a.ldb;
    ob.nc = a.k;
    ob.row0 = ob.col0 = col0;
    typename GroupAcc<EL>::type acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
    const int64_t steps = (kdim + STEP - 1) / STEP;
    if (steps > 0) {
      oa.fetch(0);
      ob.fetch(0);
      oa.put(lds[0][0], 0);
      ob.put(lds[0][1], 0);
    }
    __syncthreads();
    for (int64_t s = 0; s < steps; ++s) {
      const int cur = (int)(s & 1);
      if (s + 1 < steps) {
        oa.fetch((s + 1) * STEP);
        ob.fetch((s + 1) * STEP);
      }
#pragma unroll
      for (int sk = 0; sk < 4; ++sk) {
        u32x4 fa[2], fb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          fa[i] = oa.frag(lds[cur][0], wm * 64 + i * 32, sk);
          fb[i] = ob.frag(lds[cur][1], wn * 64 + i * 32, sk);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = group_mfma<EL>(fb[j], fa[i], acc[i][j]);
      }
      // the other buffer was last read in step s - 1, before its barrier
      if (s + 1 < steps) {
        oa.put(lds[cur ^ 1][0], (s + 1) * STEP);
        ob.put(lds[cur ^ 1][1], (s + 1) * STEP);
      }
      __syncthreads();
    }
    char *cbase = a.c + (OP == kGroupDw ? (int64_t)g * welems : gr.lo * a.ldc) * (OUT32 ? 4 : 2);
    const int64_t ldc = OP == kGroupDw ? a.k : a.ldc;
    // Results through the (idle) LDS, so that a wavefront stores two
    // neighbouring elements a lane along a row, whatever its alignment:
    // stored from the accumulators' order, 2 bytes a lane over 32 rows, a
    // weight gradient of few steps spent most of its time here.  Chunk c of
    // 16 bytes of row r lies at c ^ (r % 32).
    char *tile = &lds[0][0][0];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = wm * 64 + i * 32 + (lane & 31);
          const int c = wn * 16 + j * 8 + q * 2 + (lane >> 5);
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][j][4 * q + e];
          *(f32x4 *)(tile + row * 512 + ((c ^ (row & 31)) * 16)) = v;
        }
    __syncthreads();
    const int col = col0 + 2 * lane;
    const int rows_here = (int)min((int64_t)kGenTile, (int64_t)out_rows - row0);
    float cs[2] = {1.0f, 1.0f};
    if constexpr (I8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) cs[i] = a.cs[(int64_t)g * a.n + min(col + i, ncol - 1)];
    }
    for (int row = wave; row < rows_here; row += kGenThreads / kWave) {
      const char *at = tile + row * 512 + (((lane >> 1) ^ (row & 31)) * 16) + (lane & 1) * 8;
      float v[2] = {((const float *)at)[0], ((const float *)at)[1]};
      if constexpr (I8) {
        const float rs = a.rs[(gr.lo + row0 + row) * a.ldrs];
        v[0] = scaled_sum(v[0], rs, cs[0]);
        v[1] = scaled_sum(v[1], rs, cs[1]);
      }
      char *out = cbase + ((int64_t)(row0 + row) * ldc + col) * (OUT32 ? 4 : 2);
      const int n = min(2, ncol - col);  // elements of this lane that exist
      if (n <= 0) continue;
      using E = std::conditional_t<OUT32, float, uint16_t>;
      E e[2] = {0, 0};
      if (a.accumulate) {
        if (n == 2)
          __builtin_memcpy(e, out, sizeof(e));
        else
          __builtin_memcpy(e, out, sizeof(E));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (OUT32)
          e[i] = a.accumulate ? v[i] + e[i] : v[i];
        else
          e[i] = to_half_bits<F16>(a.accumulate ? v[i] + from_half_bits<F16>(e[i]) : v[i]);
      }
      if (n == 2)
        __builtin_memcpy(out, e, sizeof(e));
      else
        __builtin_memcpy(out, e, sizeof(E));
    }
    __syncthreads();  // the tile is read out before the next one's operands come
  }
}

// The fast kernel: tiles of this XCD's contiguous part of the list
// (workgroup id mod 8 is the XCD), every (gridDim / 8)-th of them.  A tile's
// first loads are issued before the previous tile's results are stored.
// ACC (dw): results are added to what is there.  TILE: 256, or 128 with two
// workgroups on a CU.
template <int OP, int TILE>
using FullTile = TileShape<OP != kGroupDw, OP == kGroupProduct, TILE, TILE, 3, TILE / 64>;
template <int OP>
using WideTile = TileShape<OP != kGroupDw, OP == kGroupProduct, 128, 512, 2, 4>;

// SPLIT: the reduction in a.parts parts, neighbouring units of a tile, whose
// fp32 sums go to the workspace (then OUT32).
template <int OP, GroupElem EL, bool F16, bool OUT32, bool ACC, int TILE, bool SPLIT>
__global__ __launch_bounds__(kGemmWaves *kWave, TILE == 128 ? 2 : 1) void group_tile_kernel(
    GroupArgs a) {
  constexpr int ES = OUT32 ? 4 : 2;
  using Full = FullTile<OP, TILE>;
  using Wide = WideTile<OP>;
  constexpr bool WIDE = OP != kGroupDw && TILE == 256;
  static_assert(!SPLIT || (OUT32 && !ACC && TILE == 128), "parts are fp32 tiles of 128");
  extern __shared__ __align__(1024) char smem[];
  // sums in accumulation registers: that form of the MFMAs draws less power
  asm volatile("" ::: "a0");
  const int ncol = OP == kGroupProduct ? a.n : a.k;
  const int64_t welems = (int64_t)a.n * a.k;
  const int mt = (a.n + TILE - 1) / TILE, nt = (ncol + TILE - 1) / TILE;  // dw: tiles of a group
  TileMap<kGemmWaves * kWave> map;
  if constexpr (OP == kGroupDw)
    map.total = (int64_t)a.groups * mt * nt;
  else
    map.init(a, (int64_t *)smem,
             [&](int rows) { return row_tile_units(row_tiles<TILE>(rows, ncol)); });

  GroupTile t;
  bool wide = false;
  auto tile_at = [&](int64_t unit) __attribute__((always_inline)) {
    int g, r;
    const int64_t L = SPLIT ? unit / a.parts : unit;
    const int part = SPLIT ? (int)(unit - L * a.parts) : 0;
    if constexpr (OP == kGroupDw) {
      g = (int)(L / (mt * nt));
      r = (int)(L - (int64_t)g * (mt * nt));
    } else {
      map.find(L, (int32_t *)smem, g, r);
    }
    const GroupRows gr = group_rows(a, g);
    const int rows = uniform(gr.n);
    const int64_t lo = gr.lo;
    t.rot = 0;
    t.lda = (uint32_t)(a.lda * 2);
    t.ldb = (uint32_t)(a.ldb * 2);
    if constexpr (OP == kGroupDw) {
      // bands of four column tiles, row-major inside: the workgroups of an
      // XCD share about eight panels of dy and four of x
      const int band = r / (mt * 4), bw = min(4, nt - band * 4);
      const int rr = r - band * mt * 4;
      const int row0 = rr / bw * TILE, col0 = (band * 4 + rr % bw) * TILE;
      t.a = a.a + lo * a.lda * 2;
      t.b = a.b + lo * a.ldb * 2;
      t.a_cols = row0;
      t.b_cols = col0;
      t.a_width = a.n;
      t.b_width = a.k;
      t.a_rows = t.b_rows = 0;
      t.kdim = rows;
      t.ldc = (int64_t)a.k * ES;
      t.c = SPLIT ? (char *)(a.ws + (int64_t)part * a.groups * welems) : a.c;
      t.c += (g * welems + (int64_t)row0 * a.k + col0) * ES;
      t.c_rows = min(TILE, a.n - row0);
      t.c_cols = min(TILE, a.k - col0);
    } else {
      int row0, col0;
      row_tile_at<TILE>(row_tiles<TILE>(rows, ncol), r, row0, col0, wide);
      row0 = uniform(row0);
      col0 = uniform(col0);
      t.a = a.a + (lo + row0) * a.lda * 2;
      t.a_rows = min(TILE, rows - row0);
      t.kdim = OP == kGroupProduct ? a.k : a.n;
      t.a_cols = t.a_width = 0;
      if (OP == kGroupProduct && !SPLIT && a.k % 2048 == 0 && a.rows <= 256 * (int64_t)a.groups)
        t.rot = uniform((col0 / TILE + 3 * g) % (a.k / 64));
      t.b = a.b + g * welems * 2;
      if (OP == kGroupProduct) t.b += (int64_t)col0 * a.ldb * 2;
      t.b_rows = min(wide ? 512 : TILE, ncol - col0);
      t.b_cols = col0;
      t.b_width = a.k;
      const int64_t ldc = SPLIT ? ncol : a.ldc;
      t.ldc = ldc * ES;
      t.c = SPLIT ? (char *)(a.ws + (int64_t)part * a.rows * ncol) : a.c;
      t.c += ((lo + row0) * ldc + col0) * ES;
      t.c_rows = t.a_rows;
      t.c_cols = t.b_rows;
      if constexpr (EL == kElemI8) {
        t.rs = a.rs + (lo + row0) * a.ldrs;
        t.ldrs = a.ldrs;
        t.cs = a.cs + (int64_t)g * a.n + col0;
      }
    }
    if constexpr (SPLIT) {
      // this part's steps (none: it leaves zeros)
      const int64_t steps = (t.kdim + 63) / 64;
      const int64_t kb = steps * part / a.parts, ke = steps * (part + 1) / a.parts;
      t.a += OP == kGroupDw ? kb * 64 * t.lda : kb * 128;
      t.b += OP == kGroupProduct ? kb * 128 : kb * 64 * t.ldb;
      t.kdim = min(t.kdim - kb * 64, (ke - kb) * 64);
    }
    if constexpr (WIDE)
      if (wide) {
        Wide::start(t, smem);
        return;
      }
    Full::start(t, smem);
  };

  const int xcd = blockIdx.x % kNumXcd;
  const int64_t units = SPLIT ? map.total * a.parts : map.total;
  const int64_t end = units * (xcd + 1) / kNumXcd;
  const int64_t stride = gridDim.x / kNumXcd;
  int64_t L = units * xcd / kNumXcd + blockIdx.x / kNumXcd;
  if (L >= end) return;
  tile_at(L);
  bool stored = false;
  for (; L < end; L += stride) {
    const GroupTile now = t;
    auto next = [&]() __attribute__((always_inline)) {
      if (L + stride < end) tile_at(L + stride);
    };
    if constexpr (WIDE)
      if (wide) {
        stored = run_group_tile<Wide, EL, F16, OUT32, ACC, SPLIT>(now, smem, stored, next);
        continue;
      }
    stored = run_group_tile<Full, EL, F16, OUT32, ACC, SPLIT>(now, smem, stored, next);
  }
}

// Split reductions: products of at most kPartTiles tiles of 128 and at least
// kSplitSteps steps of 64, into parts of at least kPartSteps.  Unsplit and
// split: 64 tiles of 16 steps 12.4 and 16 us, 16 tiles of 22 steps 10 and 13,
// 12 tiles of 32 steps 17 and 15, 32 tiles of 64 steps 37 and 15, 128 tiles
// of 64 steps 39 and 32, 9 tiles of 209 steps 109 and 22, 4 tiles of 1024
// steps 556 and 49.
constexpr int kPartTiles = 128, kSplitSteps = 32, kPartSteps = 8, kMaxParts = 16;

// Largest grid: enough workgroups that the hardware's own hand-out levels
// uneven tiles; the kernels take further tiles in a loop.
constexpr int64_t kMaxGrid = 4096;

// Upper bound of the tiles of a call.  Rows of a group: at most one partly
// filled row of tiles for every group with rows.
template <int OP, int TILE>
int64_t tile_bound(const GroupArgs &a) {
  const int64_t ncol = OP == kGroupProduct ? a.n : a.k, ct = (ncol + TILE - 1) / TILE;
  return OP == kGroupDw ? (int64_t)a.groups * ct * ((a.n + TILE - 1) / TILE)
                        : (a.rows / TILE + std::min<int64_t>(a.groups, a.rows)) * ct;
}

// Tiles of TILE as if the rows were spread evenly over the groups.
int64_t even_tiles(GroupOp op, int tile, int64_t groups, int64_t rows, int64_t n, int64_t k) {
  const int64_t ct = ((op == kGroupProduct ? n : k) + tile - 1) / tile;
  if (op == kGroupDw) return groups * ct * ((n + tile - 1) / tile);
  const int64_t g = std::max<int64_t>(1, std::min(groups, rows));
  const int64_t avg = (rows + g - 1) / g, rem = avg % tile;
  const bool half = tile == 256 && rem <= 128;
  return g * (avg / tile * ct + (rem == 0 ? 0 : (half ? (ct + 1) / 2 : ct)));
}

// Tiles of 128 where those of 256 would leave a third of the CUs idle: 128
// tiles of 256 ran 93 us and as tiles of 128 68 us (1 group, 4096 x 2048 x
// 4096, dw), 116 of them 78 and 54 us, but 196 of them 51 and 58 us, and 256
// of them 113 and 141 us (8 groups, 4096 x 4096 x 4096, product).
template <int OP>
bool small_tiles(const GroupArgs &a) {
  return 3 * even_tiles((GroupOp)OP, 256, a.groups, a.rows, a.n, a.k) < 2 * kNumCus;
}

// The 8-bit product besides: tiles of 128 where those of 256 end in a round
// that few CUs take part in.  A group of uneven rows ends anywhere in a row of
// tiles and has on average half of one more than its rows fill; with tiles of
// 256 a quarter, since up to 128 rows take half as many tiles, wide ones.  A
// round of 128 x 128 tiles, two a CU, takes 0.575 of one of 256 x 256.  (256
// and 128, in us: 8 groups, 4096 rows, 4096 x 4096 100 and 85; 32 groups, 8192
// rows, 2048 x 2048 60 and 53; but 8 groups, 8192 rows, 4096 x 14336 538 and
// 553, 1 group of 8192 rows, 4096 x 7168 195 and 230, 256 groups, 65536 rows,
// 7168 x 2048 1221 and 1468.)  Not for groups of up to 128 rows, whose wide
// tiles are as small: 8 groups, 1000 rows, 14336 x 4096 104 and 110.
inline bool short_last_round(const GroupArgs &a) {
  const int64_t live = std::min<int64_t>(a.groups, a.rows);
  if (a.rows <= 128 * live) return false;
  auto rounds = [&](int tile) {
    const int64_t ct = (a.n + tile - 1) / tile;
    const int64_t more = live > 1 ? live * ct / (tile == 256 ? 4 : 2) : 0;
    const int64_t at_once = tile == 256 ? kNumCus : 2 * kNumCus;
    return (even_tiles(kGroupProduct, tile, a.groups, a.rows, a.n, a.k) + more + at_once - 1) /
           at_once;
  };
  // (0.93: the smaller tiles read more and have to win clearly)
  return 575 * rounds(128) < 930 * rounds(256);
}

template <int OP, GroupElem EL, bool F16, bool OUT32>
hipError_t launch_general(const GroupArgs &a, hipStream_t st) {
  const int64_t tiles = tile_bound<OP, kGenTile>(a);
  if (tiles == 0) return hipSuccess;
  const dim3 grid((uint32_t)std::min(tiles, kMaxGrid)), block(kGenThreads);
  if (EL == kElemI8 ? a.k < 16 : a.n < 8 || a.k < 8)
    hipLaunchKernelGGL((group_general_kernel<OP, EL, F16, OUT32, true>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((group_general_kernel<OP, EL, F16, OUT32, false>), grid, block, 0, st, a);
  return hipGetLastError();
}

template <int OP, GroupElem EL, bool F16, bool OUT32, int TILE>
hipError_t launch_tiles(const GroupArgs &a, hipStream_t st) {
  const int64_t tiles = tile_bound<OP, TILE>(a);
  if (tiles == 0) return hipSuccess;
  // whole XCDs
  const int64_t grid = std::min((tiles + kNumXcd - 1) / kNumXcd * kNumXcd, kMaxGrid);
  const dim3 g((uint32_t)grid), b(kGemmWaves * kWave);
  constexpr int lds = FullTile<OP, TILE>::LDS_BYTES;
  if (OP == kGroupDw && a.accumulate)
    hipLaunchKernelGGL((group_tile_kernel<OP, EL, F16, OUT32, OP == kGroupDw, TILE, false>), g, b,
                       lds, st, a);
  else
    hipLaunchKernelGGL((group_tile_kernel<OP, EL, F16, OUT32, false, TILE, false>), g, b, lds, st,
                       a);
  return hipGetLastError();
}

// C = the parts' sums, in order (dw: added to what is there).  Block y is a
// group; its elements of a part are contiguous, rows of C columns.
template <int OP, GroupElem EL, bool F16, bool OUT32>
__global__ __launch_bounds__(256) void group_parts_kernel(GroupArgs a) {
  const int g = blockIdx.y;
  const int64_t cols = OP == kGroupProduct ? a.n : a.k;
  int64_t lo = (int64_t)g * a.n, n = a.n, part = (int64_t)a.groups * a.n * cols;
  if (OP != kGroupDw) {
    const GroupRows gr = group_rows(a, g);
    lo = gr.lo;
    n = gr.n;
    part = (int64_t)a.rows * cols;
  }
  const float *ws = a.ws + lo * cols;
  // four elements a thread (columns are a multiple of 8)
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n * cols;
       i += (int64_t)gridDim.x * 1024) {
    using Sum = std::conditional_t<EL == kElemI8, i32x4, f32x4>;
    Sum sum = *(const Sum *)(ws + i);
    for (int p = 1; p < a.parts; ++p) sum += *(const Sum *)(ws + p * part + i);
    const int64_t row = lo + i / cols, col = i % cols;
    f32x4 s;
    if constexpr (EL == kElemI8) {
      const float rs = a.rs[row * a.ldrs];
      const f32x4 cs = *(const f32x4 *)(a.cs + (int64_t)g * cols + col);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = scaled_sum((float)sum[e], rs, cs[e]);
    } else {
      s = sum;
    }
    char *c = a.c + (row * (OP == kGroupDw ? cols : a.ldc) + col) * (OUT32 ? 4 : 2);
    if constexpr (OUT32) {
      if (a.accumulate) s += *(const f32x4 *)c;
      *(f32x4 *)c = s;
    } else {
      u32x2 d;
      if (a.accumulate) {
        d = *(const u32x2 *)c;
        const uint32_t d0 = d.x, d1 = d.y;
        s[0] += from_half_bits<F16>((uint16_t)d0);
        s[1] += from_half_bits<F16>((uint16_t)(d0 >> 16));
        s[2] += from_half_bits<F16>((uint16_t)d1);
        s[3] += from_half_bits<F16>((uint16_t)(d1 >> 16));
      }
      d.x = pack_half<F16>(s[0], s[1]);
      d.y = pack_half<F16>(s[2], s[3]);
      *(u32x2 *)c = d;
    }
  }
}

template <int OP, GroupElem EL, bool F16, bool OUT32>
hipError_t launch_split(const GroupArgs &a, hipStream_t st) {
  const int64_t tiles = tile_bound<OP, 128>(a);
  if (tiles == 0) return hipSuccess;
  const int64_t units = tiles * a.parts;
  const int64_t grid = std::min((units + kNumXcd - 1) / kNumXcd * kNumXcd, kMaxGrid);
  hipLaunchKernelGGL((group_tile_kernel<OP, EL, F16, true, false, 128, true>), dim3((uint32_t)grid),
                     dim3(kGemmWaves * kWave), (FullTile<OP, 128>::LDS_BYTES), st, a);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int64_t cols = OP == kGroupProduct ? a.n : a.k;
  const int64_t elems = OP == kGroupDw ? a.n * cols : (a.rows + a.groups - 1) / a.groups * cols;
  const int64_t gx = std::min<int64_t>(std::max<int64_t>(1, (elems + 1023) / 1024), 1024);
  hipLaunchKernelGGL((group_parts_kernel<OP, EL, F16, OUT32>), dim3((uint32_t)gx, a.groups), dim3(256),
                     0, st, a);
  return hipGetLastError();
}

template <int OP, GroupElem EL, bool F16, bool OUT32>
hipError_t launch_either(bool aligned, const GroupArgs &a, hipStream_t st) {
  if (!aligned) return launch_general<OP, EL, F16, OUT32>(a, st);
  if (a.parts > 1) return launch_split<OP, EL, F16, OUT32>(a, st);
  return small_tiles<OP>(a) || (EL == kElemI8 && short_last_round(a))
             ? launch_tiles<OP, EL, F16, OUT32, 128>(a, st)
             : launch_tiles<OP, EL, F16, OUT32, 256>(a, st);
}

template <int OP>
hipError_t launch_op(bool f16, bool out_f32, bool aligned, const GroupArgs &a, hipStream_t st) {
  if constexpr (OP == kGroupDw)
    if (out_f32)
      return f16 ? launch_either<OP, kElemF16, true, true>(aligned, a, st)
                 : launch_either<OP, kElemBf16, false, true>(aligned, a, st);
  return f16 ? launch_either<OP, kElemF16, true, false>(aligned, a, st)
             : launch_either<OP, kElemBf16, false, false>(aligned, a, st);
}

}  // namespace
}  // namespace cco
