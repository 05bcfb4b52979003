// group_tile.h -- one tile of the products grouped by expert for rows of
// whole 16 bytes: the fast kernel's work, included by group.hip.
//
// Four wavefronts, one per SIMD, each with 128 x 128 of the output as 4 x 4
// blocks of 32x32x16 MFMAs whose sums sit in the 256 accumulation registers.
// A SIMD then reads 8 KiB of fragments from LDS per 16 MFMAs, which the
// MFMAs' time covers (two wavefronts per SIMD with half the block each would
// read 12 KiB).  Full tile 256 x 256; the last rows of a group, if at most
// 128, take a 128 x 512 tile, so that few rows do not cost a whole tile.
//
// Operands go global -> LDS by direct 16-byte loads into two rings of
// reduction steps of 64: two slots of A and three of B (the weights, or x in
// the weight gradient, come from HBM and run two steps ahead, A one); the
// wide tile has two of each.  Loads outside a matrix return zeros by the
// buffer's range check, which ends the reduction of any length:
//   k-contiguous operand  rows past the last and chunks past the end of the
//                         row (the offset's top bit is set there)
//   k-major operand       one descriptor per step, as long as the rows left
// Fragments of a k-major operand come from LDS by transposing reads.
//
// A step is four MFMA sub-steps on two fragment buffers in turn: while one
// is multiplied the other is read, and the loads of a later step are spread
// between the MFMAs.  One barrier per step, in the last sub-step: after it
// the step's slots are free and the next step's are complete.
#pragma once

#include "group_common.h"

namespace cco {
namespace {

// Where a tile sits: its operands' first elements, row distances in bytes
// and extents.
struct GroupTile {
  const char *a, *b;    // k-contiguous: first row of the tile; k-major: first k row, column 0
  uint32_t lda, ldb;    // bytes
  int32_t a_cols, b_cols;  // k-major: first column of the tile ..
  int32_t a_rows, b_rows;  // k-contiguous: rows of the tile that exist
  int32_t a_width, b_width;  // k-major: columns of the matrix
  int64_t kdim;         // reduction length
  char *c;              // the tile's first output element
  int64_t ldc;          // bytes
  int32_t c_rows, c_cols;  // rows and columns of the tile that exist
};

// One operand's direct loads: W rows (k-contiguous) or columns (k-major).
template <bool KC, int W>
struct TileLoads {
  static constexpr int BYTES = W * 128;            // one step
  static constexpr int N = BYTES / 1024 / kGemmWaves;  // loads per wavefront
  static constexpr int KM_LANES = KC ? 1 : (W / 8 < kWave ? W / 8 : kWave);  // lanes per k row
  const char *base;
  uint32_t ld, records, voff, kbyte, step_ld;
  int64_t kdim;

  __device__ __forceinline__ void init(const char *p, uint32_t ld_, int col0, int rows, int width,
                                       int64_t kdim_, int wave, int lane) {
    base = uniform(p);
    ld = uniform((int)ld_);
    kdim = kdim_;
    if constexpr (KC) {
      const int row = wave * 8 + lane / 8;
      // (the swizzle of row + 32 q is that of row)
      kbyte = ((lane % 8) ^ swz<8>(row)) * 16;
      voff = (uint32_t)row * ld + kbyte;
      records = (uint32_t)uniform((int)((uint32_t)(rows - 1) * ld + (uint32_t)(kdim * 2)));
      step_ld = 32 * ld;
    } else {
      constexpr int RPL = kWave / KM_LANES;  // k rows per load
      const int k = wave * RPL + lane / KM_LANES;
      // (the swizzle of k + 4 RPL q is that of k; with one k row per load the
      // rows wave + 4 q share it too)
      const int col = col0 + ((lane % KM_LANES) ^ kswz(k)) * 8;
      voff = col < width ? (uint32_t)k * ld + (uint32_t)col * 2 : 0x80000000u;
      step_ld = 4 * RPL * ld;
    }
    asm volatile("" : "+v"(voff));
  }

  // The descriptor and offsets of step kt (wavefront-uniform).
  struct Step {
    __amdgpu_buffer_rsrc_t r;
    uint32_t soff, v;
  };
  __device__ __forceinline__ Step step(int kt) const {
    Step s;
    if constexpr (KC) {
      // past the row's end the top bit puts the load out of range; the
      // scalar offset itself stays inside the range
      const uint32_t k2 = (uint32_t)(kdim * 2), at = (uint32_t)kt * 128u;
      s.r = byte_range_rsrc(base, records);
      s.soff = at < k2 ? at : 0u;
      s.v = kbyte + at < k2 ? voff : voff | 0x80000000u;
    } else {
      const int64_t k0 = (int64_t)kt * 64;
      int64_t left = kdim - k0;
      left = left < 0 ? 0 : (left > 64 ? 64 : left);
      s.r = byte_range_rsrc(base + k0 * ld, (uint32_t)left * ld);
      s.soff = 0;
      s.v = voff;
    }
    return s;
  }
  // load q of this wavefront's share, into the slot at `lds`
  __device__ __forceinline__ void issue(const Step &s, int q, char *lds, int wave) const {
    buffer_load_lds_16(s.r, s.v + (uint32_t)q * step_ld, s.soff, lds + (q * kGemmWaves + wave) * 1024);
  }
};

// This lane's fragment addresses in a slot of W rows or columns.  Blocks of
// 32 rows / columns: first, first + STRIDE, ...
template <bool KC, int W, int STRIDE>
struct TileFrags {
  static constexpr int PARTS = KC ? 1 : 2;  // LDS reads per fragment
  uint32_t addr[4];  // k-contiguous: per sub-step; k-major: per block

  __device__ __forceinline__ void init(uint32_t lds, int first, int lane) {
    if constexpr (KC) {
      const int l = lane & 31;
#pragma unroll
      for (int sk = 0; sk < 4; ++sk) {
        addr[sk] = lds + (uint32_t)((first * 32 + l) * 128 +
                                    (((sk * 2 + (lane >> 5)) ^ swz<8>(l)) * 16));
        asm volatile("" : "+v"(addr[sk]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        addr[i] = lds + kmajor_offset<W>(lane, (first + i * STRIDE) * 32);
        asm volatile("" : "+v"(addr[i]));
      }
    }
  }
  // part P of the fragment of block I, sub-step SK, slot at byte `slot`
  template <int I, int SK, int P>
  __device__ __forceinline__ void read(u32x4 &f, uint32_t slot) const {
    if constexpr (KC) {
      f = *(lds_cu32x4_t *)(uintptr_t)(addr[SK] + slot + I * STRIDE * 32 * 128);
    } else {
      const u32x2 v = lds_read_tr(addr[I] + slot + (SK * 16 + P * 4) * W * 2);
      if constexpr (P == 0) {
        f.x = v.x;
        f.y = v.y;
      } else {
        f.z = v.x;
        f.w = v.y;
      }
    }
  }
};

template <bool AKC, bool BKC, bool F16, bool OUT32, int BM, int BN, int RB>
__device__ __forceinline__ void run_group_tile(const GroupTile &t, char *smem, bool accumulate) {
  constexpr int WM = BM / 128, WN = kGemmWaves / WM, FM = 4, FN = 4;
  using LdA = TileLoads<AKC, BM>;
  using LdB = TileLoads<BKC, BN>;
  using FrA = TileFrags<AKC, BM, WM>;
  using FrB = TileFrags<BKC, BN, 1>;
  constexpr int LA = LdA::N, LB = LdB::N, LPS = LA + LB;
  constexpr int A_BYTES = LdA::BYTES, B_BYTES = LdB::BYTES, B_OFF = 2 * A_BYTES;
  static_assert(BM * WN == 128 * kGemmWaves && BN == WN * 128, "128 x 128 per wavefront");
  static_assert(B_OFF + RB * B_BYTES <= kGemmLdsBytes, "the rings must fit the LDS");
  static_assert(RB == 2 || RB == 3, "two or three slots of B");
  static_assert(LPS < 64, "vmcnt range");

  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = uniform(tid / kWave);
  const int wm = wave / WN, wn = wave % WN;
  LdA la;
  LdB lb;
  la.init(t.a, t.lda, t.a_cols, t.a_rows, t.a_width, t.kdim, wave, lane);
  lb.init(t.b, t.ldb, t.b_cols, t.b_rows, t.b_width, t.kdim, wave, lane);
  FrA ra;
  FrB rb;
  ra.init(lds_addr(smem), wm, lane);
  rb.init(lds_addr(smem) + B_OFF, wn * 4, lane);
  const int64_t steps = (t.kdim + 63) / 64;
  const int nk = uniform((int)(steps > 0 ? steps : 1));  // no rows: one step of zeros
  const int mblocks = (t.c_rows + 31) / 32;
  const int nact = uniform(min(FM, max(0, (mblocks - wm + WM - 1) / WM)));

  auto k_loop = [&](auto nact_c) __attribute__((always_inline)) {
    constexpr int NACT = decltype(nact_c)::value;
    constexpr int NF = NACT > 0 ? NACT : 1;
    f32x16 acc[NF][FN];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    // fragments of two sub-steps; read order: B's, then A's
    u32x4 fa[2][NF], fb[2][FN];
    constexpr int NRB = NACT > 0 ? FN * FrB::PARTS : 0;
    constexpr int NRD = NRB + NACT * FrA::PARTS;
    auto read = [&](auto buf_c, auto sk_c, auto r_c, uint32_t aslot, uint32_t bslot)
                    __attribute__((always_inline)) {
      constexpr int BUF = decltype(buf_c)::value, SK = decltype(sk_c)::value;
      constexpr int r = decltype(r_c)::value;
      if constexpr (r < NRB)
        rb.template read<r / FrB::PARTS, SK, r % FrB::PARTS>(fb[BUF][r / FrB::PARTS], bslot);
      else
        ra.template read<(r - NRB) / FrA::PARTS, SK, (r - NRB) % FrA::PARTS>(
            fa[BUF][(r - NRB) / FrA::PARTS], aslot);
    };
    // item q of a step's batch: A's loads of one step into slot aslot, then
    // B's of another into slot bslot
    auto load = [&](int q, const typename LdA::Step &sa, const typename LdB::Step &sb, char *aslot,
                    char *bslot) __attribute__((always_inline)) {
      if (q < LA)
        la.issue(sa, q, aslot, wave);
      else
        lb.issue(sb, q - LA, bslot, wave);
    };
    // One sub-step: multiply buffer BUFM, read the fragments of (RSK, the
    // slots) into the other one, issue loads [Q0, Q0 + NQ).  Items are
    // spread evenly over the MFMAs; with SYNC they start after the first row
    // and the barrier.  A row starts once its A fragment (and B's) are in:
    // LDS reads return in order.
    auto substep = [&](auto bufm_c, auto rsk_c, uint32_t raslot, uint32_t rbslot, auto q0_c,
                       auto nq_c, const typename LdA::Step &sa, const typename LdB::Step &sb,
                       char *laslot, char *lbslot, auto sync_c) __attribute__((always_inline)) {
      constexpr int BUFM = decltype(bufm_c)::value;
      constexpr int Q0 = decltype(q0_c)::value, NQ = decltype(nq_c)::value;
      constexpr bool SYNC = decltype(sync_c)::value;
      constexpr int NIT = NRD + NQ;
      constexpr int NM = SYNC ? (NACT > 0 ? (NACT - 1) * FN : 0) : NACT * FN;  // MFMAs with items
      constexpr int ND = NM > 0 ? NM : 1;
      auto items = [&](auto from_c, auto to_c) __attribute__((always_inline)) {
        constexpr int FROM = decltype(from_c)::value, TO = decltype(to_c)::value;
        static_for<TO - FROM>([&](auto d_c) __attribute__((always_inline)) {
          constexpr int m = FROM + decltype(d_c)::value;
          if constexpr (m < NRD)
            read(std::integral_constant<int, 1 - BUFM>{}, rsk_c, std::integral_constant<int, m>{},
                 raslot, rbslot);
          else
            load(Q0 + m - NRD, sa, sb, laslot, lbslot);
        });
      };
      auto sync = [&]() __attribute__((always_inline)) {
        wait_lgkmcnt<0>();
        wait_vmcnt<(RB == 3 ? LB : 0)>();
        stage_barrier();
      };
      static_for<NACT>([&](auto i_c) __attribute__((always_inline)) {
        constexpr int i = decltype(i_c)::value;
        constexpr int M0 = SYNC ? (i == 0 ? 0 : (i - 1) * FN) : i * FN;  // items' MFMAs before
        constexpr int DONE = M0 * NIT / ND;
        constexpr int ISSUED = DONE < NRD ? DONE : NRD;
        constexpr int LEFT = (NACT - 1 - i) * FrA::PARTS + ISSUED;
        wait_lgkmcnt<(LEFT < 15 ? LEFT : 15)>();
        static_for<FN>([&](auto j_c) __attribute__((always_inline)) {
          constexpr int j = decltype(j_c)::value;
          acc[i][j] = mfma_32x32x16<F16>(fb[BUFM][j], fa[BUFM][i], acc[i][j]);
          if constexpr (!(SYNC && i == 0)) {
            constexpr int m = M0 + j;
            items(std::integral_constant<int, m * NIT / ND>{},
                  std::integral_constant<int, (m + 1) * NIT / ND>{});
          }
        });
        if constexpr (SYNC && i == 0) sync();
      });
      if constexpr (SYNC && NACT == 0) sync();
      if constexpr (NM == 0)
        items(std::integral_constant<int, 0>{}, std::integral_constant<int, NIT>{});
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    using IT = std::true_type;
    using IF = std::false_type;
    constexpr int L3 = LPS / 4, L0 = LPS / 2, L1 = LPS - L3 - L0;
    char *const bring = smem + B_OFF;

    // steps 0 .. RB - 2 of B and step 0 of A in flight; step 0 complete; its
    // first fragments into buffer 0
    {
      const auto a0 = la.step(0);
      const auto b0 = lb.step(0);
#pragma unroll
      for (int q = 0; q < LA; ++q) la.issue(a0, q, smem, wave);
#pragma unroll
      for (int q = 0; q < LB; ++q) lb.issue(b0, q, bring, wave);
      if constexpr (RB == 3) {
        const auto b1 = lb.step(1);
#pragma unroll
        for (int q = 0; q < LB; ++q) lb.issue(b1, q, bring + B_BYTES, wave);
      }
      wait_vmcnt<(RB == 3 ? LB : 0)>();
      stage_barrier();
      static_for<NRD>([&](auto r_c) __attribute__((always_inline)) { read(I0{}, I0{}, r_c, 0u, 0u); });
    }
    // Step kt: A slot AS = kt % 2, B slot bs = kt % RB.  The batch issued
    // after its barrier: A of kt + 2 and B of kt + RB, into the same slots.
    auto step = [&](auto as_c, int kt, int bs) __attribute__((always_inline)) {
      constexpr uint32_t AS = decltype(as_c)::value;
      const int bs1 = bs == RB - 1 ? 0 : bs + 1;
      const int bsp = bs == 0 ? RB - 1 : bs - 1;  // slot of kt - 1
      const uint32_t ao = AS * A_BYTES, an = (1 - AS) * A_BYTES;
      const uint32_t bo = (uint32_t)bs * B_BYTES, bn = (uint32_t)bs1 * B_BYTES;
      // the rest of the batch of kt - 1
      const auto sa = la.step(kt + 1);
      const auto sb = lb.step(kt - 1 + RB);
      char *const pa = smem + an, *const pb = bring + bsp * B_BYTES;
      substep(I0{}, I1{}, ao, bo, std::integral_constant<int, L3>{},
              std::integral_constant<int, L0>{}, sa, sb, pa, pb, IF{});
      substep(I1{}, I2{}, ao, bo, std::integral_constant<int, L3 + L0>{},
              std::integral_constant<int, L1>{}, sa, sb, pa, pb, IF{});
      substep(I0{}, I3{}, ao, bo, I0{}, I0{}, sa, sb, pa, pb, IF{});
      // the barrier; the next step's first fragments; the first of the batch
      // of kt
      const auto na = la.step(kt + 2);
      const auto nb = lb.step(kt + RB);
      substep(I1{}, I0{}, an, bn, I0{}, std::integral_constant<int, L3>{}, na, nb, smem + ao,
              bring + bo, IT{});
    };
    {
      const auto sa = la.step(1);
      const auto sb = lb.step(RB - 1);
#pragma unroll
      for (int q = 0; q < L3; ++q) load(q, sa, sb, smem + A_BYTES, bring + (RB - 1) * B_BYTES);
    }
    int kt = 0, bs = 0;
    for (; kt + 2 <= nk; kt += 2) {
      step(I0{}, kt, bs);
      bs = bs == RB - 1 ? 0 : bs + 1;
      step(I1{}, kt + 1, bs);
      bs = bs == RB - 1 ? 0 : bs + 1;
    }
    if (kt < nk) step(I0{}, kt, bs);
    wait_lgkmcnt<0>();
    wait_vmcnt<0>();  // the loads past the last step land before the rings are reused
    __syncthreads();

    // Epilogue through the idle rings, so that rows leave in whole lines:
    // lane l holds row l % 32 of a block, columns 8 q + 4 (l / 32) + 0..3.
    // The empty asm keeps the accumulator reads of one block together.
    if constexpr (OUT32) {
      // 128 columns of fp32 at a time
      constexpr int OROWB = 128 * 4 + 16;
      static_assert(BM * OROWB <= kGemmLdsBytes, "half a tile must fit the LDS");
#pragma unroll
      for (int h = 0; h < WN; ++h) {
        if (wn == h)
          static_for<NACT>([&](auto i_c) __attribute__((always_inline)) {
            constexpr int i = decltype(i_c)::value;
            char *orow = smem + ((wm + i * WM) * 32 + (lane & 31)) * OROWB + (lane / 32) * 16;
            static_for<FN>([&](auto j_c) __attribute__((always_inline)) {
              constexpr int j = decltype(j_c)::value;
              asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *(float4 *)(orow + j * 128 + q * 32) =
                    make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                acc[i][j][4 * q + 3]);
            });
          });
        __syncthreads();
        const int cols = min(128, t.c_cols - h * 128);
        for (int idx = tid; idx < t.c_rows * 32; idx += kGemmWaves * kWave) {
          const int row = idx / 32, ch = idx % 32;
          if (ch * 4 < cols) {
            float4 v = *(const float4 *)(smem + row * OROWB + ch * 16);
            float4 *p = (float4 *)(t.c + row * t.ldc + (h * 128 + ch * 4) * 4);
            if (accumulate) {
              const float4 o = *p;
              v.x += o.x;
              v.y += o.y;
              v.z += o.z;
              v.w += o.w;
            }
            *p = v;
          }
        }
        __syncthreads();
      }
    } else {
      constexpr int OROWB = BN * 2 + 16;
      static_assert(BM * OROWB <= kGemmLdsBytes, "the output tile must fit the LDS");
      // accumulation adds to what is there before the one rounding, so the
      // sums meet the old values in registers
      static_for<NACT>([&](auto i_c) __attribute__((always_inline)) {
        constexpr int i = decltype(i_c)::value;
        const int row = (wm + i * WM) * 32 + (lane & 31);
        char *orow = smem + row * OROWB + (lane / 32) * 8;
        static_for<FN>([&](auto j_c) __attribute__((always_inline)) {
          constexpr int j = decltype(j_c)::value;
          asm volatile("" : "+a"(acc[i][j]));
          const int col = wn * 128 + j * 32;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = acc[i][j][4 * q + c];
            if (accumulate) {
              const int cc = col + q * 8 + (lane / 32) * 4;
              if (row < t.c_rows && cc < t.c_cols) {
                const u32x2 o = *(const u32x2 *)(t.c + row * t.ldc + cc * 2);
                v[0] += from_half_bits<F16>((uint16_t)o.x);
                v[1] += from_half_bits<F16>((uint16_t)(o.x >> 16));
                v[2] += from_half_bits<F16>((uint16_t)o.y);
                v[3] += from_half_bits<F16>((uint16_t)(o.y >> 16));
              }
            }
            u32x2 w;
            w.x = (uint32_t)to_half_bits<F16>(v[0]) | ((uint32_t)to_half_bits<F16>(v[1]) << 16);
            w.y = (uint32_t)to_half_bits<F16>(v[2]) | ((uint32_t)to_half_bits<F16>(v[3]) << 16);
            *(u32x2 *)(orow + (col + q * 8) * 2) = w;
          }
        });
      });
      __syncthreads();
      constexpr int CHUNKS = BN / 8;
      for (int idx = tid; idx < t.c_rows * CHUNKS; idx += kGemmWaves * kWave) {
        const int row = idx / CHUNKS, ch = idx % CHUNKS;
        if (ch * 8 < t.c_cols)
          *(u32x4 *)(t.c + row * t.ldc + ch * 16) = *(const u32x4 *)(smem + row * OROWB + ch * 16);
      }
      __syncthreads();
    }
  };
  // one specialisation per count of active row blocks (wavefront-uniform)
  static_for<FM + 1>([&](auto c) __attribute__((always_inline)) {
    if (nact == decltype(c)::value) k_loop(c);
  });
}

// ------------------------------------------------------- the tile lists --
// Rows of a group in the product and dx: q = rows / 256 full tiles of rows
// and a remainder, which is one more full tile or, if at most 128 rows, a
// wide tile (when there is more than one column tile).  Bands of 8 row
// tiles, column-major inside a band, so that the workgroups of one XCD,
// which take neighbouring tiles, share a few row panels and a few column
// panels in its L2.  In the last band the wide tile of a column pair stands
// before the full tiles of the same columns.
constexpr int kBand = 8;
struct RowTiles {
  int full, rem_half, ntl, nwide, bands;
};
__device__ __forceinline__ RowTiles row_tiles(int rows, int ncol) {
  RowTiles t;
  t.ntl = (ncol + 255) / 256;
  const int q = rows / 256, rem = rows % 256;
  const bool half = rem > 0 && rem <= 128 && t.ntl > 1;
  t.full = q + (rem > 0 && !half);
  t.rem_half = half ? rem : 0;
  t.nwide = half ? (t.ntl + 1) / 2 : 0;
  t.bands = max(1, (t.full + kBand - 1) / kBand);
  return t;
}
__device__ __forceinline__ int row_tile_units(const RowTiles &t) { return t.full * t.ntl + t.nwide; }

// Unit r: its first row, first column, and whether it is a wide tile.
__device__ __forceinline__ void row_tile_at(const RowTiles &t, int r, int &row0, int &col0,
                                            bool &wide) {
  const int band = min(r / (kBand * t.ntl), t.bands - 1);
  r -= band * kBand * t.ntl;
  const int qb = min(kBand, t.full - band * kBand);
  wide = false;
  int m, n;
  if (band == t.bands - 1 && t.rem_half) {
    const int per = 2 * qb + 1, j = r / per, rr = r - j * per;
    if (rr == 0) {
      wide = true;
      row0 = t.full * 256;
      col0 = j * 512;
      return;
    }
    n = 2 * j + (rr - 1) / qb;
    m = (rr - 1) % qb;
  } else {
    n = r / qb;
    m = r % qb;
  }
  row0 = (band * kBand + m) * 256;
  col0 = n * 256;
}

}  // namespace
}  // namespace cco
