// group_tile.h -- one tile of the products grouped by expert for rows of
// whole 16 bytes: the fast kernel's work, included by group_kernels.h.
//
// Four wavefronts, one per SIMD, each with 128 x 128 of the output as 4 x 4
// blocks of 32x32x16 MFMAs whose sums sit in the 256 accumulation registers.
// A SIMD then reads 8 KiB of fragments from LDS per 16 MFMAs, which the
// MFMAs' time covers (two wavefronts per SIMD with half the block each would
// read 12 KiB).  Full tile 256 x 256; the last rows of a group, if at most
// 128, take a 128 x 512 tile, so that few rows do not cost a whole tile.
// Where 256 x 256 tiles would be few, or end after a few reduction steps,
// tiles of 128 x 128 (2 x 2 blocks a wavefront) with two workgroups on a CU:
// four times the tiles, and one workgroup's stores and first loads run while
// the other multiplies.
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
// Measured: 8 groups of 1024 rows by 14336 x 4096, product and dx 1.22
// PFLOP/s, one group of 65536 rows by 4096 x 4096, dw 1.28 (bound by the
// matrix cores' clock under load and the operands' way through LDS, no bank
// conflicts); 256 groups of 8 rows by 7168 x 2048, product 5.9 TB/s of
// weights.  A tile's results and first loads cost about 17000 cycles, a step
// about 3400, so reductions of few steps stay below (16 steps: 1.08 PFLOP/s,
// with fp32 results 0.85 to 0.94: loads and stores complete in one order, A's
// step 1 is loaded behind the last tile's stores, and so the second step
// waits for them).
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
  int32_t rot;          // k-contiguous operands: the step the reduction begins with
  char *c;              // the tile's first output element
  int64_t ldc;          // bytes
  int32_t c_rows, c_cols;  // rows and columns of the tile that exist
};

// One operand's direct loads: W rows (k-contiguous) or columns (k-major).
// ROT (both operands k-contiguous): the steps run from `rot` on and around.
// Where rows are a multiple of 4 KiB apart, a step of every tile touches the
// same few memory channels if all begin at 0; begun at steps of their own,
// 64 groups of 8 rows by 2048 x 2048 took 97 us instead of 131, and a
// decoding step's 256 groups by 7168 x 2048 5 % less.  Other distances gain
// nothing and keep rot 0.
template <bool KC, int W, bool ROT>
struct TileLoads {
  static constexpr int BYTES = W * 128;            // one step
  static constexpr int N = BYTES / 1024 / kGemmWaves;  // loads per wavefront
  static constexpr int KM_LANES = KC ? 1 : (W / 8 < kWave ? W / 8 : kWave);  // lanes per k row
  const char *base;
  uint32_t ld, records, voff, kbyte, step_ld;
  int32_t rot, nk;
  int64_t kdim;

  __device__ __forceinline__ void init(const char *p, uint32_t ld_, int col0, int rows, int width,
                                       int64_t kdim_, int rot_, int wave, int lane) {
    rot = rot_;
    nk = (int)((kdim_ + 63) / 64);
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
    if constexpr (ROT)
      if (kt < nk) kt = kt + rot < nk ? kt + rot : kt + rot - nk;
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
    buffer_load_lds_16(s.r, s.v + (uint32_t)q * step_ld, s.soff,
                       lds + (q * kGemmWaves + wave) * 1024);
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

// A tile shape with its rings, and the loads a tile starts with: step 0 of
// both operands, and step 1 of B where it has three slots.
// RB slots of B; each wavefront has FB x FB blocks of 32 x 32.
template <bool AKC_, bool BKC_, int BM_, int BN_, int RB_, int FB_>
struct TileShape {
  static constexpr bool AKC = AKC_, BKC = BKC_;
  static constexpr int BM = BM_, BN = BN_, RB = RB_, FB = FB_;
  static constexpr int WM = BM / (32 * FB), WN = kGemmWaves / WM;
  using LdA = TileLoads<AKC, BM, AKC && BKC>;
  using LdB = TileLoads<BKC, BN, AKC && BKC>;
  static constexpr int LA = LdA::N, LB = LdB::N;
  static constexpr int A_BYTES = LdA::BYTES, B_BYTES = LdB::BYTES, B_OFF = 2 * A_BYTES;
  static constexpr int LDS_BYTES = B_OFF + RB * B_BYTES;
  // Where results are staged: 32 rows of FB * 64 bytes for every wavefront,
  // at the rings' end, which the first loads of no shape of its kernel fill.
  static constexpr int STAGE_ROW = FB * 64, STAGE_BYTES = 32 * STAGE_ROW;
  static constexpr int STAGE_OFF = LDS_BYTES - kGemmWaves * STAGE_BYTES;
  static_assert(BN == WN * 32 * FB && WM * WN == kGemmWaves, "the wavefronts' blocks");
  static_assert(LDS_BYTES <= kGemmLdsBytes, "the rings must fit the LDS");
  static_assert(RB == 2 || RB == 3, "two or three slots of B");
  static_assert(LA + LB < 64, "vmcnt range");
  static_assert(B_OFF + (RB - 1) * B_BYTES <= STAGE_OFF, "the first loads leave the staging area");

  __device__ static __forceinline__ void init(const GroupTile &t, LdA &la, LdB &lb, int wave,
                                              int lane) {
    la.init(t.a, t.lda, t.a_cols, t.a_rows, t.a_width, t.kdim, t.rot, wave, lane);
    lb.init(t.b, t.ldb, t.b_cols, t.b_rows, t.b_width, t.kdim, t.rot, wave, lane);
  }
  __device__ static __forceinline__ void start(const GroupTile &t, char *smem) {
    const int lane = threadIdx.x & (kWave - 1), wave = uniform((int)threadIdx.x / kWave);
    LdA la;
    LdB lb;
    init(t, la, lb, wave, lane);
    const auto a0 = la.step(0);
    const auto b0 = lb.step(0);
#pragma unroll
    for (int q = 0; q < LA; ++q) la.issue(a0, q, smem, wave);
#pragma unroll
    for (int q = 0; q < LB; ++q) lb.issue(b0, q, smem + B_OFF, wave);
    if constexpr (RB == 3) {
      const auto b1 = lb.step(1);
#pragma unroll
      for (int q = 0; q < LB; ++q) lb.issue(b1, q, smem + B_OFF + B_BYTES, wave);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
};

// Lanes 32..63 of a trade places with lanes 0..31 of b.
__device__ __forceinline__ void swap_halves(uint32_t &a, uint32_t &b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// Stores one wavefront makes of a tile whose row blocks all exist.
template <class Shape, bool OUT32>
constexpr int kTileStores = Shape::FB * Shape::FB * (OUT32 ? 4 : 2);

// The tile whose first loads `start` has issued.  stored_before: the
// previous tile of this workgroup left all its kTileStores behind those
// loads (false: any number).  next(): called once the operands are used up
// and the rings are idle; it issues the next tile's first loads, which then
// run while this tile's results are stored.
template <class Shape, bool F16, bool OUT32, bool ACC, class Next>
__device__ __forceinline__ bool run_group_tile(const GroupTile &t, char *smem, bool stored_before,
                                               Next &&next) {
  constexpr int WM = Shape::WM, WN = Shape::WN, FM = Shape::FB, FN = Shape::FB;
  constexpr int RB = Shape::RB;
  using LdA = typename Shape::LdA;
  using LdB = typename Shape::LdB;
  using FrA = TileFrags<Shape::AKC, Shape::BM, WM>;
  using FrB = TileFrags<Shape::BKC, Shape::BN, 1>;
  constexpr int LA = Shape::LA, LB = Shape::LB, LPS = LA + LB;
  constexpr int A_BYTES = Shape::A_BYTES, B_BYTES = Shape::B_BYTES, B_OFF = Shape::B_OFF;

  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = uniform(tid / kWave);
  const int wm = wave / WN, wn = wave % WN;
  LdA la;
  LdB lb;
  Shape::init(t, la, lb, wave, lane);
  FrA ra;
  FrB rb;
  ra.init(lds_addr(smem), wm, lane);
  rb.init(lds_addr(smem) + B_OFF, wn * FN, lane);
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

    // step 0 complete everywhere; its first fragments into buffer 0.  Behind
    // its loads are those of B's step 1 and the last tile's stores; both
    // counts are issue counts, and the operations complete in order.
    constexpr int BEHIND = RB == 3 ? LB : 0;
    constexpr int STORED = BEHIND + kTileStores<Shape, OUT32>;
    if (stored_before)
      wait_vmcnt<(STORED < 63 ? STORED : 63)>();
    else
      wait_vmcnt<BEHIND>();
    stage_barrier();
    static_for<NRD>([&](auto r_c) __attribute__((always_inline)) {
      read(I0{}, I0{}, r_c, 0u, 0u);
    });
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
    stage_barrier();
    next();

    // Results, 32 rows of STAGE_ROW bytes at a time, through a piece of LDS
    // of this wavefront's own (past every slot the next tile's first loads
    // fill), so that a store covers whole lines of a row.  Lane l holds row
    // l % 32 of a block and columns 8 q + 4 (l / 32) + 0..3.  Chunk c of
    // staged row r lies at c ^ (r % chunks).
    // Rows and columns that do not exist are cut off by the buffer's range
    // (columns by the offset's top bit): every store is issued.
    // The stores' whole offset is in the vector register: with a scalar
    // register added, the compiler takes the stored registers to be free at
    // once, and an instruction right behind a 16-byte store that writes them
    // was seen to change what lanes 12..15 of 16 store.  Without one it keeps
    // the distance.
    constexpr int ES = OUT32 ? 4 : 2;
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4_rw;
    constexpr int SROW = Shape::STAGE_ROW, CH = SROW / 16;  // bytes and chunks of a row
    constexpr int RPS = kWave / CH, ITS = 32 / RPS;          // rows a store, stores
    const uint32_t stage = lds_addr(smem) + Shape::STAGE_OFF + wave * Shape::STAGE_BYTES;
    const uint32_t ldc = (uint32_t)uniform((int)t.ldc);
    const __amdgpu_buffer_rsrc_t rc =
        byte_range_rsrc(uniform(t.c), (uint32_t)(t.c_rows - 1) * ldc + (uint32_t)t.c_cols * ES);
    const int r32 = lane & 31, half = lane >> 5;
    // the chunk this lane stores
    const int srow = lane / CH, schunk = lane % CH;
    // fp32 staging (fp32 results, or 16-bit ones that are added to what is
    // there, which round once): two passes a row block, of FN / 2 blocks
    auto stage_f32 = [&](auto i_c, auto pass_c) __attribute__((always_inline)) {
      constexpr int i = decltype(i_c)::value, pass = decltype(pass_c)::value;
      static_for<FN / 2>([&](auto jj_c) __attribute__((always_inline)) {
        constexpr int j = pass * (FN / 2) + decltype(jj_c)::value;
        asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = acc[i][j][4 * q + e];
          const int c = decltype(jj_c)::value * 8 + q * 2 + half;
          *(lds_u32x4_rw *)(uintptr_t)(stage + r32 * SROW + ((c ^ (r32 % CH)) * 16)) =
              __builtin_bit_cast(u32x4, w);
        }
      });
      const int col = wn * FN * 32 + pass * FN * 16 + schunk * 4;
      const uint32_t v0 = ((uint32_t)((wm + i * WM) * 32 + srow) * ldc + (uint32_t)col * ES) |
                          (col < t.c_cols ? 0u : 0x80000000u);
      u32x4 w[ITS];
#pragma unroll
      for (int it = 0; it < ITS; ++it) {
        const int row = it * RPS + srow;
        w[it] = *(lds_cu32x4_t *)(uintptr_t)(stage + row * SROW + ((schunk ^ (row % CH)) * 16));
      }
      if constexpr (OUT32) {
        if constexpr (ACC) {
          u32x4 o[ITS];
#pragma unroll
          for (int it = 0; it < ITS; ++it)
            o[it] = __builtin_amdgcn_raw_buffer_load_b128(
                rc, (int)(v0 + (uint32_t)(it * RPS) * ldc), 0, 0);
#pragma unroll
          for (int it = 0; it < ITS; ++it)
            w[it] = __builtin_bit_cast(u32x4, __builtin_bit_cast(f32x4, w[it]) +
                                                  __builtin_bit_cast(f32x4, o[it]));
        }
#pragma unroll
        for (int it = 0; it < ITS; ++it)
          __builtin_amdgcn_raw_buffer_store_b128(w[it], rc, (int)(v0 + (uint32_t)(it * RPS) * ldc), 0,
                                                 0);
      } else {
        u32x2 o[ITS];
#pragma unroll
        for (int it = 0; it < ITS; ++it)
          o[it] = __builtin_amdgcn_raw_buffer_load_b64(rc, (int)(v0 + (uint32_t)(it * RPS) * ldc), 0,
                                                 0);
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
          const f32x4 f = __builtin_bit_cast(f32x4, w[it]);
          const uint32_t o0 = o[it].x, o1 = o[it].y;
          u32x2 d;
          d.x = pack_half<F16>(f[0] + from_half_bits<F16>((uint16_t)o0),
                               f[1] + from_half_bits<F16>((uint16_t)(o0 >> 16)));
          d.y = pack_half<F16>(f[2] + from_half_bits<F16>((uint16_t)o1),
                               f[3] + from_half_bits<F16>((uint16_t)(o1 >> 16)));
          __builtin_amdgcn_raw_buffer_store_b64(d, rc, (int)(v0 + (uint32_t)(it * RPS) * ldc), 0,
                                                 0);
        }
      }
    };
    auto stage_half = [&](auto i_c) __attribute__((always_inline)) {
      constexpr int i = decltype(i_c)::value;
      static_for<FN>([&](auto j_c) __attribute__((always_inline)) {
        constexpr int j = decltype(j_c)::value;
        asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // columns 16 q ..
          uint32_t d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            d[e] = pack_half<F16>(acc[i][j][8 * q + 2 * e], acc[i][j][8 * q + 2 * e + 1]);
          // lanes l and l ^ 32 trade halves: eight columns a lane
          swap_halves(d[0], d[2]);
          swap_halves(d[1], d[3]);
          const int c = j * 4 + q * 2 + half;
          *(lds_u32x4_rw *)(uintptr_t)(stage + r32 * SROW + ((c ^ (r32 % CH)) * 16)) =
              u32x4{d[0], d[1], d[2], d[3]};
        }
      });
      const int col = wn * FN * 32 + schunk * 8;
      const uint32_t v0 = ((uint32_t)((wm + i * WM) * 32 + srow) * ldc + (uint32_t)col * 2) |
                          (col < t.c_cols ? 0u : 0x80000000u);
      u32x4 w[ITS];
#pragma unroll
      for (int it = 0; it < ITS; ++it) {
        const int row = it * RPS + srow;
        w[it] = *(lds_cu32x4_t *)(uintptr_t)(stage + row * SROW + ((schunk ^ (row % CH)) * 16));
      }
#pragma unroll
      for (int it = 0; it < ITS; ++it)
        __builtin_amdgcn_raw_buffer_store_b128(w[it], rc, (int)(v0 + (uint32_t)(it * RPS) * ldc), 0,
                                                 0);
    };
    if constexpr (OUT32 || ACC)
      static_for<NACT>([&](auto i_c) __attribute__((always_inline)) {
        stage_f32(i_c, I0{});
        stage_f32(i_c, I1{});
      });
    else
      static_for<NACT>([&](auto i_c) __attribute__((always_inline)) { stage_half(i_c); });
    __builtin_amdgcn_sched_barrier(0);
  };
  // one specialisation per count of active row blocks (wavefront-uniform)
  static_for<FM + 1>([&](auto c) __attribute__((always_inline)) {
    if (nact == decltype(c)::value) k_loop(c);
  });
  return nact == FM;
}

// ------------------------------------------------------- the tile lists --
// Rows of a group in the product and dx, TILE rows and columns a tile:
// q = rows / TILE full tiles of rows and a remainder, which is one more full
// tile or, with tiles of 256 and at most 128 rows left, a wide tile (when
// there is more than one column tile).  Bands of 8 row tiles, column-major
// inside a band, so that the workgroups of one XCD, which take neighbouring
// tiles, share a few row panels and a few column panels in its L2.  In the
// last band the wide tile of a column pair stands before the full tiles of
// the same columns.
constexpr int kBand = 8;
struct RowTiles {
  int full, rem_half, ntl, nwide, bands;
};
template <int TILE>
__device__ __forceinline__ RowTiles row_tiles(int rows, int ncol) {
  RowTiles t;
  t.ntl = (ncol + TILE - 1) / TILE;
  const int q = rows / TILE, rem = rows % TILE;
  const bool half = TILE == 256 && rem > 0 && rem <= 128 && t.ntl > 1;
  t.full = q + (rem > 0 && !half);
  t.rem_half = half ? rem : 0;
  t.nwide = half ? (t.ntl + 1) / 2 : 0;
  t.bands = max(1, (t.full + kBand - 1) / kBand);
  return t;
}
__device__ __forceinline__ int row_tile_units(const RowTiles &t) {
  return t.full * t.ntl + t.nwide;
}

// Unit r: its first row, first column, and whether it is a wide tile.
template <int TILE>
__device__ __forceinline__ void row_tile_at(const RowTiles &t, int r, int &row0, int &col0,
                                            bool &wide) {
  const int band = min(r / (kBand * t.ntl), t.bands - 1);
  r -= band * kBand * t.ntl;
  const int qb = min(kBand, t.full - band * kBand);
  wide = false;
  int m, n;
  if (TILE == 256 && band == t.bands - 1 && t.rem_half) {
    const int per = 2 * qb + 1, j = r / per, rr = r - j * per;
    if (rr == 0) {
      wide = true;
      row0 = t.full * TILE;
      col0 = j * 2 * TILE;
      return;
    }
    n = 2 * j + (rr - 1) / qb;
    m = (rr - 1) % qb;
  } else {
    n = r / qb;
    m = r % qb;
  }
  row0 = (band * kBand + m) * TILE;
  col0 = n * TILE;
}

}  // namespace
}  // namespace cco
