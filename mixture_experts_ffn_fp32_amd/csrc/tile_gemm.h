// MFMA tile pipeline of the products beside the layer (grouped products,
// Newton-Schulz products): one (BM x BN) tile of C = A B^T per block at a
// time, k-steps landing in an LDS ring by direct-to-LDS loads while an earlier
// slot is multiplied.  Three sizes of tile (TgBig, TgMid, TgSmall below).
//
// An operand is read in one of two layouts:
//   row layout     its rows are contiguous along the contraction; a k-step is
//                  BM rows of 128 bytes.
//   column layout  its rows run along the contraction (a transposed operand in
//                  its stored order); a k-step is 64 rows of BM columns, and
//                  MFMA fragments come from transposing LDS reads.
// and in one of three precisions (1, 2 or 3 parts a value):
//   single  bfloat16, 64 contraction indices per k-step.
//   split   a float32 value v as two float16, hi = f16(v), lo = f16(v - hi):
//           22 bits of v survive (|lo| <= 2^-11 |v|, |v - hi - lo| <= 2^-23 |v|
//           while lo is a normal float16), and hi hi' + hi lo' + lo hi' leaves
//           out lo lo' <= 2^-22 |v v'| (root mean square 2^-24.5).  Three float16
//           products at the full matrix rate thus give float32 accuracy, to two
//           or three bits at worst, at a third of that rate, against a ninth
//           that the float32 matrix instructions reach.  Values are scaled
//           by powers of two beforehand so that neither part leaves the
//           float16 range.  Stored per row in units of 128 bytes: 32 hi, then
//           the 32 lo of the same indices; a k-step is one unit of each row
//           (32 contraction indices), so both precisions load alike, and the
//           two halves of a unit are read from LDS once for three products.
//   triple  a float32 value v as three bfloat16, each the rounded rest of the ones before:
//           v = hi + mid + lo exactly (8 significant bits each; |mid| <= 2^-8 |v|, |lo| <=
//           2^-16 |v|), and hi hi' + hi mid' + mid hi' + mid mid' + hi lo' + lo hi' leaves
//           out mid lo' + lo mid' + lo lo' <= 2^-22.99 |v v'|.  Having float32's exponents the
//           parts need no scale, so a product is as exact as a float32 one whatever its
//           neighbours along the contraction or in other rows are; that costs six bfloat16
//           products for the three of `split`.  Values are stored times 2^24 (kTgLift), which
//           keeps the parts of the smallest ones normal numbers (and takes values from 2^104 and
//           sums from 2^80 on out of the range, as infinities and NaN, which the caller has to
//           replace).  The parts of a matrix are planes in its rows, and a block of 64
//           contraction indices takes six k-steps of the single kind, one per product
//           (tg_offset).
#pragma once

#include "lds_dma.h"
#include "moe_internal.h"

namespace moe {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short tg_v4s __attribute__((ext_vector_type(4)));

// WM x WN wavefronts of FM x FN fragments of 32 x 32; a ring of S k-steps, S - 1 of
// them in flight; ACOL / BCOL: operand in column layout; SWAP: B as the MFMA's first
// operand, so that a lane holds four consecutive columns of one row instead of four
// consecutive rows of one column.
template <int WM_, int WN_, int FM_, int FN_, int S_, int BPC_, bool AHEAD_>
struct TgShape {
  static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_, S = S_, BPC = BPC_;
  static constexpr bool AHEAD = AHEAD_;  // fragments a whole k-step ahead (tg_step_ahead)
  static constexpr int BM = WM * FM * 32, BN = WN * FN * 32, THREADS = WM * WN * 64;
  static constexpr int SLOT = (BM + BN) * 128;        // bytes of a ring slot
  static constexpr int NI = BM / (4 * WM * WN);       // loads per wavefront per k-step
  static_assert(BM == BN, "the first half of the wavefronts loads A, the other B");
};
// 64 x 64, the k-steps dealt to the four wavefronts, each multiplying whole tiles of its
// own k-steps (4 fragments, 1 LDS read per MFMA) from a ring of its own: no barrier in
// the loop.  Their sums are added through LDS, in wavefront order; then each wavefront
// writes one fragment (WM, WN, FM, FN are those of the epilogue).
struct TgSmall {
  static constexpr int WM = 2, WN = 2, FM = 1, FN = 1, S = 2, BPC = 1, WAVES = 4;
  static constexpr bool AHEAD = false;
  static constexpr int BM = 64, BN = 64, THREADS = 256;
  static constexpr int SLOT = (BM + BN) * 128;
  static constexpr int NI = BM / 8;                   // loads per operand per k-step
};
// 256 x 256, eight wavefronts of 64 x 128, one block per CU: 0.75 LDS reads per MFMA.
// 128 x 128, four wavefronts of 64 x 64, 1 read per MFMA, two blocks per CU that fill each
// other's barriers and epilogues; its fragments are read a whole k-step ahead (one group
// of four MFMAs does not cover an LDS read).  Then TgSmall.
//
// The larger tile is taken as soon as it gives more than half of the CUs one: a CU's time
// is then one such tile, and the next smaller size needs as many rounds at a lower rate
// (four tiles for one, over two blocks or the same CUs).  Measured, larger | smaller:
//   256 | 128  update of 8 matrices of 1408 x 2048, symmetric products of 168 tiles on 256
//              CUs, 2357 | 2637 us; of one of 4096 x 4096, 136 tiles, 3974 | 4325 us; grouped
//              y (bfloat16), 192 tiles, 51 | 58 us; 128 tiles, 36 | 29 us
//   128 | 64   update of 64 matrices of 256 x 512, 192 tiles, 362 | 384 us; of one of 2048 x
//              2048, 136 tiles, 861 | 858 us; grouped y (float32), 128 tiles, 50 | 40 us
using TgBig = TgShape<4, 2, 2, 4, 2, 1, false>;
using TgMid = TgShape<2, 2, 2, 2, 2, 2, true>;

template <class Shape, bool ACOL_, bool BCOL_, int PARTS_, bool SWAP_>
struct TgConfig : Shape {
  static constexpr int PARTS = PARTS_;
  static constexpr bool ACOL = ACOL_, BCOL = BCOL_, SPLIT = PARTS == 2, SWAP = SWAP_;
  static constexpr int KS = SPLIT ? 32 : 64;          // contraction indices per k-step
  static constexpr bool SMALL = Shape::BM == TgSmall::BM;
  static constexpr int LDS = Shape::S * Shape::SLOT * (SMALL ? TgSmall::WAVES : 1);
  static constexpr int WAVES_PER_SIMD = Shape::BPC * Shape::THREADS / 256;
};

// One operand of a tile.  Row layout: `rows` rows of `pitch` bytes, k-step s at
// byte 128 s of each.  Column layout: `rows` contraction rows of `pitch` bytes
// (later ones read as zeros), `width` columns (a multiple of 8).  All-int
// members beside the pointer: bools would be copied through memory.
struct TgOperand {
  const uint8_t* p;
  uint32_t pitch;
  int rows, width;
  uint32_t plane;  // triple: bytes from one part of a row to the next
};

// Triple: which part of A and of B the j-th k-step of a block takes, two bits each (hi 0,
// mid 1, lo 2); neighbours share an operand.
constexpr int kTgProducts = 6;
constexpr int tg_parts(int a, int b, int c, int d, int e, int f) {
  return a | b << 2 | c << 4 | d << 6 | e << 8 | f << 10;
}
constexpr int kTgPartsA = tg_parts(0, 0, 0, 1, 1, 2), kTgPartsB = tg_parts(2, 1, 0, 0, 1, 0);
// The power of two that stored values carry, and what takes it back out of a product.
constexpr float kTgLift = 0x1p24f, kTgUnlift = 0x1p-48f;

// Loading state of one wavefront for a tile.
struct TgLoad {
  const uint8_t* base;
  uint32_t step;   // bytes from one k-step to the next
  int rows;        // column layout: contraction rows; row layout: -(k-steps)
  uint32_t pitch;
  uint32_t plane;  // triple
  int parts;       // triple: kTgPartsA or kTgPartsB
};
// Bytes from its base to k-step s.
template <class C>
__device__ __forceinline__ size_t tg_offset(const TgLoad& l, int s) {
  if constexpr (C::PARTS == 3) {
    const int b = s / kTgProducts, part = (l.parts >> (2 * (s - kTgProducts * b))) & 3;
    return (size_t)b * l.step + (size_t)part * l.plane;
  }
  return (size_t)s * l.step;
}

// In a column-layout tile of W columns the 16-byte chunk c of contraction row k lies at
// position c ^ 4 j(k): a transposing read of 32 lanes touches 64 bytes of each of four
// consecutive rows, and the rotation puts them on distinct banks (rows of 128 bytes
// share a bank window in pairs).
template <int W>
__device__ __forceinline__ int tg_rotation(int k) {
  return W >= 128 ? k & 3 : (k >> 1) & 1;
}
template <class C, bool COL>
__device__ __forceinline__ TgLoad tg_prepare_side(const TgOperand& o, int parts, int t0, int steps,
                                                  int w, int lane, uint32_t (&off)[C::NI]) {
  constexpr int W = C::BM;
  TgLoad l;
  l.pitch = uni((int)o.pitch);
  l.plane = C::PARTS == 3 ? uni((int)o.plane) : 0;
  l.parts = parts;
  if constexpr (COL) {
    constexpr int RPI = 1024 / (2 * W);  // contraction rows per load instruction
    constexpr int CPR = W / 8;           // chunks per row
    l.base = uni(o.p);
    l.step = l.pitch * C::KS;
    l.rows = uni(o.rows);
#pragma unroll
    for (int i = 0; i < C::NI; ++i) {
      const int k = (w * C::NI + i) * RPI + lane / CPR;  // LDS row 0..63
      const int c = (lane % CPR) ^ (tg_rotation<W>(k) << 2);
      // columns past the last one reread the last chunk (never stored)
      const int col = min(t0 + 8 * c, o.width - 8);
      if constexpr (C::SPLIT)
        off[i] = (uint32_t)(k & 31) * l.pitch + (col >> 5) * 128 + (col & 31) * 2 + (k >> 5) * 64;
      else
        off[i] = (uint32_t)k * l.pitch + col * 2;
    }
  } else {
    const int r0 = min(t0, o.rows - 1);
    l.base = uni(o.p + (size_t)r0 * o.pitch);
    l.step = 128;
    // a wavefront whose rows all lie past the last one loads nothing (range 0)
    l.rows = t0 + w * C::NI * 8 < o.rows ? -uni(steps) : 0;
#pragma unroll
    for (int i = 0; i < C::NI; ++i) {
      const int r = (w * C::NI + i) * 8 + (lane >> 3);
      // rows past the last one reread it (never stored)
      off[i] = (uint32_t)(min(t0 + r, o.rows - 1) - r0) * l.pitch +
               (((lane & 7) ^ ((r >> 1) & 7)) << 4);
    }
  }
  return l;
}

// This wavefront's loads of a tile at (m0, n0): A in the first half of them, B in the other.
template <class C>
__device__ __forceinline__ TgLoad tg_prepare(const TgOperand& A, const TgOperand& B, int m0, int n0,
                                             int steps, int wave, int lane,
                                             uint32_t (&off)[C::NI]) {
  constexpr int H = C::WM * C::WN / 2;
  if (wave < H) return tg_prepare_side<C, C::ACOL>(A, kTgPartsA, m0, steps, wave, lane, off);
  return tg_prepare_side<C, C::BCOL>(B, kTgPartsB, n0, steps, wave - H, lane, off);
}

// Bytes from the k-step's base that its loads may touch; later ones read zeros.
template <class C>
__device__ __forceinline__ int tg_range(const TgLoad& l, int s) {
  if (l.rows < 0) return s < -l.rows ? 0x7fffffff : 0;
  if constexpr (C::PARTS == 3) s /= kTgProducts;
  return min(max(l.rows - C::KS * s, 0), C::KS) * (int)l.pitch;
}

__device__ __forceinline__ uint2 tg_read_tr(const uint8_t* p) {
  const tg_v4s v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) tg_v4s*)(__attribute__((address_space(3))) const uint8_t*)p);
  return __builtin_bit_cast(uint2, v);
}

// Fragment of k-group kg (16 indices), 32 rows (columns) of a tile, at 32 u: lane l
// holds row l % 32, indices 8 (l / 32) .. of the group.
//
// Column layout, transposing reads: within each 16-lane group lane l names contraction
// row k = 8 (l / 32) + (l % 16) / 4 (+ 4 for the upper four) of the group at column
// 16 ((l / 16) % 2) + 4 (l % 4) of the fragment.  Its chunk is 4 u + c, c < 4, rotated
// to 4 (u ^ j(k)) + c: everything but u % 4 and the lane is a constant offset.
template <int W, bool COL>
__device__ __forceinline__ u32x4 tg_frag(const uint8_t* rd, int kg, int u_const, int u_wave,
                                         int lane) {
  if constexpr (COL) {
    const int k = 8 * (lane >> 5) + ((lane & 15) >> 2), n = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    // u = u_const + u_wave: the low two bits of u_const + u_wave, without a carry
    const int low = ((u_const & 3) + u_wave) ^ tg_rotation<W>(k);
    const uint8_t* p = rd + k * (2 * W) + low * 64 + (n >> 3) * 16 + (n & 7) * 2 +
                       (kg * 16 * (2 * W) + (u_const >> 2) * 256);
    const uint2 lo = tg_read_tr(p), hi = tg_read_tr(p + 4 * 2 * W);
    return u32x4{lo.x, lo.y, hi.x, hi.y};
  } else {
    return *(const u32x4*)(rd + lds_chunk_offset(u_wave * 32 + (lane & 31), kg * 2 + (lane >> 5)) +
                           u_const * 32 * 128);
  }
}

// The wavefronts' fragments interleave: fragment (fm, fn) of wavefront (wm, wn) is
// rows (WM fm + wm) 32 .. and columns (WN fn + wn) 32 .. of the tile, so a tile whose
// matrix ends after half its rows (or half its columns) leaves out whole fragments
// of every wavefront, and they stay balanced.
template <class C, int FMA>
__device__ __forceinline__ void tg_frags_a(const uint8_t* __restrict__ rd, int kg, int wm, int lane,
                                           u32x4 (&f)[C::FM]) {
#pragma unroll
  for (int i = 0; i < FMA; ++i) f[i] = tg_frag<C::BM, C::ACOL>(rd, kg, C::WM * i, wm, lane);
}
template <class C, int FNA>
__device__ __forceinline__ void tg_frags_b(const uint8_t* __restrict__ rd, int kg, int wn, int lane,
                                           u32x4 (&f)[C::FN]) {
#pragma unroll
  for (int i = 0; i < FNA; ++i)
    f[i] = tg_frag<C::BN, C::BCOL>(rd + C::BM * 128, kg, C::WN * i, wn, lane);
}

// The fragments a tile multiplies: FMA x FNA of the configuration's FM x FN;
// TRI leaves out the lower left quarter (a symmetric product's diagonal tile).
template <class C, bool TRI>
__device__ __forceinline__ constexpr bool tg_skip(int fm, int fn) {
  return TRI && fm >= C::FM / 2 && fn < C::FN / 2;
}
template <class C, int FMA, int FNA, bool TRI>
__device__ __forceinline__ void tg_products(const u32x4 (&a)[C::FM], const u32x4 (&b)[C::FN],
                                            f32x16 (&acc)[C::FM][C::FN]) {
#pragma unroll
  for (int fm = 0; fm < FMA; ++fm)
#pragma unroll
    for (int fn = 0; fn < FNA; ++fn) {
      if (tg_skip<C, TRI>(fm, fn)) continue;
      const u32x4 x = C::SWAP ? b[fn] : a[fm], y = C::SWAP ? a[fm] : b[fn];
      if constexpr (C::SPLIT)
        acc[fm][fn] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            __builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), acc[fm][fn], 0, 0, 0);
      else
        acc[fm][fn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), acc[fm][fn], 0, 0, 0);
    }
}

// Order of one group of MF MFMAs with NR LDS reads and ND loads: the reads directly
// behind the first MFMAs (one each, two where there are more), so that the rest of the
// group covers their latency, also before a barrier that waits for them; the loads
// behind the reads, which the next group needs first.
template <int MF, int NR, int ND>
__device__ __forceinline__ void tg_order() {
  constexpr int PER = (NR + MF - 1) / MF > 1 || (ND > 0 && MF > 2) ? 2 : 1;
  constexpr int RM = PER > 0 ? (NR + PER - 1) / PER : 0;            // MFMAs followed by reads
  constexpr int DM = MF - (RM < MF ? RM : MF - 1);                  // MFMAs followed by loads
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
    for (int r = m * PER; r < (m + 1) * PER && r < NR; ++r)
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    if (m >= MF - DM) {
      const int i = m - (MF - DM);
#pragma unroll
      for (int r = i * ND / DM; r < (i + 1) * ND / DM; ++r)
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
  }
#pragma unroll
  for (int r = MF * PER; r < NR; ++r) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
}

// Fragments that pass from one k-step to the next: on entry a[0] / b[0] hold the first
// group of 16 indices (split: of its hi halves).
template <class C>
struct TgFrags {
  u32x4 a[2][C::FM], b[2][C::FN];
};

// One k-step out of ring slot `rd`, every fragment read one group ahead of its use.
// The barrier stands before the last group, whose fragments are in registers by
// then: `rd` is free, the next k-step (slot `nx`) has landed, and the last group's
// MFMAs cover both the reads of the next k-step's first fragments and the loads of
// the one after it (`db` + off into `wr`, range `nrec`: 0 reads zeros without
// touching memory).  `wr` is `rd` again, under a name of its own: with the loads and
// the reads in separate restrict scopes the compiler does not make every fragment
// read wait for the loads in flight, and the barrier's fences keep their order.
template <class C, int FMA, int FNA, bool TRI>
__device__ __forceinline__ void tg_step(const uint8_t* __restrict__ rd,
                                        const uint8_t* __restrict__ nx, int wm, int wn, int lane,
                                        TgFrags<C>& f, f32x16 (&acc)[C::FM][C::FN],
                                        const uint8_t* db, const uint32_t (&off)[C::NI],
                                        uint8_t* __restrict__ wr, int nrec, bool landed) {
  constexpr int MF = FMA * FNA - (TRI ? C::FM * C::FN / 4 : 0);
  constexpr int RA = FMA * (C::ACOL ? 2 : 1), RB = FNA * (C::BCOL ? 2 : 1);
  if constexpr (C::SPLIT) {
    // per 16 indices: hi hi', hi lo', lo hi'
    u32x4 al[C::FM], bl[C::FN];
    tg_frags_b<C, FNA>(rd, 2, wn, lane, bl);
    tg_products<C, FMA, FNA, TRI>(f.a[0], f.b[0], acc);
    tg_frags_a<C, FMA>(rd, 2, wm, lane, al);
    tg_products<C, FMA, FNA, TRI>(f.a[0], bl, acc);
    tg_frags_a<C, FMA>(rd, 1, wm, lane, f.a[1]);
    tg_frags_b<C, FNA>(rd, 1, wn, lane, f.b[1]);
    tg_products<C, FMA, FNA, TRI>(al, f.b[0], acc);
    tg_frags_b<C, FNA>(rd, 3, wn, lane, bl);
    tg_products<C, FMA, FNA, TRI>(f.a[1], f.b[1], acc);
    tg_frags_a<C, FMA>(rd, 3, wm, lane, al);
    tg_products<C, FMA, FNA, TRI>(f.a[1], bl, acc);
    tg_order<MF, RB, 0>();
    tg_order<MF, RA, 0>();
    tg_order<MF, RA + RB, 0>();
    tg_order<MF, RB, 0>();
    tg_order<MF, RA, 0>();
    if (!landed) MOE_WAIT_VMCNT((C::S - 2) * C::NI);
    lds_sync();
    tg_frags_a<C, FMA>(nx, 0, wm, lane, f.a[0]);
    tg_frags_b<C, FNA>(nx, 0, wn, lane, f.b[0]);
#pragma unroll
    for (int i = 0; i < C::NI; ++i) dma16(db, off[i], wr + i * 1024, nrec);
    tg_products<C, FMA, FNA, TRI>(al, f.b[1], acc);
    tg_order<MF, RA + RB, C::NI>();
  } else {
#pragma unroll
    for (int kg = 0; kg < 3; ++kg) {
      tg_frags_a<C, FMA>(rd, kg + 1, wm, lane, f.a[(kg + 1) & 1]);
      tg_frags_b<C, FNA>(rd, kg + 1, wn, lane, f.b[(kg + 1) & 1]);
      tg_products<C, FMA, FNA, TRI>(f.a[kg & 1], f.b[kg & 1], acc);
    }
    tg_order<MF, RA + RB, 0>();
    tg_order<MF, RA + RB, 0>();
    tg_order<MF, RA + RB, 0>();
    if (!landed) MOE_WAIT_VMCNT((C::S - 2) * C::NI);
    lds_sync();
    tg_frags_a<C, FMA>(nx, 0, wm, lane, f.a[0]);
    tg_frags_b<C, FNA>(nx, 0, wn, lane, f.b[0]);
#pragma unroll
    for (int i = 0; i < C::NI; ++i) dma16(db, off[i], wr + i * 1024, nrec);
    tg_products<C, FMA, FNA, TRI>(f.a[1], f.b[1], acc);
    tg_order<MF, RA + RB, C::NI>();
  }
}

// All fragments of a k-step.
template <class C>
struct TgWhole {
  u32x4 a[4][C::FM], b[4][C::FN];
};
template <class C, int FMA, int FNA>
__device__ __forceinline__ void tg_read_whole(const uint8_t* __restrict__ rd, int wm, int wn,
                                              int lane, TgWhole<C>& f) {
#pragma unroll
  for (int kg = 0; kg < 4; ++kg) {
    tg_frags_a<C, FMA>(rd, kg, wm, lane, f.a[kg]);
    tg_frags_b<C, FNA>(rd, kg, wn, lane, f.b[kg]);
  }
}

// One k-step from registers (f), the next one's fragments (slot `nx`) read into g
// meanwhile.  The barrier stands before it: every wavefront has read this k-step's
// slot, which takes the loads of the k-step S further on (as in tg_step).
template <class C, int FMA, int FNA, bool TRI>
__device__ __forceinline__ void tg_step_ahead(const uint8_t* __restrict__ nx, int wm, int wn,
                                              int lane, const TgWhole<C>& f, TgWhole<C>& g,
                                              f32x16 (&acc)[C::FM][C::FN], const uint8_t* db,
                                              const uint32_t (&off)[C::NI],
                                              uint8_t* __restrict__ wr, int nrec, bool landed) {
  constexpr int MF = FMA * FNA - (TRI ? C::FM * C::FN / 4 : 0);
  constexpr int NR = 4 * (FMA * (C::ACOL ? 2 : 1) + FNA * (C::BCOL ? 2 : 1));
  if (!landed) MOE_WAIT_VMCNT((C::S - 2) * C::NI);
  lds_sync();
  tg_read_whole<C, FMA, FNA>(nx, wm, wn, lane, g);
#pragma unroll
  for (int i = 0; i < C::NI; ++i) dma16(db, off[i], wr + i * 1024, nrec);
  if constexpr (C::SPLIT) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      tg_products<C, FMA, FNA, TRI>(f.a[h], f.b[h], acc);
      tg_products<C, FMA, FNA, TRI>(f.a[h], f.b[2 + h], acc);
      tg_products<C, FMA, FNA, TRI>(f.a[2 + h], f.b[h], acc);
    }
    tg_order<6 * MF, NR, C::NI>();
  } else {
#pragma unroll
    for (int kg = 0; kg < 4; ++kg) tg_products<C, FMA, FNA, TRI>(f.a[kg], f.b[kg], acc);
    tg_order<4 * MF, NR, C::NI>();
  }
}

// Row and column (inside the tile) of accumulator register r of fragment (fm, fn).
template <class C>
__device__ __forceinline__ int tg_row(int wm, int fm, int lane, int r) {
  return (C::WM * fm + wm) * 32 + (C::SWAP ? (lane & 31) : 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3));
}
template <class C>
__device__ __forceinline__ int tg_col(int wn, int fn, int lane, int r) {
  return (C::WN * fn + wn) * 32 + (C::SWAP ? 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3) : (lane & 31));
}

// The four 8-byte groups a lane holds of a fragment's 32 consecutive elements
// (group g: elements 8g + 4 (lane / 32) ..) as two 16-byte runs: after exchanging
// halves between lanes l and l + 32, r0 is elements 8 (lane / 32) .. and r1 the same
// 16 further on.
__device__ __forceinline__ void tg_runs16(uint2 (&w)[4], u32x4& r0, u32x4& r1) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0].x, w[1].x, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[0].y, w[1].y, false, false);
  const auto c = __builtin_amdgcn_permlane32_swap(w[2].x, w[3].x, false, false);
  const auto d = __builtin_amdgcn_permlane32_swap(w[2].y, w[3].y, false, false);
  r0 = u32x4{a[0], b[0], a[1], b[1]};
  r1 = u32x4{c[0], d[0], c[1], d[1]};
}

// Transposes the 4 x 4 16-bit values of four neighbouring lanes: lane j holds
// values (0..3, j) and receives (j, 0..3).
__device__ __forceinline__ uint2 tg_quad_transpose(uint2 v, int lane) {
  const bool odd = lane & 1, up = lane & 2;
  // with lane ^ 1: even lanes take values 0 and 2, odd ones 1 and 3, of both
  const uint32_t tx = __builtin_amdgcn_mov_dpp(v.x, 0xB1, 0xf, 0xf, true);
  const uint32_t ty = __builtin_amdgcn_mov_dpp(v.y, 0xB1, 0xf, 0xf, true);
  const uint32_t a = odd ? (tx >> 16) | (v.x & 0xffff0000u) : (v.x & 0xffffu) | (tx << 16);
  const uint32_t b = odd ? (ty >> 16) | (v.y & 0xffff0000u) : (v.y & 0xffffu) | (ty << 16);
  // with lane ^ 2
  const uint32_t r = __builtin_amdgcn_mov_dpp(up ? a : b, 0x4E, 0xf, 0xf, true);
  return up ? uint2{r, b} : uint2{a, r};
}

// A block's tiles.  The blocks are dealt to the eight XCDs round-robin, and each XCD
// owns a contiguous range of the tiles, whose neighbours share operands in its L2.  A
// block starts with the tile of its XCD's range by its index there.  With `counters`
// (8 zeros) it claims the following ones, from its XCD's range first and then from the
// others' (the tiles differ in length and the XCDs in clock), else it takes every P-th
// (P: the XCD's blocks).  Wavefront 0 claims the tile after the next one at a tile's
// start and passes it on through LDS at its end.
// (Taking the shorter tiles last for an even end costs more than it saves: a short tile
// shares its operands with its neighbours, prefill product 328 -> 352 us.)
struct TgTiles {
  int n, X, x, y, own;       // y: the range to claim from; own: the block's place in its XCD
  int32_t* counters;

  __device__ __forceinline__ int blocks(int xcd) const { return ((int)gridDim.x - xcd + X - 1) / X; }
  // The j-th tile of an XCD's range, or -1.
  __device__ __forceinline__ int at(int xcd, int j) const {
    const int a = (int)((long long)n * xcd / X), b = (int)((long long)n * (xcd + 1) / X);
    return j < b - a ? a + j : -1;
  }
  __device__ __forceinline__ void init(int tiles, int32_t* c) {
    n = tiles;
    counters = c;
    X = min(8, (int)gridDim.x);
    x = y = blockIdx.x % X;
    own = blockIdx.x / X;
  }
  // One whole wavefront: the next tile, or -1.  A range's first entries are the tiles
  // its own blocks started with, so claims begin behind those.  Once its XCD's range is
  // used up, eight lanes look at all the counters at once.
  __device__ __forceinline__ int claim(int lane) {
    while (true) {
      int j = 0;
      if (lane == 0) j = atomicAdd(counters + y, 1);
      const int t = at(y, blocks(y) + uni(j));
      if (t >= 0) return t;
      bool some = false;
      const int z = (x + lane) % X;
      if (lane < X)
        some = at(z, blocks(z) + __hip_atomic_load(counters + z, __ATOMIC_RELAXED,
                                                   __HIP_MEMORY_SCOPE_AGENT)) >= 0;
      const uint64_t left = __ballot(some);
      if (left == 0) return -1;
      y = (x + __builtin_ctzll(left)) % X;
    }
  }
};
constexpr int kTgCounters = 8;

// The loads' place in the stream of k-steps of a block's tiles, S k-steps ahead of the
// multiplication.  Plain scalars: with the tile itself in it the structure ends
// up in scratch memory.
struct TgCursor {
  int hint;
  int s, steps;      // the tile's next k-step, its k-steps (0: the stream has ended)
};

// k-steps of a tile: S + 1 at least (after a short contraction come k-steps of zeros),
// and an even number where the fragments go through two sets of registers.
template <class C>
__device__ __forceinline__ int tg_steps(int steps) {
  const int n = max(steps, C::S + 1);
  return C::AHEAD ? (n + 1) & ~1 : n;
}

// The cursor to tile L (-1: the stream has ended).
template <class C, class P>
__device__ __forceinline__ void tg_seek(const P& p, int L, TgCursor& c, TgLoad& ld,
                                        uint32_t (&off)[C::NI], int wave, int lane) {
  c.s = 0;
  c.steps = 0;
  if (L < 0) return;
  const typename P::Tile t = p.tile(L, c.hint);
  c.hint = uni(t.hint);
  c.steps = tg_steps<C>(uni(t.steps));
  ld = tg_prepare<C>(t.A, t.B, t.m0, t.n0, t.steps, wave, lane, off);
}

// The k-steps of a tile.  As there are at least S + 1, the cursor, S ahead, passes to
// the next tile, which is next(), while this one is multiplied, behind its first barrier.
template <class C, int FMA, int FNA, bool TRI, class P, class Next>
__device__ __forceinline__ void tg_tile(const P& p, int steps, int& ph, int wave, int lane,
                                        Next next, TgCursor& c, TgLoad& ld,
                                        uint32_t (&off)[C::NI], f32x16 (&acc)[C::FM][C::FN],
                                        uint8_t* __restrict__ lds) {
  const int wm = wave / C::WN, wn = wave % C::WN;
  // (opaque: the fragments' LDS addresses stay inside the tile, where they are few,
  // and do not spill what the epilogue keeps)
  asm volatile("" : "+v"(lane));
  // The first fragments are not carried over from the last tile, which may have read
  // fewer.
  const int all = tg_steps<C>(steps);
  auto issue = [&](auto step) {
    const int after = ph + 1 < C::S ? ph + 1 : 0;
    const uint8_t* db = uni(ld.base + tg_offset<C>(ld, c.s));
    const int nrec = uni(c.steps > 0 ? tg_range<C>(ld, c.s) : 0);
    step(lds + ph * C::SLOT, lds + after * C::SLOT, db, nrec);
    c.s = uni(c.s + 1);
    if (c.s == c.steps) tg_seek<C>(p, next(), c, ld, off, wave, lane);
    ph = after;
  };
  if constexpr (C::AHEAD) {
    TgWhole<C> f, g;
    tg_read_whole<C, FMA, FNA>(lds + ph * C::SLOT, wm, wn, lane, f);
    for (int s = 0; s < all; s += 2) {
      issue([&](uint8_t* rd, const uint8_t* nx, const uint8_t* db, int nrec) {
        tg_step_ahead<C, FMA, FNA, TRI>(nx, wm, wn, lane, f, g, acc, db, off,
                                        rd + wave * C::NI * 1024, nrec, s < C::S - 1);
      });
      issue([&](uint8_t* rd, const uint8_t* nx, const uint8_t* db, int nrec) {
        tg_step_ahead<C, FMA, FNA, TRI>(nx, wm, wn, lane, g, f, acc, db, off,
                                        rd + wave * C::NI * 1024, nrec, s + 1 < C::S - 1);
      });
    }
  } else {
    TgFrags<C> f;
    tg_frags_a<C, FMA>(lds + ph * C::SLOT, 0, wm, lane, f.a[0]);
    tg_frags_b<C, FNA>(lds + ph * C::SLOT, 0, wn, lane, f.b[0]);
    for (int s = 0; s < all; ++s)
      issue([&](uint8_t* rd, const uint8_t* nx, const uint8_t* db, int nrec) {
        tg_step<C, FMA, FNA, TRI>(rd, nx, wm, wn, lane, f, acc, db, off, rd + wave * C::NI * 1024,
                                  nrec, s < C::S - 1);
      });
  }
}

// The persistent loop over a block's tiles of problem P:
//   P::Tile   { TgOperand A, B; int m0, n0, steps, rows, cols, hint; ... }, rows and
//             cols being the tile's that exist (any number above BM, BN counts as all)
//   p.tile(L, hint)    the L-th tile; uniform.  hint: an earlier tile's, or 0
//   p.tri(t)           whether its lower left quarter is left out
//   p.store(t, wm, wn, lane, acc)   the epilogue, from registers
template <class C, class P>
__device__ __forceinline__ void tg_run(const P& p, int tiles, int32_t* counters,
                                       uint8_t* __restrict__ lds, int* s_claim) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uni(tid >> 6), wm = wave / C::WN, wn = wave % C::WN;
  TgTiles q;
  q.init(tiles, counters);
  int mine = q.own;
  int L = q.at(q.x, mine);
  if (L < 0) return;
  TgCursor c{0, 0, 0};
  TgLoad ld{};
  uint32_t off[C::NI] = {};
  tg_seek<C>(p, L, c, ld, off, wave, lane);
  int ph = 0;  // ring slot of the next k-step
#pragma unroll
  for (int k = 0; k < C::S; ++k) {
    uint8_t* w = lds + k * C::SLOT + wave * C::NI * 1024;
    const uint8_t* db = uni(ld.base + tg_offset<C>(ld, c.s));
    const int nrec = uni(tg_range<C>(ld, c.s));
#pragma unroll
    for (int i = 0; i < C::NI; ++i) dma16(db, off[i], w + i * 1024, nrec);
    c.s = uni(c.s + 1);
  }
  // the next tile
  if (counters != nullptr && wave == 0) {
    const int p1 = q.claim(lane);
    if (lane == 0) *s_claim = p1;
  }
  pipe_sync();
  int L1 = -1;
  auto next = [&]() -> int {
    L1 = counters != nullptr ? uni(*s_claim) : q.at(q.x, mine += q.blocks(q.x));
    return L1;
  };
  int hint = 0;
  while (true) {
    const typename P::Tile t = p.tile(L, hint);
    hint = t.hint;
    int claimed = -1;
    if (counters != nullptr && wave == 0) claimed = q.claim(lane);
    f32x16 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    static_assert(C::FM == 2, "half tiles leave out whole fragments");
    constexpr int H = C::FN / 2;
    const bool hm = t.rows <= C::BM / 2, hn = t.cols <= C::BN / 2;
    if (hm && hn) tg_tile<C, 1, H, false>(p, t.steps, ph, wave, lane, next, c, ld, off, acc, lds);
    else if (hm) tg_tile<C, 1, C::FN, false>(p, t.steps, ph, wave, lane, next, c, ld, off, acc, lds);
    else if (hn) tg_tile<C, 2, H, false>(p, t.steps, ph, wave, lane, next, c, ld, off, acc, lds);
    else if (P::SYM && p.tri(t))
      tg_tile<C, 2, C::FN, P::SYM>(p, t.steps, ph, wave, lane, next, c, ld, off, acc, lds);
    else tg_tile<C, 2, C::FN, false>(p, t.steps, ph, wave, lane, next, c, ld, off, acc, lds);
    // the loads in flight are waited for here (the next tile's first k-steps; the very
    // first one landed before the last barrier): its loop needs no wait for them
    MOE_WAIT_VMCNT(0);
    if (counters != nullptr && tid == 0) *s_claim = claimed;  // read behind its first barrier
    p.store(t, wm, wn, lane, acc);
    if (L1 < 0) break;
    L = L1;
  }
}

// One wavefront of TgSmall in its loop: a whole tile of 2 x 2 fragments.
template <class C>
struct TgOne : C {
  static constexpr int WM = 1, WN = 1, FM = 2, FN = 2;
};

// A wavefront's `mine` k-steps (wave, wave + 4, ..) of a 64 x 64 tile: two in its ring;
// a k-step's fragments are read, its slot takes the loads two further on, then they are
// multiplied.
template <class C, class One>
__device__ __forceinline__ void tg_small_loop(const TgLoad& la, const TgLoad& lb,
                                              const uint32_t (&oa)[C::NI],
                                              const uint32_t (&ob)[C::NI], int mine, int wave,
                                              int lane, f32x16 (&acc)[2][2],
                                              uint8_t* __restrict__ slot0,
                                              uint8_t* __restrict__ slot1) {
  constexpr int W = TgSmall::WAVES, NI = C::NI;
  auto issue = [&](int i, uint8_t* slot) {
    const int s = wave + W * i;
    const int na = uni(i < mine ? tg_range<C>(la, s) : 0), nb = uni(i < mine ? tg_range<C>(lb, s) : 0);
    const uint8_t* da = uni(la.base + tg_offset<C>(la, s));
    const uint8_t* db = uni(lb.base + tg_offset<C>(lb, s));
#pragma unroll
    for (int k = 0; k < NI; ++k) dma16(da, oa[k], slot + k * 1024, na);
#pragma unroll
    for (int k = 0; k < NI; ++k) dma16(db, ob[k], slot + C::BM * 128 + k * 1024, nb);
  };
  issue(0, slot0);
  issue(1, slot1);
  for (int i = 0; i < mine; ++i) {
    uint8_t* slot = i & 1 ? slot1 : slot0;
    MOE_WAIT_VMCNT(2 * NI);  // this k-step has landed, the next one may be in flight
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    TgWhole<One> f;
    tg_read_whole<One, 2, 2>(slot, 0, 0, lane, f);
    MOE_WAIT_LGKMCNT0();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    issue(i + 2, slot);
    if constexpr (C::SPLIT) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        tg_products<One, 2, 2, false>(f.a[h], f.b[h], acc);
        tg_products<One, 2, 2, false>(f.a[h], f.b[2 + h], acc);
        tg_products<One, 2, 2, false>(f.a[2 + h], f.b[h], acc);
      }
    } else {
#pragma unroll
      for (int kg = 0; kg < 4; ++kg) tg_products<One, 2, 2, false>(f.a[kg], f.b[kg], acc);
    }
  }
  MOE_WAIT_VMCNT(0);  // the sums go through the ring
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The same for TgSmall.
template <class C, class P>
__device__ __forceinline__ void tg_run_small(const P& p, int tiles, uint8_t* __restrict__ lds) {
  constexpr int W = TgSmall::WAVES, NI = C::NI;
  using One = TgOne<C>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uni(tid >> 6);
  uint8_t* ring = lds + wave * (C::S * C::SLOT);
  TgTiles q;
  q.init(tiles, nullptr);
  int hint = 0;
  for (int j = q.own;; j += q.blocks(q.x)) {
    const int L = q.at(q.x, j);
    if (L < 0) break;
    const typename P::Tile t = p.tile(L, hint);
    hint = t.hint;
    uint32_t oa[NI], ob[NI];
    const TgLoad la = tg_prepare_side<C, C::ACOL>(t.A, kTgPartsA, t.m0, t.steps, 0, lane, oa);
    const TgLoad lb = tg_prepare_side<C, C::BCOL>(t.B, kTgPartsB, t.n0, t.steps, 0, lane, ob);
    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][k][r] = 0.f;
    const int mine = t.steps > wave ? (t.steps - wave + W - 1) / W : 0;
    tg_small_loop<C, One>(la, lb, oa, ob, mine, wave, lane, acc, ring, ring + C::SLOT);
    // the four sums through this wavefront's ring, every fragment as 16-byte runs
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *(f32x4*)(ring + f * 4096 + r * 1024 + lane * 16) =
            f32x4{acc[f >> 1][f & 1][4 * r], acc[f >> 1][f & 1][4 * r + 1],
                  acc[f >> 1][f & 1][4 * r + 2], acc[f >> 1][f & 1][4 * r + 3]};
    __syncthreads();
    f32x16 sum[1][1];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const f32x4 o = *(const f32x4*)(lds + w * (C::S * C::SLOT) + wave * 4096 + r * 1024 + lane * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += o[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[0][0][4 * r + e] = v[e];
    }
    __syncthreads();  // the rings take the next tile's loads
    p.store(t, wave / C::WN, wave % C::WN, lane, sum);
  }
}

// Eight values as three bfloat16 each.
struct Split3 {
  u32x4 hi, mid, lo;
};
__device__ __forceinline__ Split3 split_three(const float (&v)[8]) {
  Split3 s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = v[2 * i], b = v[2 * i + 1];
    s.hi[i] = pack_bf16x2(a, b);
    a -= __uint_as_float(s.hi[i] << 16);
    b -= __uint_as_float(s.hi[i] & 0xffff0000u);
    s.mid[i] = pack_bf16x2(a, b);
    a -= __uint_as_float(s.mid[i] << 16);
    b -= __uint_as_float(s.mid[i] & 0xffff0000u);
    s.lo[i] = pack_bf16x2(a, b);
  }
  return s;
}

// A value as two float16.
__device__ __forceinline__ void split_f16(float v, uint16_t& hi, uint16_t& lo) {
  const _Float16 h = (_Float16)v;
  const _Float16 l = (_Float16)(v - (float)h);
  hi = __builtin_bit_cast(uint16_t, h);
  lo = __builtin_bit_cast(uint16_t, l);
}

// Bytes of a split row of n values, and the place of element j's hi in it (its lo
// is 64 bytes further).
__host__ __device__ inline long long split_pitch(int n) { return (long long)((n + 31) / 32) * 128; }
__device__ __forceinline__ long long split_at(int j) { return (long long)(j >> 5) * 128 + (j & 31) * 2; }


// Elements j .. j + 7 of a row of `width` as float32, zeros past its end.  Rows whose
// width is a whole number of 16 bytes start 16-byte aligned.
template <class E>
__device__ __forceinline__ void load_chunk(const typename E::T* __restrict__ src, long long j,
                                           long long width, float (&f)[8]) {
  if (j + 8 <= width && width % E::kPerChunk == 0) {
    if constexpr (sizeof(typename E::T) == 4) {
      const f32x4 a = *(const f32x4*)(src + j), b = *(const f32x4*)(src + j + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = a[e];
        f[4 + e] = b[e];
      }
    } else {
      const u32x4 v = *(const u32x4*)(src + j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(v[e] << 16);
        f[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = j + e < width ? load_as_f32<E>(src + j + e) : 0.f;
  }
}

// Eight values times 2^ex into a split row from element j (a multiple of 8).
__device__ __forceinline__ void store_chunk(const float (&f)[8], uint8_t* __restrict__ dst, int j,
                                            int ex = 0) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint16_t h0, l0, h1, l1;
    split_f16(ldexpf(f[2 * e], ex), h0, l0);
    split_f16(ldexpf(f[2 * e + 1], ex), h1, l1);
    h[e] = h0 | ((uint32_t)h1 << 16);
    l[e] = l0 | ((uint32_t)l1 << 16);
  }
  uint8_t* d = dst + split_at(j);
  *(u32x4*)d = u32x4{h[0], h[1], h[2], h[3]};
  *(u32x4*)(d + 64) = u32x4{l[0], l[1], l[2], l[3]};
}

}  // namespace
}  // namespace moe
