// MFMA tile pipeline of the products beside the layer (grouped products,
// Newton-Schulz products): one (BM x BN) tile of C = A B^T per block at a
// time, eight wavefronts (4 x 2), k-steps landing in a two-slot LDS ring by
// direct-to-LDS loads while the other slot is multiplied.
//
// An operand is read in one of two layouts:
//   row layout     its rows are contiguous along the contraction; a k-step is
//                  BM rows of 128 bytes.
//   column layout  its rows run along the contraction (a transposed operand in
//                  its stored order); a k-step is 64 rows of BM columns, and
//                  MFMA fragments come from transposing LDS reads.
// and in one of two precisions:
//   single  bfloat16, 64 contraction indices per k-step.
//   split   a float32 value v as two float16, hi = f16(v), lo = f16(v - hi):
//           22 bits of v survive (|v - hi - lo| <= 2^-24 |v| while lo is a
//           normal float16), and hi hi' + hi lo' + lo hi' leaves out only lo
//           lo' <= 2^-24 |v v'|.  Three float16 products at the full matrix
//           rate thus give float32 accuracy at a third of it, against a
//           sixteenth for the float32 matrix instructions.  Values are scaled
//           by powers of two beforehand so that neither part leaves the
//           float16 range.  Stored per row in units of 128 bytes: 32 hi, then
//           the 32 lo of the same indices; a k-step is one unit of each row
//           (32 contraction indices), so both precisions load alike, and the
//           two halves of a unit are read from LDS once for three products.
#pragma once

#include "lds_dma.h"
#include "moe_internal.h"

namespace moe {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef short tg_v4s __attribute__((ext_vector_type(4)));

constexpr int kTgThreads = 512;

// FM x FN fragments of 32 x 32 per wavefront; ACOL / BCOL: operand in column
// layout; SWAP: B as the MFMA's first operand, so that a lane holds four
// consecutive columns of one row instead of four consecutive rows of one
// column.
template <int FM_, int FN_, bool ACOL_, bool BCOL_, bool SPLIT_, bool SWAP_>
struct TgConfig {
  static constexpr int FM = FM_, FN = FN_, BM = FM_ * 128, BN = FN_ * 64;
  static constexpr bool ACOL = ACOL_, BCOL = BCOL_, SPLIT = SPLIT_, SWAP = SWAP_;
  static constexpr int KS = SPLIT ? 32 : 64;          // contraction indices per k-step
  static constexpr int SLOT = (BM + BN) * 128;        // bytes of a ring slot
  static constexpr int NI = BM / 32;                  // loads per wavefront per k-step
  static_assert(BM == BN, "wavefronts 0-3 load A, 4-7 load B, NI loads each");
};

// One operand of a tile.  Row layout: `rows` rows of `pitch` bytes, k-step s at
// byte 128 s of each.  Column layout: `rows` contraction rows of `pitch` bytes
// (later ones read as zeros), `width` columns (a multiple of 8).  All-int
// members beside the pointer: bools would be copied through memory.
struct TgOperand {
  const uint8_t* p;
  uint32_t pitch;
  int rows, width;
};

// Loading state of one wavefront for a tile.
struct TgLoad {
  const uint8_t* base;
  uint32_t step;   // bytes from one k-step to the next
  int rows;        // column layout: contraction rows; row layout: -1
  uint32_t pitch;
};

// Position of the 16-byte chunk `c` of contraction row k in a column-layout
// tile of W columns.  A transposing read of 32 lanes touches 64 bytes of each of
// four consecutive rows: rotating by four chunks per row puts them on distinct
// banks.
template <int W>
__device__ __forceinline__ int tg_col_offset(int k, int n) {
  return k * (W * 2) + (((n >> 3) ^ ((k & 3) << 2)) << 4) + (n & 7) * 2;
}

template <class C, bool COL>
__device__ __forceinline__ TgLoad tg_prepare_side(const TgOperand& o, int t0, int w, int lane,
                                                  uint32_t (&off)[C::NI]) {
  constexpr int W = C::BM;
  TgLoad l;
  l.pitch = uni((int)o.pitch);
  if constexpr (COL) {
    constexpr int RPI = 1024 / (2 * W);  // contraction rows per load instruction
    constexpr int CPR = W / 8;           // chunks per row
    l.base = uni(o.p);
    l.step = l.pitch * C::KS;
    l.rows = uni(o.rows);
#pragma unroll
    for (int i = 0; i < C::NI; ++i) {
      const int k = (w * C::NI + i) * RPI + lane / CPR;  // LDS row 0..63
      const int c = (lane % CPR) ^ ((k & 3) << 2);
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
    l.rows = -1;
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

// This wavefront's loads of a tile at (m0, n0): wavefronts 0-3 A, 4-7 B.
template <class C>
__device__ __forceinline__ TgLoad tg_prepare(const TgOperand& A, const TgOperand& B, int m0, int n0,
                                             int wave, int lane, uint32_t (&off)[C::NI]) {
  if (wave < 4) return tg_prepare_side<C, C::ACOL>(A, m0, wave, lane, off);
  return tg_prepare_side<C, C::BCOL>(B, n0, wave - 4, lane, off);
}

// Bytes from the k-step's base that its loads may touch; later ones read zeros.
template <class C>
__device__ __forceinline__ int tg_range(const TgLoad& l, int s) {
  if (l.rows < 0) return 0x7fffffff;
  return min(max(l.rows - C::KS * s, 0), C::KS) * (int)l.pitch;
}

__device__ __forceinline__ uint2 tg_read_tr(const uint8_t* p) {
  const tg_v4s v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) tg_v4s*)(__attribute__((address_space(3))) const uint8_t*)p);
  return __builtin_bit_cast(uint2, v);
}

// Fragment of k-group kg (16 indices), 32 rows (columns) from `at`: lane l
// holds row l % 32, indices 8 (l / 32) .. of the group.  Transposing reads:
// within each 16-lane group lane l names contraction row (l % 16) / 4 (+ 4 for
// the upper four) at column 16 ((l / 16) % 2) + 4 (l % 4).
template <int W, bool COL>
__device__ __forceinline__ u32x4 tg_frag(const uint8_t* rd, int kg, int at, int lane) {
  if constexpr (COL) {
    const int k = kg * 16 + 8 * (lane >> 5) + ((lane & 15) >> 2);
    const int n = at + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    const uint2 lo = tg_read_tr(rd + tg_col_offset<W>(k, n));
    const uint2 hi = tg_read_tr(rd + tg_col_offset<W>(k + 4, n));
    return u32x4{lo.x, lo.y, hi.x, hi.y};
  } else {
    return *(const u32x4*)(rd + lds_chunk_offset(at + (lane & 31), kg * 2 + (lane >> 5)));
  }
}

template <class C>
__device__ __forceinline__ void tg_frags_a(const uint8_t* __restrict__ rd, int kg, int wm, int lane,
                                           u32x4 (&f)[C::FM]) {
#pragma unroll
  for (int i = 0; i < C::FM; ++i) f[i] = tg_frag<C::BM, C::ACOL>(rd, kg, (wm * C::FM + i) * 32, lane);
}
template <class C>
__device__ __forceinline__ void tg_frags_b(const uint8_t* __restrict__ rd, int kg, int wn, int lane,
                                           u32x4 (&f)[C::FN]) {
#pragma unroll
  for (int i = 0; i < C::FN; ++i)
    f[i] = tg_frag<C::BN, C::BCOL>(rd + C::BM * 128, kg, (wn * C::FN + i) * 32, lane);
}

template <class C>
__device__ __forceinline__ void tg_products(const u32x4 (&a)[C::FM], const u32x4 (&b)[C::FN],
                                            f32x16 (&acc)[C::FM][C::FN]) {
#pragma unroll
  for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < C::FN; ++fn) {
      const u32x4 x = C::SWAP ? b[fn] : a[fm], y = C::SWAP ? a[fm] : b[fn];
      if constexpr (C::SPLIT)
        acc[fm][fn] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            __builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), acc[fm][fn], 0, 0, 0);
      else
        acc[fm][fn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), acc[fm][fn], 0, 0, 0);
    }
}

// Order of one group of FM * FN MFMAs with NR LDS reads and ND loads spread over it.
template <int MF, int NR, int ND>
__device__ __forceinline__ void tg_order() {
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
    for (int r = m * NR / MF; r < (m + 1) * NR / MF; ++r)
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
    for (int r = m * ND / MF; r < (m + 1) * ND / MF; ++r)
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
  }
}

// One k-step out of ring slot `rd`, the next one's loads (`db` + off into `wr`,
// range `nrec`: 0 reads zeros without touching memory) issued under its first
// MFMAs, every fragment read one group ahead of its use.
template <class C>
__device__ __forceinline__ void tg_step(const uint8_t* __restrict__ rd, int wm, int wn, int lane,
                                        f32x16 (&acc)[C::FM][C::FN], const uint8_t* db,
                                        const uint32_t (&off)[C::NI], uint8_t* __restrict__ wr,
                                        int nrec) {
  constexpr int MF = C::FM * C::FN, HALF = C::NI / 2;
  constexpr int RA = C::FM * (C::ACOL ? 2 : 1), RB = C::FN * (C::BCOL ? 2 : 1);
  if constexpr (C::SPLIT) {
    // per 16 indices: hi hi', hi lo', lo hi'
    u32x4 ah[2][C::FM], bh[2][C::FN], al[2][C::FM], bl[2][C::FN];
    tg_frags_a<C>(rd, 0, wm, lane, ah[0]);
    tg_frags_b<C>(rd, 0, wn, lane, bh[0]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = h * HALF; i < (h + 1) * HALF; ++i) dma16(db, off[i], wr + i * 1024, nrec);
      tg_frags_b<C>(rd, 2 + h, wn, lane, bl[h]);
      tg_products<C>(ah[h], bh[h], acc);
      tg_frags_a<C>(rd, 2 + h, wm, lane, al[h]);
      tg_products<C>(ah[h], bl[h], acc);
      if (h == 0) {
        tg_frags_a<C>(rd, 1, wm, lane, ah[1]);
        tg_frags_b<C>(rd, 1, wn, lane, bh[1]);
      }
      tg_products<C>(al[h], bh[h], acc);
    }
    __builtin_amdgcn_sched_group_barrier(0x100, RA + RB, 0);
    tg_order<MF, RB, HALF>();
    tg_order<MF, RA, 0>();
    tg_order<MF, RA + RB, 0>();
    tg_order<MF, RB, HALF>();
    tg_order<MF, RA, 0>();
    tg_order<MF, 0, 0>();
  } else {
    u32x4 a[2][C::FM], b[2][C::FN];
    tg_frags_a<C>(rd, 0, wm, lane, a[0]);
    tg_frags_b<C>(rd, 0, wn, lane, b[0]);
#pragma unroll
    for (int kg = 0; kg < 4; ++kg) {
      if (kg < 2) {
#pragma unroll
        for (int i = kg * HALF; i < (kg + 1) * HALF; ++i) dma16(db, off[i], wr + i * 1024, nrec);
      }
      if (kg < 3) {
        tg_frags_a<C>(rd, kg + 1, wm, lane, a[(kg + 1) & 1]);
        tg_frags_b<C>(rd, kg + 1, wn, lane, b[(kg + 1) & 1]);
      }
      tg_products<C>(a[kg & 1], b[kg & 1], acc);
    }
    __builtin_amdgcn_sched_group_barrier(0x100, RA + RB, 0);
    tg_order<MF, RA + RB, HALF>();
    tg_order<MF, RA + RB, HALF>();
    tg_order<MF, RA + RB, 0>();
    tg_order<MF, 0, 0>();
  }
}

// Row and column (inside the tile) of accumulator register r of fragment (fm, fn).
template <class C>
__device__ __forceinline__ int tg_row(int wm, int fm, int lane, int r) {
  return (wm * C::FM + fm) * 32 + (C::SWAP ? (lane & 31) : 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3));
}
template <class C>
__device__ __forceinline__ int tg_col(int wn, int fn, int lane, int r) {
  return (wn * C::FN + fn) * 32 + (C::SWAP ? 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3) : (lane & 31));
}

// The persistent loop over the tiles start, start + stride, .. < end of problem P:
//   P::Tile        { TgOperand A, B; int m0, n0, steps; ... }
//   p.tile(L)      the L-th tile (wavefront-uniform)
//   p.store(t, wm, wn, lane, acc)   the epilogue, from registers
// After a tile's last k-step the next tile's first one is already loading
// while the tile is written out.
template <class C, class P>
__device__ __forceinline__ void tg_run(const P& p, int start, int end, int stride,
                                       uint8_t* __restrict__ lds0, uint8_t* __restrict__ lds1) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uni(tid >> 6), wm = wave >> 1, wn = wave & 1;
  if (start >= end) return;
  typename P::Tile cur = p.tile(start);
  uint32_t off[C::NI];
  TgLoad ld = tg_prepare<C>(cur.A, cur.B, cur.m0, cur.n0, wave, lane, off);
  int ph = 0;  // ring slot of the current tile's k-step 0
  {
    uint8_t* w = lds0 + wave * C::NI * 1024;
    const int nrec = cur.steps > 0 ? tg_range<C>(ld, 0) : 0;
#pragma unroll
    for (int i = 0; i < C::NI; ++i) dma16(ld.base, off[i], w + i * 1024, nrec);
  }
  for (int L = start;;) {
    const int Ln = L + stride;
    f32x16 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    typename P::Tile nxt = cur;
    if (cur.steps == 0) {
      // nothing to multiply: the wait lands the zero loads of this slot before the
      // next tile's first k-step is loaded into it
      pipe_sync();
      if (Ln < end) {
        nxt = p.tile(Ln);
        ld = tg_prepare<C>(nxt.A, nxt.B, nxt.m0, nxt.n0, wave, lane, off);
        uint8_t* w = ((ph & 1) ? lds1 : lds0) + wave * C::NI * 1024;
        const int nrec = nxt.steps > 0 ? tg_range<C>(ld, 0) : 0;
#pragma unroll
        for (int i = 0; i < C::NI; ++i) dma16(ld.base, off[i], w + i * 1024, nrec);
      }
    }
    for (int s = 0; s < cur.steps; ++s) {
      pipe_sync();  // k-step s has landed; every wavefront is done with the other slot
      const int q = (ph + s) & 1;
      const uint8_t* rd = q ? lds1 : lds0;
      uint8_t* wr = (q ? lds0 : lds1) + wave * C::NI * 1024;
      const uint8_t* db = ld.base + (size_t)(s + 1) * ld.step;
      int nrec = tg_range<C>(ld, s + 1);
      if (s + 1 == cur.steps) {
        nrec = 0;
        db = ld.base;
        if (Ln < end) {
          nxt = p.tile(Ln);
          ld = tg_prepare<C>(nxt.A, nxt.B, nxt.m0, nxt.n0, wave, lane, off);
          db = ld.base;
          if (nxt.steps > 0) nrec = tg_range<C>(ld, 0);
        }
      }
      tg_step<C>(rd, wm, wn, lane, acc, uni(db), off, wr, uni(nrec));
    }
    p.store(cur, wm, wn, lane, acc);
    ph += cur.steps;
    if (Ln >= end) break;
    L = Ln;
    cur = nxt;
  }
  MOE_WAIT_VMCNT(0);  // no direct-to-LDS load outlives the block
}

// The tiles [start, end) and stride of this block: the blocks are dealt to the
// eight XCDs round-robin, and each XCD takes a contiguous range, whose
// neighbouring tiles share operands in its L2.
struct TgShare {
  int start, end, stride;
};
__device__ __forceinline__ TgShare tg_share(int total) {
  const int g = gridDim.x, X = min(8, g), x = blockIdx.x % X;
  TgShare s;
  s.end = (int)((long long)total * (x + 1) / X);
  s.start = (int)((long long)total * x / X) + blockIdx.x / X;
  s.stride = (g - x + X - 1) / X;
  return s;
}

// v * 2^e as two float16.
__device__ __forceinline__ void split_f16(float v, uint16_t& hi, uint16_t& lo) {
  const _Float16 h = (_Float16)v;
  const _Float16 l = (_Float16)(v - (float)h);
  hi = __builtin_bit_cast(uint16_t, h);
  lo = __builtin_bit_cast(uint16_t, l);
}
__device__ __forceinline__ float f16_to_f32(uint16_t b) {
  return (float)__builtin_bit_cast(_Float16, b);
}

// Bytes of a split row of n values, and the place of element j's hi in it (its lo
// is 64 bytes further).
__host__ __device__ inline long long split_pitch(int n) { return (long long)((n + 31) / 32) * 128; }
__device__ __forceinline__ long long split_at(int j) { return (long long)(j >> 5) * 128 + (j & 31) * 2; }

}  // namespace
}  // namespace moe
