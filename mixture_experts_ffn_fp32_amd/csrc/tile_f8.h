// MFMA tile pipeline of products of 8-bit operands with a float32 scale for each block of 128
// (gfx950): one (BM x BN) tile of C = X W per block at a time, in the shapes, LDS rings and
// tile order of tile_gemm.h.  A k-step is 128 contraction indices, which are 128 bytes of a row
// as the k-steps there are, and one block of scales:
//
//   acc += xs[row] ws[column block] (sum over the k-step of x w)
//
// The k-step's sum comes from the matrix instructions in registers of its own (a pair of
// 32x32x64, the second one on top of the first) and is added to acc by 16 multiply-adds per
// fragment while the next pair runs: 64 of its 128 cycles.  acc therefore has to lie in registers
// that the vector ALU reaches, which bounds a wavefront's tile to 64 x 128.
//
// Measured, a k-step of a 256^2 tile: 1.87 us (2300 TFLOP/s over 256 CUs, 88% of a library product
// without scales).  With its multiply-adds, loads or LDS reads left out it takes 1.67, 1.36 or 1.44
// us: no one of them alone bounds it.  A tile's start and results add 2 us to its k-steps where
// k-steps are few; the wait for its stores is what is left of that.
//
// x is read in row layout (rows contiguous along the contraction).  w is read in row layout
// (forward: its rows run along k) or in column layout (input gradient: its rows are the
// contraction's), where a k-step is 128 rows of BN bytes and fragments come from transposing
// LDS reads.  The scales ride in the ring beside their k-step, one float per row and column.
#pragma once

#include "f8.h"
#include "tile_gemm.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// Q: x's type (w is e4m3); WCOL: w in column layout; EXACT: through bfloat16 (see
// grouped_f8.hip); ODD: rows start at any byte (TgSmall).
template <class Shape, bool WCOL_, int Q_, bool EXACT_, bool ODD_ = false>
struct F8Config : Shape {
  static constexpr bool WCOL = WCOL_, EXACT = EXACT_, SWAP = true, ODD = ODD_;
  static constexpr int Q = Q_;
  static constexpr bool SMALL = Shape::BM == TgSmall::BM;
  static constexpr int DATA = Shape::SLOT;                       // bytes of x and w in a slot,
  static constexpr int SLOT = DATA + 4 * (Shape::BM + Shape::BN);  // and of their scales
  static constexpr int LDS = Shape::S * SLOT * (SMALL ? TgSmall::WAVES : 1);
  static constexpr int WAVES_PER_SIMD = Shape::BPC * Shape::THREADS / 256;
  // Loads of a k-step per wavefront (its data and 64 scales), and how many of them follow the
  // barrier that frees their slot at once (f8_step).
  static constexpr int LOADS = Shape::NI + 1, FIRST = Shape::NI / 2 - 1;
  // Places of a wavefront's fragments of w among the tile's fragments of 32 columns: the f-th
  // is column(f) + first(wn).  With four of them, two neighbours each: 128 bytes of a row of
  // bfloat16 results, a whole line, lie in one wavefront.  With two they interleave, so that the
  // wavefronts stay balanced where the matrix ends after half a tile's columns.
  static constexpr bool PAIRS = Shape::FN == 4;
  // Whether a round of few tiles is cut (F8Units), and half a tile's and a quarter's time then,
  // percent of a tile's.  128^2 are not: two of them share a CU, and one alone there is as fast as
  // its halves (4096 rows, 2048 -> 2560 x 2048, one round and a quarter, 54 us, cut 60).
  static constexpr bool CUT = PAIRS;
  static constexpr int HALF = 65, QUARTER = 50;
  static __host__ __device__ constexpr int column(int f) {
    return PAIRS ? 2 * Shape::WN * (f >> 1) + (f & 1) : Shape::WN * f;
  }
  static __host__ __device__ constexpr int first(int wn) { return PAIRS ? 2 * wn : wn; }
};

// A tile's operands.  Row layout: `rows` rows of `pitch` bytes, of which the first `length` are
// the contraction.  Column layout: `rows` contraction rows of `pitch` bytes, `width` columns (a
// multiple of 16 up to pitch).  Scales: those of row r (column c: c / 128) and k-step s lie at
// r * s_row + s * s_step (floats).
struct F8Operand {
  const uint8_t* p;
  const float* s;
  uint32_t pitch, s_row, s_step;
  int rows, width;
};

// Loading state of one wavefront: its data loads (16 bytes a lane) and its load of 64 scales.
// Load i of a k-step starts i * i_step bytes behind the first one; the lanes' offsets repeat
// every second load.
struct F8Load {
  const uint8_t *base, *scales;
  uint32_t step, s_step, i_step;  // bytes from one k-step to the next, from one load to the next
  int rows;                // column layout: contraction rows; row layout: -(k-steps)
  uint32_t pitch;
  int range;               // row layout: bytes from base to the end of the tile's rows
  int tail;                // row layout: bytes of the last k-step that exist
};

// One direct-to-LDS load of 4 bytes per lane (dma16 otherwise).
__device__ __forceinline__ void dma4(const uint8_t* base, uint32_t off, uint8_t* __restrict__ wr,
                                     int nrec) {
  const __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, nrec, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)wr, 4, off,
                                           0, 0, 0);
}

// Column layout: the 16-byte chunk c of contraction row k lies at position c ^ f8_rotation(k),
// so that a transposing read of 32 lanes (two neighbouring chunks of eight consecutive rows)
// touches every bank once.  It depends on the row's place among eight alone.
template <int W>
__device__ __forceinline__ int f8_rotation(int k) {
  return 2 * (W == 256 ? k & 7 : W == 128 ? (k >> 1) & 3 : (k >> 2) & 1);
}
// Row layout: the byte of a row's k-step that load i of this lane takes (of the rows 8 i ..).
__device__ __forceinline__ int f8_chunk_byte(int i, int lane) {
  return ((lane & 7) ^ ((4 * i + (lane >> 4)) & 7)) << 4;
}

// Loads of wavefront w (of those on this side) of the tile's side at t0; `blocks`: the scales
// are those of blocks of 128 rows (w), else of rows (x).
template <class C, bool COL>
__device__ __forceinline__ F8Load f8_prepare(const F8Operand& o, bool blocks, int t0, int steps,
                                             int length, int w, int lane, uint32_t (&off)[2],
                                             uint32_t& s_off) {
  constexpr int W = C::BM;
  F8Load l;
  l.pitch = uni((int)o.pitch);
  l.s_step = uni((int)o.s_step) * 4;
  if constexpr (COL) {
    constexpr int RPI = 1024 / W, CPR = W / 16;  // rows per load instruction, chunks per row
    l.base = uni(o.p);
    l.step = l.pitch * kF8Block;
    l.i_step = l.pitch * RPI;
    l.rows = uni(o.rows);
    l.range = l.tail = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = lane / CPR;
      // columns past the last one reread the last chunk (never stored)
      off[i] = (uint32_t)(w * C::NI * RPI + k) * l.pitch +
               min(t0 + 16 * ((lane % CPR) ^ f8_rotation<W>(k + i * RPI)), o.width - 16);
    }
    l.scales = uni((const uint8_t*)o.s);
    s_off = 4 * o.s_row * (uint32_t)(min(t0 + 64 * w + lane, o.width - 1) / kF8Block);
  } else {
    // rows past the last one lie outside the range: they read zeros
    const int r0 = t0 + w * C::NI * 8, rows = min(max(o.rows - r0, 0), C::NI * 8);
    l.base = uni(o.p + (size_t)min(r0, o.rows - 1) * o.pitch);
    l.step = kF8Block;
    l.i_step = l.pitch * 8;
    l.rows = -uni(steps);
    l.range = uni(rows) * (int)l.pitch;
    l.tail = uni(length - (steps - 1) * kF8Block);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      off[i] = (uint32_t)(lane >> 3) * l.pitch + f8_chunk_byte(i, lane);
    const int first = min(t0, o.rows - 1), r = min(t0 + 64 * w + lane, o.rows - 1);
    l.scales = uni((const uint8_t*)(o.s + (blocks ? 0 : (size_t)first * o.s_row)));
    s_off = 4 * o.s_row * (uint32_t)(blocks ? r / kF8Block : r - first);
  }
  return l;
}

// Bytes from the k-step's base that its loads may touch; later ones read zeros.
__device__ __forceinline__ int f8_range(const F8Load& l, int s) {
  if (l.rows < 0) return s < -l.rows ? max(l.range - kF8Block * s, 0) : 0;
  return min(max(l.rows - kF8Block * s, 0), kF8Block) * (int)l.pitch;
}
// A k-step that is being loaded: where its data and scales come from, uniform.
struct F8Source {
  const uint8_t *data, *scales;
  int range, s_range;
};
__device__ __forceinline__ F8Source f8_source(const F8Load& l, int s, bool on) {
  F8Source f;
  f.data = uni(l.base + (size_t)s * l.step);
  f.scales = uni(l.scales + (size_t)s * l.s_step);
  f.range = uni(on ? f8_range(l, s) : 0);
  f.s_range = uni(on ? 0x7fffffff : 0);
  return f;
}
// Load i of it (the last one the scales) of wavefront `part` into ring slot `wr`.
template <class C>
__device__ __forceinline__ void f8_load(const F8Source& f, const F8Load& l, int i,
                                        const uint32_t (&off)[2], uint32_t s_off,
                                        uint8_t* __restrict__ wr, int part) {
  if (i == C::NI)
    dma4(f.scales, s_off, wr + C::DATA + part * 256, f.s_range);
  else
    dma16(f.data + (size_t)i * l.i_step, off[i & 1], wr + (part * C::NI + i) * 1024,
          max(f.range - i * (int)l.i_step, 0));
}

// The last k-step of a row ends with the row: chunks behind it read zeros (their offset lies
// outside every range).  Only k-steps of zeros follow it.
__device__ __forceinline__ void f8_mask_tail(const F8Load& l, int s, int lane, uint32_t (&off)[2]) {
  if (l.rows < 0 && s == -l.rows - 1 && l.tail < kF8Block) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (f8_chunk_byte(i, lane) >= l.tail) off[i] = 0x7fffffffu;
  }
}

// A k-step of 32 rows (columns) of a tile: lane l holds row l % 32, in half h (64 indices)
// indices 64 h + 16 (l / 32) + 0 .. 15 and the same 32 further on.
struct F8Frag {
  i32x8 h[2];
};
// A lane's place in the first of its wavefront's fragments (fragment WN f + u is the f-th).  Row
// layout: its chunk 16 (l / 32); the other chunks are that xor 32 (the other 16 bytes of half 0),
// 64 and 96.  Column layout: its column of contraction row 16 (l / 32) + (l % 16) / 2; a
// fragment u places further on is that xor 32 u, as a fragment's columns are 32 bytes of the row.
template <int W, bool COL>
__device__ __forceinline__ int f8_place(int u, int lane) {
  if constexpr (COL) {
    const int l16 = lane & 15, k = 16 * (lane >> 5) + (l16 >> 1);
    return k * W + ((2 * u + ((lane >> 4) & 1)) ^ f8_rotation<W>(k)) * 16 + 8 * (l16 & 1);
  } else {
    return lds_chunk_offset(u * 32 + (lane & 31), lane >> 5);
  }
}
// The fragment of the operand at rd that lies u places behind the wavefront's first one.
template <int W, bool COL>
__device__ __forceinline__ F8Frag f8_frag(const uint8_t* rd, int place, int u) {
  // (opaque: the few operations that make the addresses are repeated for every fragment, as
  // kept addresses would push sums out of the registers)
  asm volatile("" : "+v"(place));
  F8Frag v;
  if constexpr (COL) {
    const uint8_t* p = rd + (place ^ (32 * u));
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // rows + 0, 8, 32, 40 of each half
      const uint8_t* from = p + (8 * (j & 1) + 32 * (j >> 1)) * W;
      const i32x2 t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (__attribute__((address_space(3))) i32x2*)(__attribute__((address_space(3)))
                                                     const uint8_t*)from);
      v.h[j >> 2][2 * (j & 3)] = t[0];
      v.h[j >> 2][2 * (j & 3) + 1] = t[1];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4 c = *(const u32x4*)(rd + (place ^ (32 * j)) + u * 32 * 128);
#pragma unroll
      for (int e = 0; e < 4; ++e) v.h[j >> 1][4 * (j & 1) + e] = (int)c[e];
    }
  }
  return v;
}
// Both places of a wavefront.
struct F8Places {
  int x, w;
};
template <class C>
__device__ __forceinline__ F8Places f8_places(int wm, int wn, int lane) {
  return F8Places{f8_place<C::BM, false>(wm, lane),
                  C::BM * 128 + f8_place<C::BN, C::WCOL>(C::first(wn), lane)};
}
template <class C>
__device__ __forceinline__ F8Frag f8_frag_x(const uint8_t* rd, const F8Places& at, int fm) {
  return f8_frag<C::BM, false>(rd, at.x, C::WM * fm);
}
template <class C>
__device__ __forceinline__ F8Frag f8_frag_w(const uint8_t* rd, const F8Places& at, int fn) {
  return f8_frag<C::BN, C::WCOL>(rd, at.w, C::column(fn));
}

// Eight 8-bit values (two words) as bfloat16, which is exact.
template <int Q>
__device__ __forceinline__ bf16x8 f8_widen(int lo, int hi) {
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int w = i < 2 ? lo : hi;
    bf16x2 two;
    if constexpr (Q == F8_E4M3)
      two = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true)
                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false);
    else
      two = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.f, true)
                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.f, false);
    v[2 * i] = two[0];
    v[2 * i + 1] = two[1];
  }
  return v;
}

// The sum of a k-step's products: a lane holds 16 columns (w's) of one row (x's).
template <class C>
__device__ __forceinline__ f32x16 f8_products(const F8Frag& w, const F8Frag& x) {
  f32x16 part;
#pragma unroll
  for (int r = 0; r < 16; ++r) part[r] = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (C::EXACT) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        part = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            f8_widen<F8_E4M3>(w.h[h][2 * i], w.h[h][2 * i + 1]),
            f8_widen<C::Q>(x.h[h][2 * i], x.h[h][2 * i + 1]), part, 0, 0, 0);
    } else {
      part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          w.h[h], x.h[h], part, 0, C::Q == F8_E5M2 ? 1 : 0, 0, 0, 0, 0);
    }
  }
  return part;
}
__device__ __forceinline__ void f8_add(f32x16& acc, const f32x16& part, float scale) {
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = fmaf(part[r], scale, acc[r]);
  // (here and not later: the compiler would sink the additions and keep every pair's sum)
  asm volatile("" : "+v"(acc));
}

// A k-step's scales as a wavefront needs them: of its rows, one a lane, and of the tile's
// blocks of 128 columns.
template <class C>
struct F8Scales {
  static constexpr int NB = C::BN > kF8Block ? C::BN / kF8Block : 1;
  float x[C::FM], w[NB];
};
template <class C>
__device__ __forceinline__ F8Scales<C> f8_scales(const uint8_t* rd, int wm, int lane) {
  const float* s = (const float*)(rd + C::DATA);
  F8Scales<C> v;
#pragma unroll
  for (int i = 0; i < C::FM; ++i) v.x[i] = s[(C::WM * i + wm) * 32 + (lane & 31)];
#pragma unroll
  for (int j = 0; j < F8Scales<C>::NB; ++j)
    v.w[j] = __uint_as_float(uni((int)__float_as_uint(s[C::BM + j * kF8Block])));
  return v;
}
template <class C>
__device__ __forceinline__ float f8_scale_of(const F8Scales<C>& s, int fm, int fn) {
  return s.x[fm] * s.w[C::column(fn) * 32 / kF8Block];
}

// 16-byte chunks of four neighbouring lanes transposed: lane j of four holds chunks (j, 0 .. 3) and
// receives (0 .. 3, j).
__device__ __forceinline__ void f8_quad_transpose(u32x4 (&c)[4], int lane) {
  const bool odd = lane & 1, up = lane & 2;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {  // with lane ^ 1
      const uint32_t t = __builtin_amdgcn_mov_dpp(odd ? c[i][e] : c[i + 1][e], 0xB1, 0xf, 0xf, true);
      c[i][e] = odd ? t : c[i][e];
      c[i + 1][e] = odd ? c[i + 1][e] : t;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // with lane ^ 2
      const uint32_t t = __builtin_amdgcn_mov_dpp(up ? c[i][e] : c[i + 2][e], 0x4E, 0xf, 0xf, true);
      c[i][e] = up ? t : c[i][e];
      c[i + 2][e] = up ? c[i + 2][e] : t;
    }
  }
}

// What passes from one k-step to the next: x's fragments and w's first one, and the last pair's
// sum, which is added behind the next pair's start.
template <class C>
struct F8State {
  F8Frag x[C::FM], w[2];
  f32x16 part;
  float scale;
};

// One k-step out of ring slot `rd`.  The barrier stands before the last of w's fragments, when
// every read of `rd` has been made: `rd` is free, the next k-step (slot `nx`) has landed, and
// the last fragment's products cover the reads of the next k-step's first ones, each into the
// registers that its last use has freed.
//
// The loads of the k-step after the next one go into `rd`: C::FIRST of them behind the barrier,
// the others in the next call, each behind an MFMA.  (All of them behind the barrier they held
// the wavefronts up: a load takes the address path 16 cycles, 72 of them of eight wavefronts
// 1150, half a k-step, and a wavefront whose load waits issues no MFMA.)  load(i, slot) issues the
// i-th load, advance() passes to the next k-step.  wr_rd and wr_nx are rd and nx again: with
// the loads and the reads in separate restrict scopes the compiler does not make every fragment
// read wait for the loads in flight, and the barrier's fences keep their order.
template <class C, int FMA, int FNA, class Advance>
__device__ __forceinline__ void f8_step(const uint8_t* __restrict__ rd,
                                        const uint8_t* __restrict__ nx, uint8_t* __restrict__ wr_rd,
                                        uint8_t* __restrict__ wr_nx, const F8Places& at, int wm,
                                        int lane, int wave, F8State<C>& f,
                                        f32x16 (&acc)[C::FM][C::FN], const F8Source& from,
                                        const F8Load& ld, const uint32_t (&off)[2],
                                        const uint32_t& s_off, Advance advance) {
  constexpr int REST = C::LOADS - C::FIRST;         // of the k-step in `nx`
  constexpr int SPREAD = FNA > 2 ? FNA - 2 : 1;     // over so many groups of products
  const F8Scales<C> s = f8_scales<C>(rd, wm, lane);
  // the products of fragments (fm, fn), and the pair's before them added
  auto pair = [&](int fn, int fm) {
    const f32x16 part = f8_products<C>(f.w[fn & 1], f.x[fm]);
    const int pm = fm > 0 ? fm - 1 : FMA - 1, pn = fm > 0 ? fn : fn > 0 ? fn - 1 : FNA - 1;
    f8_add(acc[pm][pn], f.part, f.scale);
    f.part = part;
    f.scale = f8_scale_of<C>(s, fm, fn);
  };
  // (the last group apart: in one loop the reads of rd and of nx would be merged, and lose
  // their scopes)
#pragma unroll
  for (int fn = 0; fn + 1 < FNA; ++fn) {
    f.w[(fn + 1) & 1] = f8_frag_w<C>(rd, at, fn + 1);
    const int l0 = C::FIRST + (fn < SPREAD ? fn * REST / SPREAD : REST);
    const int l1 = C::FIRST + (fn < SPREAD ? (fn + 1) * REST / SPREAD : REST);
#pragma unroll
    for (int fm = 0; fm < FMA; ++fm) {
#pragma unroll
      for (int i = l0 + fm * (l1 - l0) / FMA; i < l0 + (fm + 1) * (l1 - l0) / FMA; ++i)
        f8_load<C>(from, ld, i, off, s_off, wr_nx, wave);
      pair(fn, fm);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (fn + 1 == SPREAD) advance();
  }
  if (FNA == 1) {
#pragma unroll
    for (int i = C::FIRST; i < C::LOADS; ++i) f8_load<C>(from, ld, i, off, s_off, wr_nx, wave);
    advance();
  }
  MOE_WAIT_VMCNT(0);
  lds_sync();
  if (FNA > 1) f.w[0] = f8_frag_w<C>(nx, at, 0);
#pragma unroll
  for (int fm = 0; fm < FMA; ++fm) {
#pragma unroll
    for (int i = fm * C::FIRST / FMA; i < (fm + 1) * C::FIRST / FMA; ++i)
      f8_load<C>(from, ld, i, off, s_off, wr_rd, wave);
    pair(FNA - 1, fm);
    f.x[fm] = f8_frag_x<C>(nx, at, fm);
    __builtin_amdgcn_sched_barrier(0);
  }
  if (FNA == 1) f.w[0] = f8_frag_w<C>(nx, at, 0);
}

// The loads of this wavefront: x in the first half of them, w in the other.
template <class C, class Tile>
__device__ __forceinline__ F8Load f8_prepare_wave(const Tile& t, int wave, int lane,
                                                  uint32_t (&off)[2], uint32_t& s_off) {
  constexpr int H = C::WM * C::WN / 2;
  if (wave < H) return f8_prepare<C, false>(t.X, false, t.m0, t.steps, t.length, wave, lane, off, s_off);
  return f8_prepare<C, C::WCOL>(t.W, true, t.n0, t.steps, t.length, wave - H, lane, off, s_off);
}

// A block's tiles: every P-th of its XCD's range (TgTiles; P: the XCD's blocks), and of the last
// round, if tiles are left for few of the blocks only, halves or quarters, so that more of them
// have some.  Measured at 4096 rows and 256^2 tiles, k = 2048 (8192): one round 39 (127) us; 16, 64
// or 128 tiles more in quarters, quarters and halves + 14, 15 and 20 (54, 61, 84) us, whole + 25
// (86 .. 92).
struct F8Unit {
  int tile, ways, part;  // tile -1: none
};
template <class C>
struct F8Units {
  int first, whole, rest, ways, blocks;
  __device__ __forceinline__ F8Units(const TgTiles& q) {
    const int n = q.count(q.x);
    first = q.at(q.x, 0);
    blocks = q.blocks(q.x);
    rest = n % blocks;
    whole = n - rest;
    ways = 1;
    if constexpr (C::CUT) {
      const int two = (2 * rest + blocks - 1) / blocks * C::HALF;
      const int four = (4 * rest + blocks - 1) / blocks * C::QUARTER;
      if (min(two, four) < 100) ways = four < two ? 4 : 2;
    }
  }
  __device__ __forceinline__ F8Unit at(int j) const {
    if (j < whole) return F8Unit{first + j, 1, 0};
    const int u = j - whole;
    if (u >= rest * ways) return F8Unit{-1, 1, 0};
    return F8Unit{first + whole + u / ways, ways, u % ways};
  }
};
// The tile's part: halves of its columns (of its rows, if it has half the columns only), quarters
// of both.  A part without rows or columns has no k-steps.
template <class C, class P>
__device__ __forceinline__ typename P::Tile f8_unit(const P& p, const F8Unit& u, int hint) {
  typename P::Tile t = p.tile(u.tile, hint);
  if (C::CUT && u.ways > 1) {
    constexpr int HM = C::BM / 2, HN = C::BN / 2;
    const bool m = u.ways == 4 || t.cols <= HN, n = u.ways == 4 || !m;
    if (m) {
      t.m0 += (u.part & 1) * HM;
      t.X.rows = min(t.X.rows, t.m0 + HM);
      t.rows = t.X.rows - t.m0;
    }
    if (n) {
      const int j = u.ways == 4 ? u.part >> 1 : u.part;
      t.n0 += j * HN;
      t.cols = min(t.cols - j * HN, HN);
      if (C::WCOL) t.W.width = min(t.W.width, t.n0 + HN);
      else t.W.rows = min(t.W.rows, t.n0 + HN);
    }
    if (t.rows <= 0 || t.cols <= 0) t.steps = 0;
  }
  return t;
}

// The loads' place in the stream of k-steps of a block's tiles (see TgCursor).
struct F8Cursor {
  int hint;
  int s, steps;      // the tile's next k-step, its k-steps (0: the stream has ended)
  int real;          // those that exist
  F8Source from;
};
// k-steps of a tile: two at least, so that the loads, which are a k-step ahead, pass to the next
// tile while this one is multiplied (k-steps of zeros follow the last one).
__device__ __forceinline__ int f8_steps(int steps) { return max(steps, 2); }

// The cursor to unit u (without a tile: the stream has ended).
template <class C, class P>
__device__ __forceinline__ void f8_seek(const P& p, const F8Unit& u, F8Cursor& c, F8Load& ld,
                                        uint32_t (&off)[2], uint32_t& s_off, int wave, int lane) {
  c.s = c.steps = c.real = 0;
  if (u.tile >= 0) {
    const typename P::Tile t = f8_unit<C>(p, u, c.hint);
    c.hint = uni(t.hint);
    c.real = uni(t.steps);
    c.steps = f8_steps(c.real);
    ld = f8_prepare_wave<C>(t, wave, lane, off, s_off);
  }
}
// Ready to load the cursor's k-step.
__device__ __forceinline__ void f8_ready(F8Cursor& c, const F8Load& ld, int lane,
                                         uint32_t (&off)[2]) {
  f8_mask_tail(ld, c.s, lane, off);
  c.from = f8_source(ld, c.s, c.s < c.real);
}

// The k-steps of a tile.  On entry the first one lies in slot ph, and C::FIRST loads of the
// second one have been issued; on return the same holds of the next tile (next()).
template <class C, int FMA, int FNA, class P, class Next>
__device__ __forceinline__ void f8_tile(const P& p, int steps, int& ph, int wave, int lane, Next next,
                                        F8Cursor& c, F8Load& ld, uint32_t (&off)[2],
                                        uint32_t& s_off, f32x16 (&acc)[C::FM][C::FN],
                                        uint8_t* __restrict__ lds) {
  static_assert(C::S == 2, "one k-step is multiplied, one is loaded");
  const int wm = wave / C::WN, wn = wave % C::WN;
  asm volatile("" : "+v"(lane));  // (see tg_tile)
  const int all = f8_steps(steps);
  const F8Places at = f8_places<C>(wm, wn, lane);
  F8State<C> f;
  const uint8_t* first = lds + ph * C::SLOT;
#pragma unroll
  for (int fm = 0; fm < FMA; ++fm) f.x[fm] = f8_frag_x<C>(first, at, fm);
  f.w[0] = f8_frag_w<C>(first, at, 0);
#pragma unroll
  for (int r = 0; r < 16; ++r) f.part[r] = 0.f;
  f.scale = 0.f;
  for (int s = 0; s < all; ++s) {
    const int after = ph ^ 1;
    f8_step<C, FMA, FNA>(
        lds + ph * C::SLOT, lds + after * C::SLOT, lds + ph * C::SLOT, lds + after * C::SLOT, at, wm,
        lane, wave, f, acc, c.from, ld, off, s_off,
        [&]() {
          c.s = uni(c.s + 1);
          if (c.s >= c.steps) f8_seek<C>(p, next(), c, ld, off, s_off, wave, lane);
          f8_ready(c, ld, lane, off);
        });
    ph = after;
  }
  f8_add(acc[FMA - 1][FNA - 1], f.part, f.scale);
}

// The persistent loop over a block's tiles of problem P (as tg_run):
//   P::Tile   { F8Operand X, W; int m0, n0, steps, length, rows, cols, hint; .. }
template <class C, class P>
__device__ __forceinline__ void f8_run(const P& p, int tiles, uint8_t* __restrict__ lds) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uni(tid >> 6), wm = wave / C::WN, wn = wave % C::WN;
  TgTiles q;
  q.init(tiles, nullptr);
  const F8Units<C> units(q);
  int mine = q.own;
  F8Unit u = units.at(mine);
  if (u.tile < 0) return;
  F8Cursor c{};
  F8Load ld{};
  uint32_t off[2] = {}, s_off = 0;
  f8_seek<C>(p, u, c, ld, off, s_off, wave, lane);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    f8_ready(c, ld, lane, off);
#pragma unroll
    for (int i = 0; i < (k == 0 ? C::LOADS : C::FIRST); ++i)
      f8_load<C>(c.from, ld, i, off, s_off, lds + k * C::SLOT, wave);
    if (k == 0) c.s = 1;
  }
  pipe_sync();
  int ph = 0;  // ring slot of the next k-step
  F8Unit u1{-1, 1, 0};
  auto next = [&]() -> F8Unit { return u1 = units.at(mine += units.blocks); };
  int hint = 0;
  while (true) {
    const typename P::Tile t = f8_unit<C>(p, u, hint);
    hint = t.hint;
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
    if (hm && hn) f8_tile<C, 1, H>(p, t.steps, ph, wave, lane, next, c, ld, off, s_off, acc, lds);
    else if (hm) f8_tile<C, 1, C::FN>(p, t.steps, ph, wave, lane, next, c, ld, off, s_off, acc, lds);
    else if (hn) f8_tile<C, 2, H>(p, t.steps, ph, wave, lane, next, c, ld, off, s_off, acc, lds);
    else f8_tile<C, 2, C::FN>(p, t.steps, ph, wave, lane, next, c, ld, off, s_off, acc, lds);
    // the loads in flight are waited for here: to the compiler they could be any slot's, and
    // every fragment read of the next tile's loop would wait for loads
    MOE_WAIT_VMCNT(0);
    p.store(t, wm, wn, lane, acc);
    if (u1.tile < 0) break;
    u = u1;
  }
}

// Rows of 16 bytes and more that start at any byte: load i of a k-step (f8_load) through
// registers.  A chunk that the row's end cuts is read as the row's last 16 bytes and shifted
// when it has landed (f8_odd_cut), so that no load waits for another.
typedef u32x4 u32x4_at1 __attribute__((aligned(1)));
struct F8Place {
  int row, byte, end;  // the row's bytes end at `end`
};
template <class C, bool COL>
__device__ __forceinline__ F8Place f8_odd_place(const F8Operand& o, int t0, int length, int s, int i,
                                                int lane) {
  if constexpr (COL) {
    constexpr int W = C::BM, CPR = W / 16;
    const int k = i * (1024 / W) + lane / CPR;
    return F8Place{s * kF8Block + k, t0 + 16 * ((lane % CPR) ^ f8_rotation<W>(k)), o.width};
  } else {
    return F8Place{t0 + 8 * i + (lane >> 3), s * kF8Block + f8_chunk_byte(i & 1, lane), length};
  }
}
template <class C, bool COL>
__device__ __forceinline__ u32x4 f8_odd_load(const F8Operand& o, int t0, int length, int s, int i,
                                             int lane) {
  const F8Place at = f8_odd_place<C, COL>(o, t0, length, s, i, lane);
  return *(const u32x4_at1*)(o.p + (size_t)min(at.row, o.rows - 1) * o.pitch +
                             min(at.byte, at.end - 16));
}
template <class C, bool COL>
__device__ __forceinline__ u32x4 f8_odd_cut(u32x4 v, const F8Operand& o, int t0, int length, int s,
                                            int i, int lane) {
  const F8Place at = f8_odd_place<C, COL>(o, t0, length, s, i, lane);
  const int valid = at.row < o.rows ? min(max(at.end - at.byte, 0), 16) : 0;
  const int shift = 8 * (16 - valid);  // bits
  uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
  if (shift >= 64) {
    lo = hi;
    hi = 0;
  }
  const int b = shift & 63;
  lo = lo >> b | (b > 0 ? hi << (64 - b) : 0);
  hi >>= b;
  if (shift >= 128) lo = 0;
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// The same for TgSmall: the k-steps dealt to the four wavefronts, each with a ring of its own
// (as tg_run_small).
template <class C>
struct F8One : C {
  static constexpr int WM = 1, WN = 1, FM = 2, FN = 2;
  static __host__ __device__ constexpr int column(int f) { return f; }
  static __host__ __device__ constexpr int first(int) { return 0; }
};
template <class C, class P>
__device__ __forceinline__ void f8_run_small(const P& p, int tiles, uint8_t* __restrict__ lds) {
  constexpr int W = TgSmall::WAVES, NI = C::NI;
  using One = F8One<C>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uni(tid >> 6);
  uint8_t* ring = lds + wave * (C::S * C::SLOT);
  const F8Places at = f8_places<One>(0, 0, lane);
  TgTiles q;
  q.init(tiles, nullptr);
  int hint = 0;
  for (int j = q.own;; j += q.blocks(q.x)) {
    const int L = q.at(q.x, j);
    if (L < 0) break;
    const typename P::Tile t = p.tile(L, hint);
    hint = t.hint;
    uint32_t ox[2], ow[2], sx, sw;
    const F8Load lx = f8_prepare<C, false>(t.X, false, t.m0, t.steps, t.length, 0, lane, ox, sx);
    const F8Load lw = f8_prepare<C, C::WCOL>(t.W, true, t.n0, t.steps, t.length, 0, lane, ow, sw);
    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][k][r] = 0.f;
    const int mine = t.steps > wave ? (t.steps - wave + W - 1) / W : 0;
    auto issue = [&](int i, uint8_t* slot) {
      const int s = wave + W * i;
      const bool on = i < mine;
      f8_mask_tail(lx, s, lane, ox);
      f8_mask_tail(lw, s, lane, ow);
      const F8Source fx = f8_source(lx, s, on), fw = f8_source(lw, s, on);
#pragma unroll
      for (int k = 0; k < C::LOADS; ++k) f8_load<C>(fx, lx, k, ox, sx, slot, 0);
#pragma unroll
      for (int k = 0; k < C::LOADS; ++k) f8_load<C>(fw, lw, k, ow, sw, slot, 1);
    };
    // ODD: through registers, as loads that go straight to LDS take whole words only
    u32x4 vx[NI], vw[NI];
    float fx = 0.f, fw = 0.f;
    auto fetch = [&](int i) {
      if (i >= mine) return;
      const int s = wave + W * i;
#pragma unroll
      for (int k = 0; k < NI; ++k) {
        vx[k] = f8_odd_load<C, false>(t.X, t.m0, t.length, s, k, lane);
        vw[k] = f8_odd_load<C, C::WCOL>(t.W, t.n0, t.length, s, k, lane);
      }
      fx = *(const float*)(lx.scales + (size_t)s * lx.s_step + sx);
      fw = *(const float*)(lw.scales + (size_t)s * lw.s_step + sw);
    };
    if constexpr (C::ODD) {
      fetch(0);
    } else {
      issue(0, ring);
      issue(1, ring + C::SLOT);
    }
    for (int i = 0; i < mine; ++i) {
      uint8_t* slot = ring + (i & 1) * C::SLOT;
      if constexpr (C::ODD) {
#pragma unroll
        for (int k = 0; k < NI; ++k) {
          const int s = wave + W * i;
          *(u32x4*)(slot + k * 1024 + lane * 16) =
              f8_odd_cut<C, false>(vx[k], t.X, t.m0, t.length, s, k, lane);
          *(u32x4*)(slot + (NI + k) * 1024 + lane * 16) =
              f8_odd_cut<C, C::WCOL>(vw[k], t.W, t.n0, t.length, s, k, lane);
        }
        *(float*)(slot + C::DATA + lane * 4) = fx;
        *(float*)(slot + C::DATA + 256 + lane * 4) = fw;
        MOE_WAIT_LGKMCNT0();
      } else {
        MOE_WAIT_VMCNT(2 * NI + 2);  // this k-step has landed, the next one may be in flight
      }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      F8Frag x[2], w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        x[k] = f8_frag_x<One>(slot, at, k);
        w[k] = f8_frag_w<One>(slot, at, k);
      }
      const F8Scales<One> s = f8_scales<One>(slot, 0, lane);
      MOE_WAIT_LGKMCNT0();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (C::ODD) fetch(i + 1);
      else issue(i + 2, slot);
#pragma unroll
      for (int fn = 0; fn < 2; ++fn)
#pragma unroll
        for (int fm = 0; fm < 2; ++fm)
          f8_add(acc[fm][fn], f8_products<One>(w[fn], x[fm]), f8_scale_of<One>(s, fm, fn));
    }
    MOE_WAIT_VMCNT(0);  // the sums go through the ring
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
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
      for (int o = 0; o < W; ++o) {
        const f32x4 a =
            *(const f32x4*)(lds + o * (C::S * C::SLOT) + wave * 4096 + r * 1024 + lane * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += a[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[0][0][4 * r + e] = v[e];
    }
    __syncthreads();  // the rings take the next tile's loads
    p.store(t, wave / C::WN, wave % C::WN, lane, sum);
  }
}

}  // namespace
}  // namespace moe
