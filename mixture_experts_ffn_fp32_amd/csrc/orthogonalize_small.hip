// Newton-Schulz steps on matrices whose smaller side is at most 128: one block per matrix
// and one launch for everything (gfx950).  Products, scales and the completed square are
// those of orthogonalize.hip, which takes three launches per step and splits a matrix over
// many blocks.
//
// With p the smaller side (PP: padded to 64 or 128) and X stored p x q, a step is one pass
// over X in chunks of 64 columns:
//
//   S = A + d I and P = c S^2 + (a - c d^2) I in LDS, P's fragments into registers,
//   for each chunk: X' = P X (the chunk through transposing LDS reads), X' to LDS and to
//   the next step's X, and at once A' += X' X'^T for the next step.
//
// X lives in the workspace, which this CU's L2 share holds; chunks land by direct-to-LDS
// loads, two ahead, and X' of one chunk is multiplied while the next is formed.  One CU
// then does 6 p^2 q multiply-adds with 32 x 32 tiles per wavefront: a chunk takes 1.2 us at
// p = 64 and 2.1 us at p = 128 (2.5 GHz), of which the MFMAs are 0.4 and 1.3; the rest is
// the chain from barrier to LDS read to MFMA to split to LDS write, which one or two
// wavefronts per SIMD do not hide (MFMAs busy 32% on a CU in use, LDS 26%).  16 float32
// matrices of 128 x 256, five steps: 83 us (110 us in 17 launches), of 64 x 64: 19 us (93 us).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "ops_internal.h"
#include "tile_gemm.h"

namespace moe {
namespace {

template <int PP>
struct NsSmall {
  static constexpr int RB = PP / 32;            // 32-row blocks
  static constexpr int NW = 2 * RB;             // wavefronts: RB row blocks x 2 column blocks
  static constexpr int THREADS = NW * 64;
  static constexpr int UNIT = PP * 128;         // one unit (32 columns) of all rows
  static constexpr int CHUNK = 2 * UNIT;        // 64 columns
  static constexpr int SQUARE = RB * UNIT;      // S or P
  static constexpr int OTHER = SQUARE > 2 * CHUNK ? SQUARE : 2 * CHUNK;  // also two X' chunks
  static constexpr int SLOTS = 3;               // chunks of X
  static constexpr int NI = 2 * PP / 8 / NW;    // loads per wavefront per chunk
  static constexpr int TA = RB / 2;             // tiles of A per wavefront
  // lo lo' too: where sums are short, what it leaves out (2^-24.5 of a product typically) is what their
  // error consists of (8 x 16: 1.2e-6 -> 1.0e-6 relative, 64 x 64 1.4e-6 -> 1.2e-6, where float32 products
  // have 0.7e-6 and 1.2e-6; 5% of the time).  For sides past 64 it costs 12% and their error is
  // that of float32 products without it.
  static constexpr bool FOUR = PP == 64;
};

struct NsSmallArgs {
  const void* x;
  void* out;
  long long x_stride, out_stride;  // elements per matrix
  uint8_t* planes;                 // [B][2] split matrices of PP rows
  long long plane;                 // bytes of one
  int p, q, steps;
  int tall;                        // the matrices are stored q x p
  int out_dtype;
  int linear;                      // c = 0: P = a I + b A
  float eps, first;                // first: 2^ex
  float s_scale, s_diag, p_scale, p_diag, x_scale, last_scale;
};

__device__ __forceinline__ f32x16 ns_mfma(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Byte of 16-byte chunk c of row r of a unit: chunk positions are rotated by the row so that
// reads along the rows (16 rows of one chunk) and transposing ones (32 bytes of four
// rows, the second pair's 64 bytes away) meet each bank once.
__device__ __forceinline__ uint32_t ns_place(int r, int c) {
  const int turn = ((r >> 1) & 1) * 4 | ((r >> 2) & 1) * 2 | ((r >> 3) & 1);
  return r * 128 + ((c ^ turn) << 4);
}

// A lane's addresses of fragments, from row 0 of a unit on: the rotation of a row's chunks
// does not change over 16 rows, so everything else is a constant offset.
struct NsLane {
  uint32_t rows[2][2];  // [kg % 2][hi, lo]
  uint32_t cols[2][2];  // [hi, lo][first, second four rows]

  __device__ __forceinline__ explicit NsLane(int lane) {
    const int r = 8 * (lane >> 5) + ((lane & 15) >> 2);
    const int n = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        rows[i][j] = ns_place(lane & 31, j * 4 + i * 2 + (lane >> 5));
        cols[i][j] = ns_place(r + 4 * j, i * 4 + (n >> 3)) + (n & 7) * 2;
      }
    keep();
  }
  // The addresses are kept in registers as they are; sums of them with a slot's address are
  // derived behind each keep() again, not kept as well.
  __device__ __forceinline__ void keep() {
    asm volatile(""
                 : "+v"(rows[0][0]), "+v"(rows[0][1]), "+v"(rows[1][0]), "+v"(rows[1][1]),
                   "+v"(cols[0][0]), "+v"(cols[0][1]), "+v"(cols[1][0]), "+v"(cols[1][1]));
  }
};

// Row-layout fragment: 32 rows from `row`, indices 16 (kg % 2) .. of unit kg / 2 (part 0:
// hi, 1: lo) of a matrix of units of PP rows.
template <int PP>
__device__ __forceinline__ u32x4 ns_rows(const uint8_t* m, int row, int kg, int part,
                                         const NsLane& at) {
  return *(const u32x4*)(m + row * 128 + at.rows[kg & 1][part] + (kg >> 1) * NsSmall<PP>::UNIT);
}
// The same of the transpose: 32 columns of one unit, rows 16 kg ...
__device__ __forceinline__ u32x4 ns_cols(const uint8_t* unit, int kg, int part, const NsLane& at) {
  const uint2 lo = tg_read_tr(unit + at.cols[part][0] + kg * 2048);
  const uint2 hi = tg_read_tr(unit + at.cols[part][1] + kg * 2048);
  return u32x4{lo.x, lo.y, hi.x, hi.y};
}
// Four consecutive values of a row (column j a multiple of 4) as split values.
template <int PP>
__device__ __forceinline__ void ns_put4(uint8_t* m, int row, int j, const float (&v)[4]) {
  uint16_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) split_f16(v[e], h[e], l[e]);
  uint8_t* u = m + (j >> 5) * NsSmall<PP>::UNIT + (j & 7) * 2;
  const int c = (j & 31) >> 3;
  *(uint2*)(u + ns_place(row, c)) =
      uint2{h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16)};
  *(uint2*)(u + ns_place(row, 4 + c)) =
      uint2{l[0] | ((uint32_t)l[1] << 16), l[2] | ((uint32_t)l[3] << 16)};
}

// acc[t] += rows(row) rows(col + 32 t)^T over a group of 16 indices: its fragments, and
// its products.
template <int TA>
struct NsGram {
  u32x4 ah, al, bh[TA], bl[TA];
};
template <int PP, int TA>
__device__ __forceinline__ void ns_gram_read(const uint8_t* m, int row, int col, int kg,
                                             const NsLane& at, NsGram<TA>& g) {
  g.ah = ns_rows<PP>(m, row, kg, 0, at);
#pragma unroll
  for (int t = 0; t < TA; ++t) g.bh[t] = ns_rows<PP>(m, col + 32 * t, kg, 0, at);
#pragma unroll
  for (int t = 0; t < TA; ++t) g.bl[t] = ns_rows<PP>(m, col + 32 * t, kg, 1, at);
  g.al = ns_rows<PP>(m, row, kg, 1, at);
}
template <int PP, int TA>
__device__ __forceinline__ void ns_gram_add(const NsGram<TA>& g, f32x16 (&acc)[TA]) {
#pragma unroll
  for (int t = 0; t < TA; ++t) acc[t] = ns_mfma(g.ah, g.bh[t], acc[t]);
#pragma unroll
  for (int t = 0; t < TA; ++t) acc[t] = ns_mfma(g.ah, g.bl[t], acc[t]);
#pragma unroll
  for (int t = 0; t < TA; ++t) acc[t] = ns_mfma(g.al, g.bh[t], acc[t]);
  if constexpr (NsSmall<PP>::FOUR) {
#pragma unroll
    for (int t = 0; t < TA; ++t) acc[t] = ns_mfma(g.al, g.bl[t], acc[t]);
  }
}
template <int TA>
__device__ __forceinline__ void ns_clear(f32x16 (&acc)[TA]) {
#pragma unroll
  for (int t = 0; t < TA; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[t][r] = 0.f;
}
// Sums over 64 indices are added up apart from the total: a chain's rounding then is that of
// 12 products and of one addition per 64 indices, not of every product against the total
// (30 x 500: error 2.1e-6 -> 1.2e-6 relative, 64 x 700 1.8e-6 -> 1.4e-6, where float32 products have
// 1.6e-6 and 1.5e-6; 16 matrices of 128 x 256 75 -> 80 us, of 64 x 64 unchanged).
template <int TA>
__device__ __forceinline__ void ns_add(const f32x16 (&part)[TA], f32x16 (&acc)[TA]) {
#pragma unroll
  for (int t = 0; t < TA; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[t][r] += part[t][r];
}
// The same over KGS groups, each one's fragments read ahead of the products before.
template <int PP, int KGS, int TA>
__device__ __forceinline__ void ns_gram(const uint8_t* m, int row, int col, const NsLane& at,
                                        f32x16 (&acc)[TA]) {
  NsGram<TA> g[2];
  f32x16 part[TA];
  ns_gram_read<PP>(m, row, col, 0, at, g[0]);
#pragma unroll
  for (int kg = 0; kg < KGS; ++kg) {
    if (kg % 4 == 0) ns_clear(part);
    if (kg + 1 < KGS) ns_gram_read<PP>(m, row, col, kg + 1, at, g[(kg + 1) & 1]);
    ns_gram_add<PP>(g[kg & 1], part);
    if (kg % 4 == 3) ns_add(part, acc);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// A symmetric accumulator tile as rows of m: a lane holds rows i .. i + 3 of column j,
// written as columns i .. of row j.  Scaled, `diag` added, zero outside p x p.
template <int PP>
__device__ __forceinline__ void ns_put_square(uint8_t* m, int row, int col, const f32x16& acc,
                                              float scale, float diag, int p, int lane) {
  const int j = col + (lane & 31);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int i = row + 8 * q + 4 * (lane >> 5);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = acc[4 * q + e] * scale + (i + e == j ? diag : 0.f);
      if (i + e >= p || j >= p) v[e] = 0.f;
    }
    ns_put4<PP>(m, j, i, v);
  }
}

// The elements of a 16-byte chunk.
template <class E>
__device__ __forceinline__ void ns_unpack(u32x4 raw, float* f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (E::kPerChunk == 4) {
      f[e] = __uint_as_float(raw[e]);
    } else {
      f[2 * e] = __uint_as_float(raw[e] << 16);
      f[2 * e + 1] = __uint_as_float(raw[e] & 0xffff0000u);
    }
  }
}

// One chunk's loads from `base` (bound: 0 for zeros), each lane's offsets in off.
template <int PP>
__device__ __forceinline__ void ns_load(const uint8_t* base, int bound, int wave,
                                        const uint32_t (&off)[NsSmall<PP>::NI],
                                        uint8_t* __restrict__ slot) {
#pragma unroll
  for (int i = 0; i < NsSmall<PP>::NI; ++i)
    dma16(base, off[i], slot + (wave * NsSmall<PP>::NI + i) * 1024, bound);
}

// A chunk to the iterate in memory, as it lies in LDS (16-byte chunks rotated per row).
template <int PP>
__device__ __forceinline__ void ns_save(const uint8_t* chunk, uint8_t* to, int c, int wave, int lane,
                                        const uint32_t (&off)[NsSmall<PP>::NI]) {
  const __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc((void*)to, (short)0, 0x7fffffff, 0x00020000);
#pragma unroll
  for (int i = 0; i < NsSmall<PP>::NI; ++i)
    __builtin_amdgcn_raw_buffer_store_b128(
        *(const u32x4*)(chunk + (wave * NsSmall<PP>::NI + i) * 1024 + lane * 16), r, off[i], c * 256, 0);
}

// What a wavefront knows of itself.
template <int PP>
struct NsWave {
  int lane, wave;
  int row, col, half;  // first row of its tiles, first column of its tiles of A and S^2, its unit
  uint32_t off[NsSmall<PP>::NI];
};

// S from A's accumulators, S^2, P: P's fragments of this wavefront's rows in ph, pl.  The
// first two chunks are on their way meanwhile.  (LDS that loads in flight write and LDS
// that is read go by different restrict pointers here and below: the compiler then
// does not wait for the loads before each read.)
template <int PP>
__device__ __forceinline__ void ns_factor(const NsSmallArgs& a, const NsWave<PP>& w, const NsLane& at,
                                          const uint8_t* base0, const uint8_t* base1, int bound1,
                                          uint8_t* __restrict__ slot0,
                                          uint8_t* __restrict__ slot1, uint8_t* __restrict__ square,
                                          f32x16 (&acc)[NsSmall<PP>::TA], u32x4 (&ph)[PP / 16],
                                          u32x4 (&pl)[PP / 16]) {
  constexpr int TA = NsSmall<PP>::TA;
  ns_load<PP>(base0, 0x7fffffff, w.wave, w.off, slot0);
  ns_load<PP>(base1, bound1, w.wave, w.off, slot1);
  if (!a.linear) {
#pragma unroll
    for (int t = 0; t < TA; ++t)
      ns_put_square<PP>(square, w.row, w.col + 32 * t, acc[t], a.s_scale, a.s_diag, a.p, w.lane);
    lds_sync();
    ns_clear(acc);
    ns_gram<PP, PP / 16>(square, w.row, w.col, at, acc);
    lds_sync();
  }
#pragma unroll
  for (int t = 0; t < TA; ++t)
    ns_put_square<PP>(square, w.row, w.col + 32 * t, acc[t], a.p_scale, a.p_diag, a.p, w.lane);
  lds_sync();
#pragma unroll
  for (int kg = 0; kg < PP / 16; ++kg) {
    ph[kg] = ns_rows<PP>(square, w.row, kg, 0, at);
    pl[kg] = ns_rows<PP>(square, w.row, kg, 1, at);
  }
  ns_clear(acc);
}

// Behind the barrier of chunk c: y = P X of this wavefront's 32 rows and its unit's columns
// (APPLY), the products of X' c - 1 added to A and X' c - 1 stored (ADD): two independent
// chains of products.  X' c goes to `next` (unless this is the last step), chunk c + 2 to `wr`.
template <int PP, bool APPLY, bool ADD>
__device__ __forceinline__ void ns_chunk(const NsWave<PP>& w, NsLane at, const uint8_t* base,
                                         int bound, uint8_t* to, int c, uint8_t* __restrict__ wr,
                                         const uint8_t* __restrict__ chunk,
                                         const uint8_t* __restrict__ done, uint8_t* __restrict__ next,
                                         bool last, float scale,
                                         const u32x4 (&ph)[PP / 16], const u32x4 (&pl)[PP / 16],
                                         f32x16& y, f32x16 (&acc)[NsSmall<PP>::TA]) {
  // (the stores first: the next barrier's wait then leaves the loads outstanding, not them)
  if constexpr (ADD) ns_save<PP>(done, to, c - 1, w.wave, w.lane, w.off);
  ns_load<PP>(base, bound, w.wave, w.off, wr);
  if constexpr (APPLY) {
#pragma unroll
    for (int r = 0; r < 16; ++r) y[r] = 0.f;
  }
  at.keep();
  // every group's fragments are read ahead of the products before it
  constexpr int TA = NsSmall<PP>::TA, KGS = PP / 16;
  NsGram<TA> g[2];
  if constexpr (APPLY) {
    const uint8_t* unit = chunk + w.half * NsSmall<PP>::UNIT;
    u32x4 xh[2], xl[2];
    xh[0] = ns_cols(unit, 0, 0, at);
    xl[0] = ns_cols(unit, 0, 1, at);
#pragma unroll
    for (int kg = 0; kg < KGS; ++kg) {
      if (kg + 1 < KGS) {
        xh[(kg + 1) & 1] = ns_cols(unit, kg + 1, 0, at);
        xl[(kg + 1) & 1] = ns_cols(unit, kg + 1, 1, at);
      } else if (ADD) {
        ns_gram_read<PP>(done, w.row, w.col, 0, at, g[0]);
      }
      y = ns_mfma(xh[kg & 1], ph[kg], y);
      y = ns_mfma(xh[kg & 1], pl[kg], y);
      y = ns_mfma(xl[kg & 1], ph[kg], y);
      if constexpr (NsSmall<PP>::FOUR) y = ns_mfma(xl[kg & 1], pl[kg], y);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
    ns_gram_read<PP>(done, w.row, w.col, 0, at, g[0]);
  }
  f32x16 part[TA];
  if constexpr (ADD) {
    ns_clear(part);
#pragma unroll
    for (int kg = 0; kg < 4; ++kg) {
      if (kg + 1 < 4) ns_gram_read<PP>(done, w.row, w.col, kg + 1, at, g[(kg + 1) & 1]);
      ns_gram_add<PP>(g[kg & 1], part);
      if (kg + 1 < 4) __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (APPLY) {
    if (!last) {
      // a lane holds columns j .. j + 3 of its row
      int lane = w.lane;
      asm volatile("" : "+v"(lane));  // (addresses derived here, not kept)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = y[4 * q + e] * scale;
        ns_put4<PP>(next, w.row + (lane & 31), w.half * 32 + 8 * q + 4 * (lane >> 5), v);
      }
    }
  }
  if constexpr (ADD) ns_add(part, acc);
}

// The result's columns of chunk c: a lane holds columns j .. j + 3 of its row.  Whole runs of
// four where a row is made of them (its start is aligned to them then), else element by
// element; of a tall matrix neighbouring lanes hold neighbouring elements.
__device__ __forceinline__ void ns_write(float* to, float v) { *to = v; }
__device__ __forceinline__ void ns_write(uint16_t* to, float v) { *to = f32_to_bf16(v); }
__device__ __forceinline__ void ns_write4(float* to, const float (&v)[4]) {
  *(f32x4*)to = f32x4{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void ns_write4(uint16_t* to, const float (&v)[4]) {
  *(uint2*)to = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}
template <int PP, class O>
__device__ __forceinline__ void ns_result(const NsSmallArgs& a, O* out, const NsWave<PP>& w, int c,
                                          const f32x16& y) {
  int lane = w.lane;
  asm volatile("" : "+v"(lane));  // (addresses derived here, not kept)
  const int r = w.row + (lane & 31), j0 = c * 64 + w.half * 32 + 4 * (lane >> 5);
  if (r >= a.p) return;
  const int row_step = a.tall ? 1 : a.q, col_step = a.tall ? a.p : 1;
  const bool runs = !a.tall && a.q % 4 == 0, whole = c * 64 + 64 <= a.q;
  O* to = out + (long long)blockIdx.x * a.out_stride + r * row_step + j0 * col_step;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = y[4 * q + e] * a.last_scale;
    if (runs) {
      if (whole || j0 + 8 * q < a.q) ns_write4(to + 8 * q, v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (whole || j0 + 8 * q + e < a.q) ns_write(to + (8 * q + e) * col_step, v[e]);
    }
  }
}

template <class E, int PP>
__global__ __launch_bounds__(NsSmall<PP>::THREADS) void ns_small_kernel(NsSmallArgs a) {
  using N = NsSmall<PP>;
  using T = typename E::T;
  // (one array: between several the compiler would wait for loads in flight all the same)
  __shared__ __attribute__((aligned(1024))) uint8_t lds[N::SLOTS * N::CHUNK + N::OTHER];
  uint8_t* chunks = lds;
  uint8_t* other = lds + N::SLOTS * N::CHUNK;
  double* s_norm = (double*)other;
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int nc = (a.q + 63) >> 6;
  const T* x = (const T*)a.x + (long long)blockIdx.x * a.x_stride;
  // X_k in plane k % 2 (by arithmetic: an array of pointers would make its accesses flat
  // ones, for which every wait for LDS waits)
  uint8_t* planes = a.planes + (long long)blockIdx.x * 2 * a.plane;
  const uint32_t pitch = (uint32_t)nc * 256;

  // the norm, in float64 (the matrix is p q <= 128 q values: 32-bit indices reach them)
  const int count = a.p * a.q;
  const bool aligned = a.x_stride % E::kPerChunk == 0;  // every matrix starts 16-byte aligned
  double v = 0.0;
  if (aligned && count % E::kPerChunk == 0) {
    constexpr int AHEAD = 16;  // loads in flight per thread (past the end: of the first chunk, not counted)
    for (int i = tid * E::kPerChunk; i < count; i += AHEAD * N::THREADS * E::kPerChunk) {
      u32x4 raw[AHEAD];
#pragma unroll
      for (int w = 0; w < AHEAD; ++w) {
        const int j = i + w * N::THREADS * E::kPerChunk;
        raw[w] = *(const u32x4*)(x + (j < count ? j : 0));
      }
#pragma unroll
      for (int w = 0; w < AHEAD; ++w) {
        if (i + w * N::THREADS * E::kPerChunk >= count) break;
        float f[E::kPerChunk];
        ns_unpack<E>(raw[w], f);
#pragma unroll
        for (int e = 0; e < E::kPerChunk; ++e) v += (double)f[e] * (double)f[e];
      }
    }
  } else {
#pragma unroll 8
    for (int i = tid; i < count; i += N::THREADS) {
      const double f = (double)load_as_f32<E>(x + i);
      v += f * f;
    }
  }
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
  if (lane == 0) s_norm[wave] = v;
  __syncthreads();
  double sq = 0.0;
#pragma unroll
  for (int w = 0; w < N::NW; ++w) sq += s_norm[w];
  const double norm = sqrt(sq) + (double)a.eps;
  // X_0 = x f0, f0 = scale 2^raise: the power of two first, exact on the smallest values (an
  // all-zero matrix stays zero; f0's rounding scales the whole matrix by 1 +- 2^-24)
  int raise = 0;
  const float scale = (float)frexp(norm == 0.0 ? 0.0 : (double)a.first / norm, &raise);
  __syncthreads();

  // this lane's 16 bytes of a chunk: instruction i covers rows 8 i .. of one of its units
  NsWave<PP> w;
  w.lane = lane;
  w.wave = wave;
  w.half = wave / N::RB;
  w.row = wave % N::RB * 32;
  w.col = w.half * N::TA * 32;
#pragma unroll
  for (int i = 0; i < N::NI; ++i) {
    const int g = wave * N::NI + i, u = g / (PP / 8), r = g % (PP / 8) * 8 + (lane >> 3);
    w.off[i] = (uint32_t)r * pitch + u * 128 + (ns_place(r, lane & 7) & 127);
  }
  const NsLane at(lane);
  f32x16 acc[N::TA];
  // chunks past the last one are loaded as zeros
  auto chunk_of = [&](const uint8_t* x, int c) { return uni(x + (size_t)min(c, nc - 1) * 256); };
  auto bound_of = [&](int c) { return c < nc ? 0x7fffffff : 0; };

  // X_0 (zeros in the padding of rows and columns), a chunk at a time: two pieces of eight
  // consecutive columns of a row per thread (tall: neighbouring threads take neighbouring
  // rows, which are neighbouring elements).  Its A with it.
  ns_clear(acc);
  {
    const bool vec = !a.tall && aligned && a.q % E::kPerChunk == 0;
    const int row_step = a.tall ? 1 : a.q, col_step = a.tall ? a.p : 1;
    constexpr int NV = 8 / E::kPerChunk;
    struct Ahead {  // (vec: as raw chunks)
      u32x4 raw[2][NV];
      float one[2][8];
    } even, odd;  // two chunks on their way
    auto fetch = [&](Ahead& g, int c) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = tid + h * N::THREADS, r = a.tall ? i % PP : i >> 3;
        const int j = c * 64 + (a.tall ? i / PP : i & 7) * 8;
        if (vec) {
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int jv = j + v * E::kPerChunk;
            g.raw[h][v] = *(const u32x4*)(x + (((r < a.p) & (jv < a.q)) ? r * a.q + jv : 0));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const bool in = (r < a.p) & (j + e < a.q);
            g.one[h][e] = load_as_f32<E>(x + (in ? r * row_step + (j + e) * col_step : 0));
          }
        }
      }
    };
    auto put = [&](Ahead& g, int c) {
      uint8_t* to = other + (c & 1) * N::CHUNK;
      float f[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = tid + h * N::THREADS, r = a.tall ? i % PP : i >> 3;
        const int j = c * 64 + (a.tall ? i / PP : i & 7) * 8;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (vec) ns_unpack<E>(g.raw[h][v], g.one[h] + v * E::kPerChunk);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          f[h][e] = ((r < a.p) & (j + e < a.q)) ? ldexpf(g.one[h][e], raise) * scale : 0.f;
      }
      fetch(g, min(c + 2, nc - 1));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = tid + h * N::THREADS, r = a.tall ? i % PP : i >> 3;
        const int j = (a.tall ? i / PP : i & 7) * 8;
#pragma unroll
        for (int q = 0; q < 8; q += 4) {
          const float four[4] = {f[h][q], f[h][q + 1], f[h][q + 2], f[h][q + 3]};
          ns_put4<PP>(to, r, j + q, four);
        }
      }
      lds_sync();
      ns_gram<PP, 4>(to, w.row, w.col, at, acc);
      ns_save<PP>(to, planes, c, wave, lane, w.off);
    };
    fetch(even, 0);
    fetch(odd, min(1, nc - 1));
    for (int c = 0; c < nc; c += 2) {
      put(even, c);
      if (c + 1 < nc) put(odd, c + 1);
    }
  }
  MOE_WAIT_VMCNT(0);
  __syncthreads();

  for (int k = 0; k < a.steps; ++k) {
    const bool last = k + 1 == a.steps;
    const uint8_t* from = planes + (k & 1) * a.plane;
    uint8_t* to = planes + (~k & 1) * a.plane;
    u32x4 ph[PP / 16], pl[PP / 16];
    ns_factor<PP>(a, w, at, chunk_of(from, 0), chunk_of(from, 1), bound_of(1), chunks, chunks + N::CHUNK,
                  other, acc, ph, pl);
    // One barrier per chunk: behind it chunk c has landed, X' of chunk c - 1 is whole, and
    // the slots of chunk c - 1 and of X' c - 2 (and, at first, P) are free.
    int slot = 0;  // of chunk c
    auto step = [&](int c, auto apply, auto add) {
      // Loads land in order among themselves, so that with as many accesses outstanding as
      // chunk c + 1 has loads, chunk c has landed.  The count names no stores: whether those
      // retire in order with loads is not relied upon.
      MOE_WAIT_VMCNT(N::NI);
      lds_sync();
      f32x16 y;
      ns_chunk<PP, apply.value, add.value>(
          w, at, chunk_of(from, c + 2), bound_of(c + 2), to, c,
          chunks + (slot == 0 ? 2 : slot - 1) * N::CHUNK, chunks + slot * N::CHUNK,
          other + ((c + 1) & 1) * N::CHUNK, other + (c & 1) * N::CHUNK, last, a.x_scale, ph, pl, y, acc);
      slot = uni(slot == 2 ? 0 : slot + 1);
      if constexpr (apply.value) {
        if (last) {
          if (a.out_dtype == 0) ns_result<PP>(a, (float*)a.out, w, c, y);
          else ns_result<PP>(a, (uint16_t*)a.out, w, c, y);
        }
      }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    step(0, Yes{}, No{});
    if (last) {
      for (int c = 1; c < nc; ++c) step(c, Yes{}, No{});
    } else {
      for (int c = 1; c < nc; ++c) step(c, Yes{}, Yes{});
      step(nc, No{}, Yes{});
    }
    // this step's loads and stores are done before the next one's loads
    MOE_WAIT_VMCNT(0);
    __syncthreads();
  }
}

template <class E, int PP>
void run_small(const NsSmallArgs& s, int B, hipStream_t st) {
  ns_small_kernel<E, PP><<<B, NsSmall<PP>::THREADS, 0, st>>>(s);
}

int padded_side(int side) { return side <= 64 ? 64 : 128; }
long long plane_bytes(int m, int n) {
  return (long long)padded_side(std::min(m, n)) * ((std::max(m, n) + 63) / 64) * 256;
}

}  // namespace

// Whether one block per matrix is faster than the general path, whose launches take 90 us
// or more but spread a matrix over many blocks.  Measured (float32, five steps), general -> this
// one: one matrix of 64 x 512 98 -> 68 us, of 64 x 1024 109 -> 118 us, of 128 x 256 104 -> 81 us, of
// 128 x 512 109 -> 128 us; 16 of 64 x 1024 117 -> 127 us, of 128 x 512 114 -> 133 us; 64 of
// 64 x 2048 346 -> 263 us, of 128 x 1024 234 -> 263 us; 256 of 64 x 64 163 -> 23 us, of 128 x
// 4096 2423 -> 1580 us.  That is a limit of chunks (of 128 rows: twice) that grows with the
// CUs that the matrices occupy.
bool ortho_small_fits(int B, int m, int n) {
  const int side = std::min(m, n);
  if (side > 128) return false;
  const int work = ((std::max(m, n) + 63) / 64) * (padded_side(side) / 64);
  return work <= 10 + (long long)B * B / 64;
}

size_t ortho_small_workspace_bytes(int B, int m, int n) { return (size_t)B * 2 * plane_bytes(m, n); }

hipError_t launch_orthogonalize_small(const OrthoArgs& a, const OrthoScales& sc, void* ws, hipStream_t st) {
  NsSmallArgs s{};
  s.x = a.x;
  s.out = a.out;
  s.x_stride = a.x_stride;
  s.out_stride = a.out_stride;
  s.planes = (uint8_t*)ws;
  s.plane = plane_bytes(a.m, a.n);
  s.p = std::min(a.m, a.n);
  s.q = std::max(a.m, a.n);
  s.steps = a.steps;
  s.tall = a.m > a.n;
  s.out_dtype = a.out_dtype;
  s.linear = a.c == 0.f;
  s.eps = a.eps;
  s.first = sc.first;
  s.s_scale = sc.s_scale;
  s.s_diag = sc.s_diag;
  s.p_scale = sc.p_scale;
  s.p_diag = sc.p_diag;
  s.x_scale = sc.x_scale;
  s.last_scale = sc.last_scale;
  if (padded_side(s.p) == 64) {
    if (a.dtype == 0) run_small<ElemF32, 64>(s, a.B, st);
    else run_small<ElemBF16, 64>(s, a.B, st);
  } else {
    if (a.dtype == 0) run_small<ElemF32, 128>(s, a.B, st);
    else run_small<ElemBF16, 128>(s, a.B, st);
  }
  return hipGetLastError();
}

}  // namespace moe
