// Products grouped by expert with ragged sizes (gfx950), the products of an
// expert FFN (DeepSeekMoE paper summary, papercache.org, sec. 3.2: each token
// goes through its experts' matrices) for experts of a caller's own making:
//
//   forward   y[r]  = w[e] x[r]                  offsets[e] <= r < offsets[e+1]
//   backward  dx[r] = w[e]^T dy[r],  dw[e] = sum of dy[r] x[r]^T over e's rows
//
// One launch covers every group: each block derives the tile table from the
// offsets in LDS (clamped into [0, M] and made non-decreasing, so any offsets
// stay inside the buffers and no row belongs to two groups) and takes its share
// of the tiles.  The groups need no padding between them: an m-tile ends at its
// group's last row, and the weight gradient's contraction over a group's rows
// ends there by a bounded buffer range.
//
// bfloat16 operands are read where they are (the transposed products through
// transposing LDS reads).  float32 operands of y are first written as two float16 each
// (tile_gemm.h), with a power-of-two scale per row of x and w.  The gradients contract over
// rows of w, and of dy and x, where no scale of a row can be taken out again and
// experts, rows and channels differ by any factor: their operands are written as three
// bfloat16 each, which need no scale.
//
// The parts of an infinity are an infinity and NaN, so a float32 result with one among its
// operands comes out as NaN, and what leaves float32's range on the way as either.  Every
// float32 result that is not finite is therefore summed again from the operands themselves,
// in float64 (grouped_again).  The search of the results in registers takes up to 1% of y's
// time where all are finite; an infinity in every row of x, 28665 of 1280 values, takes y
// from 0.4 to 79 ms.
//
// Measured: y of 49152 rows in 64 groups, 1408 x 2048 bfloat16, 313 to 331 us (905 to 856 TFLOP/s of the
// 1338 that one dense product reaches here; MFMAs busy 47%); of 384 rows, 2048 x 1408, 69 us (HBM
// bound, 5.4 TB/s); both gradients of 28672 rows in 63 groups, 896 x 1280, 240 to 251 us (dw's 289 MB
// written at 2.2 TB/s, dx 635 TFLOP/s); float32 y of 8190 rows in 16 groups, 896 x 1280, 108 us, of
// which 38 us split x and w.  float32 gradients of those 28672 rows: 228 us for the parts of dy, x
// and w (1.08 GB, 4.7 TB/s), dx 423 us and dw 447 us (930 and 880 TFLOP/s of bfloat16 products).
#include <float.h>

#include <algorithm>

#include "ops_internal.h"
#include "tile_gemm.h"

namespace moe {
namespace {

enum : int { GR_FWD = 0, GR_DX = 1, GR_DW = 2 };

// ---------------------------------------------------------------- groups
struct GroupDims {
  int M, E, n, k;
};
// The groups as every block sees them in LDS: their rows (offsets clamped into [0, M]
// and made non-decreasing), and the exclusive prefix of their m-tiles.
struct GroupTables {
  int off[kGroupedMaxE + 1], tiles[kGroupedMaxE + 1];
};

template <int DIR>
__device__ __forceinline__ int group_tiles(const GroupDims& g, int rows, int bm) {
  return ((DIR == GR_DW ? (rows > 0 ? g.n : 0) : rows) + bm - 1) / bm;
}

__device__ __forceinline__ int wave_prefix(int v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// All threads of the block.
template <int DIR>
__device__ __forceinline__ void group_tables(const GroupDims& g, const int32_t* __restrict__ offsets,
                                             int bm, GroupTables& t) {
  for (int i = threadIdx.x; i <= g.E; i += blockDim.x) t.off[i] = min(max(offsets[i], 0), g.M);
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int top = t.off[0], carry = 0;
    for (int b = 0; b < g.E; b += 64) {
      const int e = b + lane;
      int hi = e < g.E ? t.off[e + 1] : 0;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(hi, o);
        if (lane >= o) hi = max(hi, y);
      }
      hi = max(hi, top);
      const int up = __shfl_up(hi, 1);
      const int own = e < g.E ? group_tiles<DIR>(g, hi - (lane == 0 ? top : up), bm) : 0;
      const int sum = wave_prefix(own, lane);
      if (e < g.E) {
        t.off[e + 1] = hi;
        t.tiles[e] = carry + sum - own;
      }
      carry += __shfl(sum, 63);
      top = __shfl(hi, 63);
    }
    if (lane == 0) t.tiles[g.E] = carry;
  }
  __syncthreads();
}

// The group of the key-th m-tile of a prefix table (tab[E] > key): the last one whose
// first is at or before it, looked for near e first (a block's tiles come in order).
__device__ __forceinline__ int group_of(const int* tab, int E, int key, int e) {
  if (key < uni(tab[e]) || key >= uni(tab[min(e + 4, E)])) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (uni(tab[mid]) <= key) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
  while (uni(tab[e + 1]) <= key) ++e;
  return e;
}

// Zeros into the rows [0, first) and [last, M) of out, this block's share.
template <class T>
__device__ __forceinline__ void zero_rows(T* out, int M, int width, int first, int last) {
  const long long n0 = (long long)first * width, n1 = (long long)(M - last) * width;
  T* tail = out + (long long)last * width;
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n0 + n1; i += stride)
    (i < n0 ? out + i : tail + (i - n0))[0] = T(0);
}

// ---------------------------------------------------------------- the product
struct GroupedProduct {
  const uint8_t* A;        // x or dy (rows of the groups)
  const uint8_t* B;        // w (forward, dx) or x (weight gradient)
  uint32_t pitch_a, pitch_b;
  uint32_t plane_a, plane_b;  // three parts: bytes of one in a row
  const int32_t* offsets;
  void* out;
  const int32_t* ea;       // two parts: exponents of x's rows, and
  const int32_t* eb;       //   of w's
  GroupDims g;
  int zero_rest;
  const float *ra, *rb;    // float32: A's and B's operands as the caller gave them
};

__device__ __forceinline__ bool not_finite(float v) { return !(fabsf(v) <= FLT_MAX); }

// sum of a[i sa] b[i sb] over n terms in float64: products are exact, no partial sum leaves the
// range, infinities and NaN come out as in any order of summation.
__device__ __forceinline__ float grouped_again(const float* a, size_t sa, const float* b, size_t sb,
                                               int n) {
  double s = 0.0;
  for (int i = 0; i < n && s == s; ++i, a += sa, b += sb) s = fma((double)*a, (double)*b, s);
  return (float)s;
}

template <class C, int DIR>
struct GroupedTiles {
  const GroupedProduct& p;
  const GroupTables& g_;

  static constexpr bool SYM = false;
  struct Tile {
    TgOperand A, B;
    int m0, n0, steps, rows, cols, hint, row0, size;
  };
  __device__ __forceinline__ bool tri(const Tile&) const { return false; }
  __device__ __forceinline__ int columns() const {
    return ((DIR == GR_FWD ? p.g.n : p.g.k) + C::BN - 1) / C::BN;
  }
  __device__ __forceinline__ Tile tile(int L, int e) const {  // group by group, m fastest
    const GroupDims& g = p.g;
    const int nt = columns();
    e = uni(group_of(g_.tiles, g.E, L / nt, e));
    const int first = uni(g_.tiles[e]), mt = uni(g_.tiles[e + 1]) - first, local = L - first * nt;
    const int m = local % mt, n = local / mt;
    Tile t;
    t.hint = e;
    t.row0 = uni(g_.off[e]);
    t.size = uni(g_.off[e + 1]) - t.row0;
    t.m0 = m * C::BM;
    t.n0 = n * C::BN;
    t.rows = (DIR == GR_DW ? g.n : t.size) - t.m0;
    t.cols = (DIR == GR_FWD ? g.n : g.k) - t.n0;
    t.A.p = p.A + (size_t)t.row0 * p.pitch_a;
    t.A.pitch = p.pitch_a;
    t.A.rows = t.size;
    t.A.width = (g.n + 31) & ~31;
    t.A.plane = p.plane_a;
    t.B.pitch = p.pitch_b;
    t.B.plane = p.plane_b;
    if (DIR == GR_DW) {
      t.B.p = p.B + (size_t)t.row0 * p.pitch_b;
      t.B.rows = t.size;
      t.B.width = (g.k + 31) & ~31;
      t.steps = (t.size + C::KS - 1) / C::KS;
    } else {
      t.B.p = p.B + (size_t)t.hint * g.n * p.pitch_b;
      t.B.rows = g.n;
      t.B.width = (g.k + 31) & ~31;
      t.steps = ((DIR == GR_FWD ? g.k : g.n) + C::KS - 1) / C::KS;
    }
    if (C::PARTS == 1) {  // a bfloat16 row holds what its pitch says
      t.A.width = min(t.A.width, (int)(p.pitch_a / 2));
      t.B.width = min(t.B.width, (int)(p.pitch_b / 2));
    } else if (C::PARTS == 3) {
      t.steps *= kTgProducts;
      t.A.width = min(t.A.width, (int)(p.plane_a / 2));
      t.B.width = min(t.B.width, (int)(p.plane_b / 2));
    }
    return t;
  }

  __device__ __forceinline__ void store(const Tile& t, int wm, int wn, int lane,
                                        f32x16 (&acc)[C::FM][C::FN]) const {
    const GroupDims& g = p.g;
    if constexpr (DIR == GR_DW) {
      float* out = (float*)p.out + (size_t)t.hint * g.n * g.k;
      bool bad = false;
#pragma unroll
      for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int m = t.m0 + tg_row<C>(wm, fm, lane, r);
          if (m >= g.n) continue;
#pragma unroll
          for (int fn = 0; fn < C::FN; ++fn) {
            const int n = t.n0 + tg_col<C>(wn, fn, lane, r);
            if (n < g.k) {
              const float v = C::PARTS == 3 ? acc[fm][fn][r] * kTgUnlift : acc[fm][fn][r];
              out[(size_t)m * g.k + n] = v;
              bad |= not_finite(v);
            }
          }
        }
      if (C::PARTS == 3 && bad) again(t, wm, wn, lane);
    } else {
      // a lane holds four consecutive columns of one row
      const int N = DIR == GR_FWD ? g.n : g.k;
      bool bad = false;
      const bool vec = N % (C::PARTS > 1 ? 4 : 8) == 0;  // whole 16-byte runs
#pragma unroll
      for (int fm = 0; fm < C::FM; ++fm) {
        const int mr = tg_row<C>(wm, fm, lane, 0);
        if (mr >= t.rows) continue;
        const size_t row = (size_t)(t.row0 + t.m0 + mr);
        const int ea = C::SPLIT ? p.ea[row] : 0;
#pragma unroll
        for (int fn = 0; fn < C::FN; ++fn) {
          const int n0 = t.n0 + tg_col<C>(wn, fn, 0, 0);  // the fragment's first column
          if (n0 >= N) continue;
          if constexpr (C::PARTS > 1) {
            float* c = (float*)p.out + row * N;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int n = n0 + 8 * q + 4 * (lane >> 5);
              float v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[e] = acc[fm][fn][4 * q + e];
                if (n + e < N) {
                  if constexpr (C::SPLIT) v[e] = ldexpf(v[e], -ea - p.eb[(size_t)t.hint * g.n + n + e]);
                  else v[e] *= kTgUnlift;
                  bad |= not_finite(v[e]);
                }
              }
              if (vec) {
                if (n < N) *(f32x4*)(c + n) = f32x4{v[0], v[1], v[2], v[3]};
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (n + e < N) c[n + e] = v[e];
              }
            }
          } else {
            uint16_t* c = (uint16_t*)p.out + row * N;
            uint2 w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = uint2{pack_bf16x2(acc[fm][fn][4 * q], acc[fm][fn][4 * q + 1]),
                           pack_bf16x2(acc[fm][fn][4 * q + 2], acc[fm][fn][4 * q + 3])};
            if (vec) {
              u32x4 r0, r1;
              tg_runs16(w, r0, r1);
              const int n = n0 + 8 * (lane >> 5);
              if (n < N) *(u32x4*)(c + n) = r0;
              if (n + 16 < N) *(u32x4*)(c + n + 16) = r1;
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int n = n0 + 8 * q + 4 * (lane >> 5);
                const uint32_t b[2] = {w[q].x, w[q].y};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (n + e < N) c[n + e] = (uint16_t)(b[e >> 1] >> (16 * (e & 1)));
              }
            }
          }
        }
      }
      if (C::PARTS > 1 && bad) again(t, wm, wn, lane);
    }
  }

  // This lane's float32 results that are not finite, as it stored them, summed again.
  __device__ __forceinline__ void again(const Tile& t, int wm, int wn, int lane) const {
    const GroupDims& g = p.g;
    const int M = DIR == GR_DW ? g.n : t.size, N = DIR == GR_FWD ? g.n : g.k;
    float* out = (float*)p.out + (DIR == GR_DW ? (size_t)t.hint * g.n : (size_t)t.row0) * N;
    const float* a = p.ra + (size_t)t.row0 * (DIR == GR_FWD ? g.k : g.n);
    const float* b = p.rb + (DIR == GR_DW ? (size_t)t.row0 : (size_t)t.hint * g.n) * g.k;
    for (int i = 0; i < C::FM * C::FN * 16; ++i) {
      const int f = i >> 4, m = t.m0 + tg_row<C>(wm, f / C::FN, lane, i & 15);
      const int n = t.n0 + tg_col<C>(wn, f % C::FN, lane, i & 15);
      if (m >= M || n >= N) continue;
      float* to = out + (size_t)m * N + n;
      if (!not_finite(*to)) continue;
      if (DIR == GR_FWD) *to = grouped_again(a + (size_t)m * g.k, 1, b + (size_t)n * g.k, 1, g.k);
      if (DIR == GR_DX) *to = grouped_again(a + (size_t)m * g.n, 1, b + n, g.k, g.n);
      if (DIR == GR_DW) *to = grouped_again(a + m, g.n, b + n, g.k, t.size);
    }
  }
};

template <class C, int DIR>
__global__ __launch_bounds__(C::THREADS, C::WAVES_PER_SIMD) void grouped_kernel(
    GroupedProduct p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::LDS];
  __shared__ GroupTables t;
  group_tables<DIR>(p.g, p.offsets, C::BM, t);
  if (DIR != GR_DW && p.zero_rest) {
    const int width = DIR == GR_FWD ? p.g.n : p.g.k;
    if (C::PARTS > 1) zero_rows((float*)p.out, p.g.M, width, t.off[0], t.off[p.g.E]);
    else zero_rows((uint16_t*)p.out, p.g.M, width, t.off[0], t.off[p.g.E]);
  }
  if (DIR == GR_DW) {  // groups without rows have no tiles
    const size_t per = (size_t)p.g.n * p.g.k;
    for (int e = 0; e < p.g.E; ++e)
      if (t.off[e] == t.off[e + 1])
        for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < per;
             i += (size_t)gridDim.x * blockDim.x)
          ((float*)p.out)[e * per + i] = 0.f;
  }
  const GroupedTiles<C, DIR> tiles{p, t};
  const int n = uni(t.tiles[p.g.E]) * tiles.columns();
  if constexpr (C::SMALL) tg_run_small<C>(tiles, n, lds);
  else tg_run<C>(tiles, n, nullptr, lds, nullptr);
}

// ---------------------------------------------------------------- operand preparation
// float32 rows -> split rows.  One wavefront per row; lane l takes the 8-element chunks
// l, l + 64, ..: 32 bytes read, 16 bytes of hi and of lo written, each row read once
// (it stays in registers between the maximum and the split; longer ones are read
// again).  HBM bound.
constexpr int kRowChunks = 4;  // chunks per lane held in registers: rows up to 2048

// Exponent that brings a largest magnitude to [2^13, 2^14); 0 if all is zero.
__device__ __forceinline__ int split_exponent(float most) {
  return most > 0.f ? 13 - ilogbf(most) : 0;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) v = fmaxf(v, __shfl_xor(v, k));
  return v;
}

// (of the finite values: an infinity or NaN stays one in its own products and takes no
// other value's scale)
__device__ __forceinline__ float chunk_max(const float (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]) <= FLT_MAX ? fabsf(f[e]) : 0.f);
  return m;
}
// Splits one row; returns its exponent.
__device__ __forceinline__ int split_row(const float* __restrict__ src, int width,
                                         uint8_t* __restrict__ dst, int lane) {
  const int padded = (width + 31) & ~31;
  float f[kRowChunks][8], m = 0.f;
#pragma unroll
  for (int c = 0; c < kRowChunks; ++c) load_chunk<ElemF32>(src, 8 * (lane + 64 * c), width, f[c]);
#pragma unroll
  for (int c = 0; c < kRowChunks; ++c) m = fmaxf(m, chunk_max(f[c]));
  for (int j = 8 * (lane + 64 * kRowChunks); j < width; j += 512) {
    float g[8];
    load_chunk<ElemF32>(src, j, width, g);
    m = fmaxf(m, chunk_max(g));
  }
  const int ex = split_exponent(wave_max(m));
#pragma unroll
  for (int c = 0; c < kRowChunks; ++c) {
    const int j = 8 * (lane + 64 * c);
    if (j < padded) store_chunk(f[c], dst, j, ex);
  }
  for (int j = 8 * (lane + 64 * kRowChunks); j < padded; j += 512) {
    float g[8];
    load_chunk<ElemF32>(src, j, width, g);
    store_chunk(g, dst, j, ex);
  }
  return ex;
}

// One kind of rows of a launch: four rows per block.
struct SplitRows {
  const float* src;
  uint8_t* dst;
  int32_t* ex;      // per row
  long long rows;
  uint32_t pitch;
  int width;
};
// Blocks that prepare an operand.  A launch holds fewer than 2^32 threads: past kMostBlocks
// each block takes further rows.
constexpr long long kMostBlocks = 1 << 20;
__host__ __device__ inline unsigned blocks_of(long long rows) {
  const long long b = (rows + 3) / 4;
  return (unsigned)(b < kMostBlocks ? b : kMostBlocks);
}
__device__ __forceinline__ void split_rows(const SplitRows& a, unsigned block) {
  const int lane = threadIdx.x & 63;
  for (long long r = (long long)block * 4 + (threadIdx.x >> 6); r < a.rows; r += 4 * kMostBlocks) {
    const int ex = split_row(a.src + r * a.width, a.width, a.dst + r * a.pitch, lane);
    if (lane == 0) a.ex[r] = ex;
  }
}
// The forward's operands, in one launch.
__global__ __launch_bounds__(256) void split_two_kernel(SplitRows a, SplitRows b) {
  const unsigned n = blocks_of(a.rows);
  if (blockIdx.x < n) split_rows(a, blockIdx.x);
  else split_rows(b, blockIdx.x - n);
}

// float32 rows as three bfloat16 each (tile_gemm.h), times kTgLift, zeros behind the last
// element; a lane takes 8 elements, 2^shift lanes a row.  HBM bound: 4 bytes read, 6 written.
struct PartRows {
  const float* src;
  uint8_t* dst;
  long long rows;
  uint32_t plane;    // bytes of a row's part, a multiple of 16; three of them a row
  int width, shift;
  unsigned blocks;
};
// dy is dx's A too, whose k-steps read 64 elements of a row.
uint32_t part_plane_dy(int n) { return (uint32_t)((n + 63) / 64 * 128); }
uint32_t part_plane(int k) { return (uint32_t)((k + 7) / 8 * 16); }
PartRows part_rows(const void* src, uint8_t* dst, long long rows, int width, uint32_t plane) {
  PartRows a{(const float*)src, dst, rows, plane, width, 0, 0};
  while (a.shift < 6 && (16u << a.shift) < plane) ++a.shift;
  const long long per = 4 << (6 - a.shift);  // rows per block
  a.blocks = (unsigned)std::min((rows + per - 1) / per, kMostBlocks);
  return a;
}
__device__ __forceinline__ void part_rows(const PartRows& a, unsigned block) {
  const int lane = threadIdx.x & 63;
  long long r = (((long long)block * 4 + (threadIdx.x >> 6)) << (6 - a.shift)) + (lane >> a.shift);
  for (; r < a.rows; r += 4 * kMostBlocks << (6 - a.shift)) {
    const float* src = a.src + r * a.width;
    uint8_t* dst = a.dst + 3 * r * a.plane;
    for (int j = 8 * (lane & ((1 << a.shift) - 1)); j < (int)(a.plane / 2); j += 8 << a.shift) {
      float f[8];
      load_chunk<ElemF32>(src, j, a.width, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= kTgLift;
      const Split3 s = split_three(f);
      uint8_t* to = dst + 2 * (size_t)j;
      *(u32x4*)to = s.hi;
      *(u32x4*)(to + a.plane) = s.mid;
      *(u32x4*)(to + 2 * (size_t)a.plane) = s.lo;
    }
  }
}
// The gradients' operands, in one launch (x is dw's, w dx's: no blocks without them).
__global__ __launch_bounds__(256) void parts_kernel(PartRows dy, PartRows x, PartRows w) {
  const unsigned b = blockIdx.x;
  if (b < dy.blocks) part_rows(dy, b);
  else if (b < dy.blocks + x.blocks) part_rows(x, b - dy.blocks);
  else part_rows(w, b - dy.blocks - x.blocks);
}

// bfloat16 rows whose length does not suit the loads, copied into rows of whole
// 128-byte units with zeros behind the last element.
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* __restrict__ src,
                                                       long long rows, int width,
                                                       uint8_t* __restrict__ dst, uint32_t pitch) {
  const int lane = threadIdx.x & 63;
  for (long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); r < rows; r += 4 * kMostBlocks) {
    const uint16_t* s = src + r * width;
    for (int j = 2 * lane; j < (int)(pitch / 2); j += 128) {
      const uint32_t a = j < width ? s[j] : 0, b = j + 1 < width ? s[j + 1] : 0;
      *(uint32_t*)(dst + r * pitch + 2 * j) = a | (b << 16);
    }
  }
}

// ---------------------------------------------------------------- launch
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// ---------------------------------------------------------------- float32, few rows per group
// With few rows the product is bound by reading w once (64 groups of 6 rows, w 2048 x 1408:
// 738 MB), and writing w's split form and reading it back would treble that.  Here w's
// rows go from memory to registers and are split there, into three bfloat16:
// (the triple precision of tile_gemm.h), which need no scale of w's rows (whose maximum
// would take a read of its own).  x is split likewise beforehand (it is small).
//
// A block takes 64 columns of y and up to 32 rows of a group; its four wavefronts deal the
// k-steps of 32 indices among themselves, each with four fragments of 16 w rows against one
// or two of x rows, loads two k-steps ahead and no barrier; the four sums are added through
// LDS in wavefront order.  Loads of fragments touch many rows, and what they cost is lines:
// a lane of quarter g takes the indices 4 g .. 4 g + 3 and 16 + 4 g .. of a k-step (any order
// does that x and w share), so a load takes 64 bytes of 16 rows, and x lies in that order
// (fragments of 32 rows, 32 bytes of each per load, and x by rows: 209 us for the 174 below).
//
// dx = w^T dy likewise, contracting over w's rows: a lane of quarter g and index i loads 4
// consecutive values of the rows 4 g .. 4 g + 3 and 16 + 4 g .. of a k-step, from column 4 i of
// the tile on, a load 256 bytes of four rows; fragment c takes the c-th of each four (its row i
// is column 4 i + c of the tile), so that a lane ends with runs of four columns.
constexpr int kFewRows = 32, kFewCols = 64;
struct FewProduct {
  const float* w;
  const u32x4* x;          // (dx: dy) [k-step][quarter][hi, mid, lo][M]: a lane's eight values of a row
  const int32_t* offsets;
  float* out;
  GroupDims g;
  int zero_rest;
  const float* rows;       // x or dy themselves
};
// Bytes of x's split row.
__host__ __device__ inline long long few_pitch(int k) { return (long long)((k + 31) / 32) * 192; }

// x's rows (of a multiple of 4 values; 128 kGroupedMaxE at most), one wavefront each.
__global__ __launch_bounds__(256) void split_three_kernel(const float* __restrict__ x, int rows, int k,
                                                          u32x4* __restrict__ out) {
  const long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (r >= rows) return;
  const float* src = x + r * k;
  float f[8];
  for (int c = lane; c < (k + 31) / 32 * 4; c += 64) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = c / 4 * 32 + h * 16 + c % 4 * 4;
      const f32x4 v = j < k ? *(const f32x4*)(src + j) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) f[4 * h + i] = v[i] * kTgLift;
    }
    const Split3 s = split_three(f);
    u32x4* to = out + (long long)c * 3 * rows + r;
    to[0] = s.hi;
    to[rows] = s.mid;
    to[2LL * rows] = s.lo;
  }
}

__device__ __forceinline__ f32x4 few_mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A wavefront's operands of a k-step.
template <int RF>
struct FewLoad {
  f32x4 w[4][2];
  Split3 x[RF];
};
// The sums of this wavefront's k-steps for 64 columns and 16 RF rows.
template <bool DX, int RF>
__device__ __forceinline__ void few_tile(const FewProduct& p, int e, int row0, int rows, int n0,
                                         int wave, int lane, f32x4 (&acc)[4][RF]) {
  const int n = p.g.n, k = p.g.k, length = DX ? n : k;
  const int steps = (length + 31) / 32, g = lane >> 4, i16 = lane & 15;
  // rows past the last one (of w, of the group) reread it and are never stored
  const float* w[DX ? 1 : 4];
  if constexpr (DX) {
    w[0] = p.w + (size_t)e * n * k + (n0 + 4 * i16 < k ? n0 + 4 * i16 : 0);
  } else {
#pragma unroll
    for (int f = 0; f < 4; ++f) w[f] = p.w + ((size_t)e * n + min(n0 + 16 * f + i16, n - 1)) * k;
  }
  const u32x4* x[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) x[f] = p.x + row0 + min(16 * f + i16, rows - 1);
  // index j of a lane's eight in a k-step (four of them are inside the contraction or past it)
  auto index = [&](int s, int j) { return 32 * s + 16 * (j >> 2) + 4 * g + (j & 3); };
  auto load = [&](int s, FewLoad<RF>& d) {
    s = min(s, steps - 1);
#pragma unroll
    for (int f = 0; f < RF; ++f) {
      const u32x4* from = x[f] + (size_t)(s * 4 + g) * 3 * p.g.M;
      d.x[f] = Split3{from[0], from[p.g.M], from[2LL * p.g.M]};
    }
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (DX) {
          d.w[f][h] = *(const f32x4*)(w[0] + (size_t)min(index(s, 4 * h + f), n - 1) * k);
        } else {
          const int j = index(s, 4 * h);
          d.w[f][h] = *(const f32x4*)(w[f] + (j < k ? j : 0));
        }
      }
  };
  auto multiply = [&](int s, const FewLoad<RF>& d) {
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      float v[8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[4 * h + i] = index(s, 4 * h) < length ? (DX ? d.w[i][h][f] : d.w[f][h][i]) * kTgLift : 0.f;
      const Split3 t = split_three(v);
#pragma unroll
      for (int r = 0; r < RF; ++r) {
        acc[f][r] = few_mfma(t.lo, d.x[r].hi, acc[f][r]);
        acc[f][r] = few_mfma(t.hi, d.x[r].lo, acc[f][r]);
        acc[f][r] = few_mfma(t.mid, d.x[r].mid, acc[f][r]);
        acc[f][r] = few_mfma(t.mid, d.x[r].hi, acc[f][r]);
        acc[f][r] = few_mfma(t.hi, d.x[r].mid, acc[f][r]);
        acc[f][r] = few_mfma(t.hi, d.x[r].hi, acc[f][r]);
      }
    }
  };
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int r = 0; r < RF; ++r) acc[f][r] = f32x4{0.f, 0.f, 0.f, 0.f};
  FewLoad<RF> a, b;
  load(2 * wave, a);
  load(2 * wave + 1, b);
  for (int s = 2 * wave; s < steps; s += 8) {
    multiply(s, a);
    load(s + 8, a);
    if (s + 1 < steps) multiply(s + 1, b);
    load(s + 9, b);
  }
}
// Sums and stores a tile, a lane four columns of one row: wavefront q fragment q's (dx: the
// q-th values of the four fragments, which are neighbours).
template <bool DX, int RF>
__device__ __forceinline__ void few_store(const FewProduct& p, int e, int row0, int rows, int n0, int wave,
                                          int lane, const f32x4 (&acc)[4][RF],
                                          f32x4 (*__restrict__ sum)[4][2][64]) {
  const int width = DX ? p.g.k : p.g.n;
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int r = 0; r < RF; ++r) sum[wave][f][r][lane] = acc[f][r];
  __syncthreads();
#pragma unroll
  for (int r = 0; r < RF; ++r) {
    const int i = 16 * r + (lane & 15);
    const int n = n0 + (DX ? 16 * (lane >> 4) + 4 * wave : 16 * wave + 4 * (lane >> 4));
    if (i >= rows || n >= width) continue;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      if constexpr (DX) {
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] += ((const float*)&sum[o][c][r][lane])[wave];
      } else {
        v += sum[o][wave][r][lane];
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] *= kTgUnlift;
    float* y = p.out + (size_t)(row0 + i) * width + n;
    bool bad = false;
    if (DX || width % 4 == 0) {
      *(f32x4*)y = v;
#pragma unroll
      for (int c = 0; c < 4; ++c) bad |= not_finite(v[c]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (n + c < width) {
          y[c] = v[c];
          bad |= not_finite(v[c]);
        }
    }
    if (bad) {
      const float* a = p.rows + (size_t)(row0 + i) * (DX ? p.g.n : p.g.k);
      const float* w = p.w + (size_t)e * p.g.n * p.g.k;
      for (int c = 0; c < 4 && n + c < width; ++c)
        if (not_finite(y[c]))
          y[c] = DX ? grouped_again(a, 1, w + n + c, p.g.k, p.g.n)
                    : grouped_again(a, 1, w + (size_t)(n + c) * p.g.k, 1, p.g.k);
    }
  }
  __syncthreads();
}
template <bool DX>
__global__ __launch_bounds__(256, 2) void grouped_few_kernel(FewProduct p) {
  __shared__ GroupTables t;
  __shared__ f32x4 sum[4][4][2][64];
  const int width = DX ? p.g.k : p.g.n;
  group_tables<GR_FWD>(p.g, p.offsets, kFewRows, t);
  if (p.zero_rest) zero_rows(p.out, p.g.M, width, t.off[0], t.off[p.g.E]);
  const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
  const int nt = (width + kFewCols - 1) / kFewCols, total = uni(t.tiles[p.g.E]) * nt;
  int e = 0;
  for (int L = blockIdx.x; L < total; L += gridDim.x) {
    e = uni(group_of(t.tiles, p.g.E, L / nt, e));
    const int first = uni(t.tiles[e]), mt = uni(t.tiles[e + 1]) - first, local = L - first * nt;
    const int row0 = uni(t.off[e]) + local % mt * kFewRows, n0 = local / mt * kFewCols;
    const int rows = uni(t.off[e + 1]) - row0;
    if (rows > 16) {
      f32x4 acc[4][2];
      few_tile<DX, 2>(p, e, row0, rows, n0, wave, lane, acc);
      few_store<DX, 2>(p, e, row0, rows, n0, wave, lane, acc, sum);
    } else {
      f32x4 acc[4][1];
      few_tile<DX, 1>(p, e, row0, rows, n0, wave, lane, acc);
      few_store<DX, 1>(p, e, row0, rows, n0, wave, lane, acc, sum);
    }
  }
}
// `in`: x or dy, split into `planes` first.
template <bool DX>
hipError_t run_few(const GroupedArgs& a, const void* in, uint8_t* planes, void* out, hipStream_t st) {
  const int width = DX ? a.k : a.n, length = DX ? a.n : a.k;
  const FewProduct p{(const float*)a.w, (const u32x4*)planes, a.offsets, (float*)out,
                     GroupDims{a.M, a.E, a.n, a.k}, a.zero_rest, (const float*)in};
  split_three_kernel<<<blocks_of(a.M), 256, 0, st>>>((const float*)in, a.M, length, (u32x4*)planes);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const long long most =
      ((long long)a.M / kFewRows + std::min(a.M, a.E)) * ((width + kFewCols - 1) / kFewCols);
  const long long room = 2LL * device_cu_count();
  grouped_few_kernel<DX><<<(unsigned)std::min(most, room), 256, 0, st>>>(p);
  return hipGetLastError();
}

// y: up to 64 rows per group on average.  w 1408 x 2048 and 64 groups, general path -> this one: 6 rows
// 461 -> 175 us (4.2 TB/s), 32 rows 482 -> 222 us, 64 rows 473 -> 384 us; 65 rows 491 | 477 us and 96
// rows, for which it reads w three times, 499 | 541 us; 128 groups of 65 rows, 1000 x 1000, 373 | 482 us.
// Uneven groups read w more often, on either path: of 64 rows on average with sizes as 1 / rank
// (the largest 881 rows) 495 -> 432 us, all rows in one group 363 -> 283 us.
// dx: up to 128 rows, as the general path has six products there: 6 rows 625 -> 157 us, 64 rows 663 -> 311
// us, 96 rows 712 -> 464 us, 128 rows 735 -> 570 us, 160 rows 784 | 779 us (2048 x 1408: 905 | 834 us, 128
// groups of 1000 x 1000: 641 | 720 us); uneven, 64 rows, the largest 881, 747 -> 360 us.
// The widths keep the workspace of fewer rows the smaller one (few_pitch(n) M against w's parts),
// and the tile's 64 columns in use.
bool few_rows(int dtype, int M, int E, int n, int k) {
  return dtype == 0 && k % 4 == 0 && n >= 32 && M <= 64LL * E;
}
bool few_rows_dx(int dtype, int M, int E, int n, int k) {
  return dtype == 0 && k % 4 == 0 && n % 4 == 0 && n >= 32 && k >= 192 && M <= (k >= 256 ? 128LL : 64LL) * E;
}

struct Carve {
  uint8_t* base;
  size_t at = 0;
  uint8_t* take(size_t bytes) {
    uint8_t* p = base != nullptr ? base + at : nullptr;
    at = up256(at + bytes);
    return p;
  }
};

uint32_t pad_pitch(int n) { return (uint32_t)((n + 63) / 64 * 128); }

// About how many tiles of b x b a product has: the offsets are on the device, so half a
// tile's rows are taken as lost per group, and every row as in a group.
long long tiles_of(int dir, const GroupedArgs& a, long long b) {
  auto ct = [](long long x, long long y) { return (x + y - 1) / y; };
  const long long groups = std::min(a.M, a.E);
  if (dir == GR_DW) return ct(a.n, b) * ct(a.k, b) * groups;
  return std::max(groups, a.M / b + groups / 2) * ct(dir == GR_FWD ? a.n : a.k, b);
}

template <class C, int DIR>
hipError_t run_product(const GroupedProduct& p, hipStream_t st) {
  auto ct = [](long long x, long long b) { return (x + b - 1) / b; };
  const GroupDims& g = p.g;
  const long long most =
      DIR == GR_DW ? g.E * ct(g.n, C::BM) * ct(g.k, C::BN)
                   : (ct(g.M, C::BM) + g.E) * ct(DIR == GR_FWD ? g.n : g.k, C::BN);
  const long long blocks = (long long)device_cu_count() * C::BPC;
  grouped_kernel<C, DIR><<<(unsigned)std::max(1LL, std::min(most, blocks)), C::THREADS, 0, st>>>(p);
  return hipGetLastError();
}

template <int DIR, int PARTS>
hipError_t pick_product(const GroupedArgs& a, const GroupedProduct& p, hipStream_t st) {
  constexpr bool AC = DIR == GR_DW, BC = DIR != GR_FWD, SW = DIR != GR_DW;
  const int cus = device_cu_count();
  // The largest tiles that give three quarters of the CUs one (tile_gemm.h; ragged groups
  // fill fewer than half: 8190 rows in 16 uneven groups, y 896 x 1280 float32, 160 tiles of 256
  // rows 137 us, of 128 rows 115 us), and 256 rows only where groups hold more than half of
  // that (64 groups of 64 rows, y 1408 x 2048 bfloat16: 118 us, of 128 rows 107 us; 64 of
  // 256: 138 and 147 us).
  if (4 * tiles_of(DIR, a, 256) >= 3 * cus && (DIR == GR_DW || a.M > 128LL * a.E))
    return run_product<TgConfig<TgBig, AC, BC, PARTS, SW>, DIR>(p, st);
  if (4 * tiles_of(DIR, a, 128) >= 3 * cus)
    return run_product<TgConfig<TgMid, AC, BC, PARTS, SW>, DIR>(p, st);
  return run_product<TgConfig<TgSmall, AC, BC, PARTS, SW>, DIR>(p, st);
}

// The workspace's regions: which are needed, and where they lie.
struct GroupedPlan {
  uint8_t *x = nullptr, *w = nullptr, *dy = nullptr;        // prepared operands
  uint8_t* few = nullptr;                                   // dy, few rows per group
  int32_t *ex = nullptr, *ew = nullptr;                     // exponents
  size_t bytes = 0;
};
GroupedPlan plan_forward(int dtype, int M, int E, int n, int k, void* ws) {
  GroupedPlan p;
  Carve c{(uint8_t*)ws};
  if (few_rows(dtype, M, E, n, k)) {
    p.x = c.take((size_t)M * few_pitch(k));
  } else if (dtype == 0) {
    p.x = c.take((size_t)M * split_pitch(k));
    p.w = c.take((size_t)E * n * split_pitch(k));
    p.ex = (int32_t*)c.take((size_t)M * 4);
    p.ew = (int32_t*)c.take((size_t)E * n * 4);
  } else if (k % 64 != 0) {
    p.x = c.take((size_t)M * pad_pitch(k));
    p.w = c.take((size_t)E * n * pad_pitch(k));
  }
  p.bytes = c.at;
  return p;
}
GroupedPlan plan_backward(int dtype, int M, int E, int n, int k, bool dx, bool dw, void* ws) {
  GroupedPlan p;
  Carve c{(uint8_t*)ws};
  if (M == 0) dx = false;
  if (dx && few_rows_dx(dtype, M, E, n, k)) {
    p.few = c.take((size_t)M * few_pitch(n));
    dx = false;
  }
  if (dtype == 0) {
    if (dx || dw) p.dy = c.take(3 * (size_t)M * part_plane_dy(n));
    if (dx) p.w = c.take(3 * (size_t)E * n * part_plane(k));
    if (dw) p.x = c.take(3 * (size_t)M * part_plane(k));
  } else if (dtype != 0) {
    if (n % (dx ? 64 : 8) != 0) p.dy = c.take((size_t)M * pad_pitch(n));
    if (dx && k % 8 != 0) p.w = c.take((size_t)E * n * pad_pitch(k));
    if (dw && k % 8 != 0) p.x = c.take((size_t)M * pad_pitch(k));
  }
  p.bytes = c.at;
  return p;
}

}  // namespace

int device_cu_count() {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) == hipSuccess &&
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess &&
      cus > 0)
    return cus;
  return 256;
}

size_t grouped_workspace_bytes(int dtype, int M, int E, int n, int k) {
  return plan_forward(dtype, M, E, n, k, nullptr).bytes;
}
size_t grouped_backward_workspace_bytes(int dtype, int M, int E, int n, int k, bool dx, bool dw) {
  return plan_backward(dtype, M, E, n, k, dx, dw, nullptr).bytes;
}

hipError_t launch_grouped(int dtype, const GroupedArgs& a, void* ws, hipStream_t st) {
  const GroupedPlan w = plan_forward(dtype, a.M, a.E, a.n, a.k, ws);
  GroupedProduct p{};
  p.A = (const uint8_t*)a.x;
  p.B = (const uint8_t*)a.w;
  p.pitch_a = p.pitch_b = (uint32_t)a.k * 2;
  p.offsets = a.offsets;
  p.out = a.y;
  p.g = GroupDims{a.M, a.E, a.n, a.k};
  p.zero_rest = a.zero_rest;
  const long long wr = (long long)a.E * a.n;
  if (few_rows(dtype, a.M, a.E, a.n, a.k)) {
    return run_few<false>(a, a.x, w.x, a.y, st);
  }
  if (dtype == 0) {
    p.pitch_a = p.pitch_b = (uint32_t)split_pitch(a.k);
    const SplitRows rx{(const float*)a.x, w.x, w.ex, a.M, p.pitch_a, a.k};
    const SplitRows rw{(const float*)a.w, w.w, w.ew, wr, p.pitch_b, a.k};
    split_two_kernel<<<blocks_of(a.M) + blocks_of(wr), 256, 0, st>>>(rx, rw);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    p.A = w.x;
    p.B = w.w;
    p.ea = w.ex;
    p.eb = w.ew;
    p.ra = (const float*)a.x;
    p.rb = (const float*)a.w;
    return pick_product<GR_FWD, 2>(a, p, st);
  }
  if (w.x != nullptr) {
    p.pitch_a = p.pitch_b = pad_pitch(a.k);
    pad_rows_kernel<<<blocks_of(a.M), 256, 0, st>>>((const uint16_t*)a.x, a.M, a.k, w.x, p.pitch_a);
    pad_rows_kernel<<<blocks_of(wr), 256, 0, st>>>((const uint16_t*)a.w, wr, a.k, w.w, p.pitch_b);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    p.A = w.x;
    p.B = w.w;
  }
  return pick_product<GR_FWD, 1>(a, p, st);
}

hipError_t launch_grouped_backward(int dtype, const GroupedArgs& a, void* ws, hipStream_t st) {
  bool dx = a.dx != nullptr;
  const bool dw = a.dw != nullptr;
  const GroupedPlan w = plan_backward(dtype, a.M, a.E, a.n, a.k, dx, dw, ws);
  if (w.few != nullptr) {
    const hipError_t e = run_few<true>(a, a.dy, w.few, a.dx, st);
    if (e != hipSuccess || !dw) return e;
    dx = false;
  }
  const long long wr = (long long)a.E * a.n;
  GroupedProduct p{};
  p.offsets = a.offsets;
  p.g = GroupDims{a.M, a.E, a.n, a.k};
  p.zero_rest = a.zero_rest;
  const uint8_t *x = (const uint8_t*)a.x, *wt = (const uint8_t*)a.w, *dy = (const uint8_t*)a.dy;
  uint32_t px = a.k * 2, pw = a.k * 2, py = a.n * 2;
  if (dtype == 0) {
    p.plane_a = part_plane_dy(a.n);
    p.plane_b = part_plane(a.k);
    py = 3 * p.plane_a;
    px = pw = 3 * p.plane_b;
    if (a.M > 0) {
      const PartRows ry = part_rows(a.dy, w.dy, a.M, a.n, p.plane_a);
      PartRows rx{}, rw{};
      if (dw) rx = part_rows(a.x, w.x, a.M, a.k, p.plane_b);
      if (dx) rw = part_rows(a.w, w.w, wr, a.k, p.plane_b);
      parts_kernel<<<ry.blocks + rx.blocks + rw.blocks, 256, 0, st>>>(ry, rx, rw);
    }
    dy = w.dy;
    wt = w.w;
    x = w.x;
  } else {
    if (w.dy != nullptr && a.M > 0) {
      py = pad_pitch(a.n);
      pad_rows_kernel<<<blocks_of(a.M), 256, 0, st>>>((const uint16_t*)a.dy, a.M, a.n, w.dy, py);
      dy = w.dy;
    }
    if (w.w != nullptr) {
      pw = pad_pitch(a.k);
      pad_rows_kernel<<<blocks_of(wr), 256, 0, st>>>((const uint16_t*)a.w, wr, a.k, w.w, pw);
      wt = w.w;
    }
    if (w.x != nullptr && a.M > 0) {
      px = pad_pitch(a.k);
      pad_rows_kernel<<<blocks_of(a.M), 256, 0, st>>>((const uint16_t*)a.x, a.M, a.k, w.x, px);
      x = w.x;
    }
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  p.A = dy;
  p.pitch_a = py;
  p.ra = (const float*)a.dy;
  if (dx && a.M > 0) {
    p.B = wt;
    p.pitch_b = pw;
    p.rb = (const float*)a.w;
    p.out = a.dx;
    e = dtype == 0 ? pick_product<GR_DX, 3>(a, p, st) : pick_product<GR_DX, 1>(a, p, st);
    if (e != hipSuccess) return e;
  }
  if (dw) {
    p.B = x;
    p.pitch_b = px;
    p.rb = (const float*)a.x;
    p.out = a.dw;
    e = dtype == 0 ? pick_product<GR_DW, 3>(a, p, st) : pick_product<GR_DW, 1>(a, p, st);
  }
  return e;
}

}  // namespace moe
