// Groups of rows with ragged sizes, as every block of a product over them sees them (gfx950).
#pragma once

#include "lds_dma.h"
#include "ops_internal.h"

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
__host__ __device__ __forceinline__ int group_tiles(const GroupDims& g, int rows, int bm) {
  const int v = DIR == GR_DW ? (rows > 0 ? g.n : 0) : rows;  // (up to 2^31 - 1)
  return v / bm + (v % bm != 0);
}

__device__ __forceinline__ int wave_prefix(int v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// All threads of the block.  offsets NULL: one group of all the rows.
template <int DIR>
__device__ __forceinline__ void group_tables(const GroupDims& g, const int32_t* __restrict__ offsets,
                                             int bm, GroupTables& t) {
  for (int i = threadIdx.x; i <= g.E; i += blockDim.x)
    t.off[i] = offsets != nullptr ? min(max(offsets[i], 0), g.M) : i > 0 ? g.M : 0;
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

}  // namespace
}  // namespace moe
