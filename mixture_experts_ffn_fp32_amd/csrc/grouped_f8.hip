// Products of 8-bit operands grouped by expert with ragged sizes (gfx950), the grouped products
// of grouped.hip for experts held in 8 bits with a float32 scale for each block of 128 (f8.h):
//
//   forward   y[r]  = sum over blocks b of k  xs[r][b] ws[e][n/128][b] sum_{k in b} xq[r][k] wq[e][n][k]
//   gradient  dx[r] = sum over blocks b of n  dys[r][b] ws[e][b][k/128] sum_{n in b} dyq[r][n] wq[e][n][k]
//
// A block's sum and the sum over blocks are float32, the result is rounded once.  The weights'
// scales hold for 128 x 128 elements, so both directions read the same weights.
//
// The 8-bit matrix instructions form exact products, but add eight neighbours along the
// contraction at the place of the largest of the eight, where what lies 13 bits below it or
// lower is cut off (measured: beside a product of 2^8, 2^-5 is kept and 2^-6 lost among the same
// eight, 2^-15 kept in any other eight; normal values give sums off by 1.5e-5, relatively, in the
// mean).  A bfloat16 result, whose own rounding is a hundred times that (1.7e-3), is computed so,
// at twice the bfloat16 rate.  A float32 result is computed from the same operands as bfloat16,
// which hold every 8-bit value, by the bfloat16 instructions, whose sums keep float32's bits
// (8e-9 in the same measurement).
#include <algorithm>

#include "f8.h"
#include "groups.h"
#include "ops_internal.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct F8Product {
  const uint8_t* x;        // x or dy: rows of the groups
  const float* xs;
  const uint8_t* w;        // [E][n][k]
  const float* ws;         // [E][nb][kb]
  const int32_t* offsets;
  void* out;
  GroupDims g;
  int zero_rest;
};

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

// w fragment times x fragment of one block of 128, from zero: a lane holds four consecutive
// columns (w's rows) 4 (lane / 16) .. of row lane % 16.
template <int Q, bool EXACT>
__device__ __forceinline__ f32x4 f8_mfma(const i32x8& w, const i32x8& x) {
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if constexpr (!EXACT)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, sum, 0, Q == F8_E5M2 ? 1 : 0, 0,
                                                            0x7f7f7f7f, 0, 0x7f7f7f7f);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f8_widen<F8_E4M3>(w[2 * i], w[2 * i + 1]),
                                                  f8_widen<Q>(x[2 * i], x[2 * i + 1]), sum, 0, 0, 0);
  return sum;
}

constexpr int kF8Tile = 64;

template <int DIR, int Q, bool F32>
__global__ __launch_bounds__(256) void grouped_f8_kernel(F8Product p) {
  __shared__ GroupTables t;
  __shared__ __attribute__((aligned(16))) uint8_t sx[kF8Tile * 128], sw[kF8Tile * 128];
  const GroupDims& g = p.g;
  group_tables<GR_FWD>(g, p.offsets, kF8Tile, t);
  const int N = DIR == GR_FWD ? g.n : g.k, K = DIR == GR_FWD ? g.k : g.n;
  if (p.zero_rest) {
    if (F32) zero_rows((float*)p.out, g.M, N, t.off[0], t.off[g.E]);
    else zero_rows((uint16_t*)p.out, g.M, N, t.off[0], t.off[g.E]);
  }
  const int nt = (N + kF8Tile - 1) / kF8Tile, nb = f8_blocks(g.n), kb = f8_blocks(g.k);
  const int steps = DIR == GR_FWD ? kb : nb;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
  const long long tiles = (long long)t.tiles[g.E] * nt;
  for (long long L = blockIdx.x; L < tiles; L += gridDim.x) {
    const int mt = uni((int)(L / nt)), n0 = uni((int)(L % nt)) * kF8Tile;
    const int e = uni(group_of(t.tiles, g.E, mt, 0));
    const int m0 = t.off[e] + (mt - t.tiles[e]) * kF8Tile, rows = min(kF8Tile, t.off[e + 1] - m0);
    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < steps; ++s) {
      __syncthreads();
      for (int i = tid; i < kF8Tile * 128; i += 256) {
        const int r = i >> 7, j = i & 127, kk = s * 128 + j;
        const int at = lds_chunk_offset(r, j >> 4) + (j & 15);
        sx[at] = r < rows && kk < K ? p.x[(size_t)(m0 + r) * K + kk] : 0;
        const size_t we = (size_t)e * g.n * g.k;
        if (DIR == GR_FWD) sw[at] = n0 + r < N && kk < K ? p.w[we + (size_t)(n0 + r) * g.k + kk] : 0;
        else sw[at] = n0 + r < N && kk < K ? p.w[we + (size_t)kk * g.k + n0 + r] : 0;
      }
      __syncthreads();
      const float wscale = DIR == GR_FWD ? p.ws[((size_t)e * nb + n0 / 128) * kb + s]
                                         : p.ws[((size_t)e * nb + s) * kb + n0 / 128];
      i32x8 xf[2], wf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 2 * (lane >> 4);
        const int rx = wm * 32 + 16 * i + (lane & 15), rw = wn * 32 + 16 * i + (lane & 15);
        const u32x4 a = *(const u32x4*)(sx + lds_chunk_offset(rx, c));
        const u32x4 b = *(const u32x4*)(sx + lds_chunk_offset(rx, c + 1));
        const u32x4 d = *(const u32x4*)(sw + lds_chunk_offset(rw, c));
        const u32x4 f = *(const u32x4*)(sw + lds_chunk_offset(rw, c + 1));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          xf[i][q] = a[q];
          xf[i][4 + q] = b[q];
          wf[i][q] = d[q];
          wf[i][4 + q] = f[q];
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = wm * 32 + 16 * i + (lane & 15);
        const float scale = r < rows ? p.xs[(size_t)(m0 + r) * steps + s] * wscale : 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const f32x4 part = f8_mfma<Q, F32>(wf[j], xf[i]);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] += scale * part[q];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = wm * 32 + 16 * i + (lane & 15);
      if (r >= rows) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = n0 + wn * 32 + 16 * j + 4 * (lane >> 4) + q;
          if (c >= N) continue;
          const size_t at = (size_t)(m0 + r) * N + c;
          if (F32) ((float*)p.out)[at] = acc[i][j][q];
          else ((uint16_t*)p.out)[at] = f32_to_bf16(acc[i][j][q]);
        }
    }
  }
}

}  // namespace

size_t grouped_f8_workspace_bytes(int, int, int, int, bool) { return 0; }

hipError_t launch_grouped_f8(int f8, bool dx, const GroupedF8Args& a, void*, hipStream_t st) {
  F8Product p{};
  p.x = (const uint8_t*)a.x;
  p.xs = a.xs;
  p.w = (const uint8_t*)a.w;
  p.ws = a.ws;
  p.offsets = a.offsets;
  p.out = a.out;
  p.g = GroupDims{a.M, a.E, a.n, a.k};
  p.zero_rest = a.zero_rest;
  const long long tiles =
      (a.M / kF8Tile + 1LL + a.E) * (((dx ? a.k : a.n) + kF8Tile - 1) / kF8Tile);
  const unsigned grid = (unsigned)std::min<long long>(tiles, 4LL * device_cu_count());
  const int which = (dx ? 4 : 0) + (f8 == F8_E5M2 ? 2 : 0) + (a.out_f32 ? 1 : 0);
  switch (which) {
    case 0: grouped_f8_kernel<GR_FWD, F8_E4M3, false><<<grid, 256, 0, st>>>(p); break;
    case 1: grouped_f8_kernel<GR_FWD, F8_E4M3, true><<<grid, 256, 0, st>>>(p); break;
    case 2: grouped_f8_kernel<GR_FWD, F8_E5M2, false><<<grid, 256, 0, st>>>(p); break;
    case 3: grouped_f8_kernel<GR_FWD, F8_E5M2, true><<<grid, 256, 0, st>>>(p); break;
    case 4: grouped_f8_kernel<GR_DX, F8_E4M3, false><<<grid, 256, 0, st>>>(p); break;
    case 5: grouped_f8_kernel<GR_DX, F8_E4M3, true><<<grid, 256, 0, st>>>(p); break;
    case 6: grouped_f8_kernel<GR_DX, F8_E5M2, false><<<grid, 256, 0, st>>>(p); break;
    default: grouped_f8_kernel<GR_DX, F8_E5M2, true><<<grid, 256, 0, st>>>(p); break;
  }
  return hipGetLastError();
}

}  // namespace moe
