// Layer norm, forward and backward (gfx950).  The DeepSeekMoE pages' block
// leaves the norm around the layer out of its equations for brevity
// (papercache.org summary, sec. A3); these are the standard ones:
//
//   mean_t = (1/d) sum_j x_tj,  rstd_t = 1 / sqrt((1/d) sum_j (x_tj - mean_t)^2 + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   g = dy w:  dx = rstd (g - mean_j(g) - xh mean_j(g xh))
//   dw = sum_t dy xh,  db = sum_t dy
//
// Both directions are bound by HBM: x (and dy) once in, y or dx once out.  A
// row therefore stays in registers between its reductions: TPR threads hold
// NCH chunks of 16 bytes each.  The variance is
// the mean of squared deviations from the mean, a second sum over registers
// (no cancellation).  Statistics, gradients and every sum are float32.
//
// The weight gradients need no second read of x and dy: a thread owns the same
// columns in every row its block takes, adds them up in registers, and each
// block writes one partial row; a second launch adds the partial rows in a
// fixed order (repeated calls give identical bits).
//
// Measured: forward of 8192 x 2048 bfloat16 14.5 us (4.6 TB/s of a copy's 5.1), of one row 3.4 us;
// backward of 16384 x 4096 bfloat16 75 us (5.4 TB/s) and 5 us for the column sums, of 3001 x
// 1283 float32 16 + 4 us.
#include <algorithm>

#include "ops_internal.h"
#include "row_chunks.h"

namespace moe {
namespace {

// Chunk c of this thread starts at column (c * TPR + i) * CH (i: the thread's index in
// its row), so a wavefront's load is contiguous.  A chunk's elements past the row's end
// are zeros.
template <class E, int TPR, int NCH, bool WHOLE>
__global__ __launch_bounds__(norm_threads<TPR>()) void norm_fwd_kernel(NormArgs a) {
  using K = Chunk<E, WHOLE>;
  using T = typename E::T;
  constexpr int CH = K::CH;
  __shared__ float s[2 * TPR / 64];
  constexpr int RPB = norm_threads<TPR>() / TPR;  // rows per block
  const int i = threadIdx.x % TPR, d = a.d;
  const float inv_d = 1.f / (float)d;
  for (long long r = (long long)blockIdx.x * RPB + threadIdx.x / TPR; r < a.T;
       r += (long long)gridDim.x * RPB) {
    const T* x = (const T*)a.x + r * d;
    u32x4 xv[NCH];
    float sum = 0.f, zero = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * TPR + i) * CH;
      xv[c] = j < d ? K::load(x, j, d) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float f[CH];
      K::unpack(xv[c], f);
#pragma unroll
      for (int e = 0; e < CH; ++e) sum += f[e];
    }
    row_sum2<TPR>(sum, zero, s);
    const float mean = sum * inv_d;
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * TPR + i) * CH;
      float f[CH];
      K::unpack(xv[c], f);
#pragma unroll
      for (int e = 0; e < CH; ++e) sq += (WHOLE ? j : j + e) < d ? (f[e] - mean) * (f[e] - mean) : 0.f;
    }
    row_sum2<TPR>(sq, zero, s);
    const float rstd = 1.f / sqrtf(sq * inv_d + a.eps);
    if (i == 0) {
      if (a.mean != nullptr) a.mean[r] = mean;
      if (a.rstd != nullptr) a.rstd[r] = rstd;
    }
    T* y = (T*)a.out + r * d;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * TPR + i) * CH;
      if (j >= d) continue;
      float f[CH], w[CH], b[CH];
      K::unpack(xv[c], f);
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        w[e] = 1.f;
        b[e] = 0.f;
      }
      if (a.weight != nullptr) K::unpack(K::load((const T*)a.weight, j, d), w);
      if (a.bias != nullptr) K::unpack(K::load((const T*)a.bias, j, d), b);
#pragma unroll
      for (int e = 0; e < CH; ++e) f[e] = (f[e] - mean) * rstd * w[e] + b[e];
      K::store(y, j, d, f);
    }
  }
}

// DW: also the block's partial weight and bias gradients (part row blockIdx.x).
template <class E, int TPR, int NCH, bool WHOLE, bool DW>
__global__ __launch_bounds__(norm_threads<TPR>()) void norm_bwd_kernel(NormArgs a) {
  using K = Chunk<E, WHOLE>;
  using T = typename E::T;
  constexpr int CH = K::CH;
  constexpr int RPB = norm_threads<TPR>() / TPR;
  // row sums, and (RPB > 1) the rows' column sums on their way into the block's
  __shared__ float s[2 * TPR / 64];
  __shared__ float s_col[(DW && RPB > 1) ? RPB * TPR * CH : 1];
  const int i = threadIdx.x % TPR, d = a.d;
  const float inv_d = 1.f / (float)d;
  float dw[DW ? NCH : 1][CH], db[DW ? NCH : 1][CH];
  if constexpr (DW) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < CH; ++e) dw[c][e] = db[c][e] = 0.f;
  }
  u32x4 wv[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int j = (c * TPR + i) * CH;
    float one[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) one[e] = 1.f;
    wv[c] = a.weight == nullptr ? K::pack(one)
            : j < d             ? K::load((const T*)a.weight, j, d)
                                : u32x4{0u, 0u, 0u, 0u};
  }
  for (long long r = (long long)blockIdx.x * RPB + threadIdx.x / TPR; r < a.T;
       r += (long long)gridDim.x * RPB) {
    const T* x = (const T*)a.x + r * d;
    const T* dy = (const T*)a.dy + r * d;
    u32x4 xv[NCH], yv[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * TPR + i) * CH;
      xv[c] = j < d ? K::load(x, j, d) : u32x4{0u, 0u, 0u, 0u};
      yv[c] = j < d ? K::load(dy, j, d) : u32x4{0u, 0u, 0u, 0u};
    }
    const float mean = a.mean[r], rstd = a.rstd[r];
    float c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float f[CH], g[CH], w[CH];
      K::unpack(xv[c], f);
      K::unpack(yv[c], g);
      K::unpack(wv[c], w);
#pragma unroll
      for (int e = 0; e < CH; ++e) {  // (past the row's end dy = 0)
        const float xh = (f[e] - mean) * rstd, gw = g[e] * w[e];
        c1 += gw;
        c2 += gw * xh;
        if constexpr (DW) {
          dw[c][e] += g[e] * xh;
          db[c][e] += g[e];
        }
      }
    }
    row_sum2<TPR>(c1, c2, s);
    c1 *= inv_d;
    c2 *= inv_d;
    T* dx = (T*)a.out + r * d;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * TPR + i) * CH;
      if (j >= d) continue;
      float f[CH], g[CH], w[CH];
      K::unpack(xv[c], f);
      K::unpack(yv[c], g);
      K::unpack(wv[c], w);
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        const float xh = (f[e] - mean) * rstd;
        f[e] = rstd * (g[e] * w[e] - c1 - xh * c2);
      }
      K::store(dx, j, d, f);
    }
  }
  if constexpr (DW) {
    float* part = a.part + (long long)blockIdx.x * 2 * d;
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int j = (c * TPR + i) * CH;
        float f[CH];
#pragma unroll
        for (int e = 0; e < CH; ++e) f[e] = which == 0 ? dw[c][e] : db[c][e];
        if constexpr (RPB > 1) {
          // the block's RPB rows of threads hold the same columns
          __syncthreads();
#pragma unroll
          for (int e = 0; e < CH; ++e) s_col[(threadIdx.x / TPR * CH + e) * TPR + i] = f[e];
          __syncthreads();
          if (threadIdx.x < TPR) {
#pragma unroll
            for (int e = 0; e < CH; ++e) {
              f[e] = 0.f;
#pragma unroll
              for (int q = 0; q < RPB; ++q) f[e] += s_col[(q * CH + e) * TPR + i];
            }
          }
        }
        if (threadIdx.x < TPR) {
          if (WHOLE ? j < d : j + CH <= d && d % 4 == 0) {
#pragma unroll
            for (int e = 0; e < CH; e += 4)
              *(f32x4*)(part + which * d + j + e) = f32x4{f[e], f[e + 1], f[e + 2], f[e + 3]};
          } else {
#pragma unroll
            for (int e = 0; e < CH; ++e)
              if (!WHOLE && j + e < d) part[which * d + j + e] = f[e];
          }
        }
      }
  }
}

// Rows too long for registers: the row is read again from the caches for each
// reduction.  One block of 1024 threads per row.
template <class E>
__global__ __launch_bounds__(1024) void norm_fwd_long_kernel(NormArgs a) {
  using T = typename E::T;
  __shared__ float s[32];
  const int d = a.d;
  const float inv_d = 1.f / (float)d;
  for (long long r = blockIdx.x; r < a.T; r += gridDim.x) {
    const T* x = (const T*)a.x + r * d;
    float sum = 0.f, sq = 0.f, zero = 0.f;
    for (int j = threadIdx.x; j < d; j += 1024) sum += load_as_f32<E>(x + j);
    row_sum2<1024>(sum, zero, s);
    const float mean = sum * inv_d;
    for (int j = threadIdx.x; j < d; j += 1024) {
      const float f = load_as_f32<E>(x + j) - mean;
      sq += f * f;
    }
    row_sum2<1024>(sq, zero, s);
    const float rstd = 1.f / sqrtf(sq * inv_d + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[r] = mean;
      if (a.rstd != nullptr) a.rstd[r] = rstd;
    }
    for (int j = threadIdx.x; j < d; j += 1024) {
      const float w = a.weight != nullptr ? load_as_f32<E>((const T*)a.weight + j) : 1.f;
      const float b = a.bias != nullptr ? load_as_f32<E>((const T*)a.bias + j) : 0.f;
      store_from_f32<E>((T*)a.out + r * d + j, (load_as_f32<E>(x + j) - mean) * rstd * w + b);
    }
  }
}
template <class E>
__global__ __launch_bounds__(1024) void norm_bwd_long_kernel(NormArgs a) {
  using T = typename E::T;
  __shared__ float s[32];
  const int d = a.d;
  const float inv_d = 1.f / (float)d;
  for (long long r = blockIdx.x; r < a.T; r += gridDim.x) {
    const T* x = (const T*)a.x + r * d;
    const T* dy = (const T*)a.dy + r * d;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float c1 = 0.f, c2 = 0.f;
    for (int j = threadIdx.x; j < d; j += 1024) {
      const float w = a.weight != nullptr ? load_as_f32<E>((const T*)a.weight + j) : 1.f;
      const float g = load_as_f32<E>(dy + j) * w;
      c1 += g;
      c2 += g * ((load_as_f32<E>(x + j) - mean) * rstd);
    }
    row_sum2<1024>(c1, c2, s);
    c1 *= inv_d;
    c2 *= inv_d;
    for (int j = threadIdx.x; j < d; j += 1024) {
      const float w = a.weight != nullptr ? load_as_f32<E>((const T*)a.weight + j) : 1.f;
      const float g = load_as_f32<E>(dy + j) * w;
      const float xh = (load_as_f32<E>(x + j) - mean) * rstd;
      store_from_f32<E>((T*)a.out + r * d + j, rstd * (g - c1 - xh * c2));
    }
  }
}
// Partial column sums of long_rows(T) rows: one thread per column.
__host__ __device__ inline int long_rows(int T) { return T <= 64 * 1024 ? 64 : (T - 1) / 1024 + 1; }
template <class E>
__global__ __launch_bounds__(256) void norm_cols_long_kernel(NormArgs a) {
  using T = typename E::T;
  const int j = blockIdx.x * 256 + threadIdx.x, d = a.d;
  if (j >= d) return;
  const int R = long_rows(a.T), r0 = blockIdx.y * R, r1 = r0 + min(R, a.T - r0);
  float dw = 0.f, db = 0.f;
  for (int r = r0; r < r1; ++r) {
    const float g = load_as_f32<E>((const T*)a.dy + (long long)r * d + j);
    dw += g * ((load_as_f32<E>((const T*)a.x + (long long)r * d + j) - a.mean[r]) * a.rstd[r]);
    db += g;
  }
  float* part = a.part + (long long)blockIdx.y * 2 * d;
  part[j] = dw;
  part[d + j] = db;
}

// dweight and dbias: column sums of the `chunks` partial rows, 32 columns per block, 32
// threads a column over the rows, then the 32 sums in order.
__global__ __launch_bounds__(1024) void norm_cols_kernel(NormArgs a, int chunks) {
  __shared__ float s[32][33];
  const int col = threadIdx.x & 31, g = threadIdx.x >> 5;
  const long long w2 = 2LL * a.d, j = (long long)blockIdx.x * 32 + col;
  float sum = 0.f;
  if (j < w2) {
#pragma unroll 8
    for (int p = g; p < chunks; p += 32) sum += a.part[p * w2 + j];
  }
  s[g][col] = sum;
  __syncthreads();
  if (g != 0 || j >= w2) return;
  sum = 0.f;
#pragma unroll
  for (int q = 0; q < 32; ++q) sum += s[q][col];
  float* out = j < a.d ? a.dweight : a.dbias;
  if (out != nullptr) out[j < a.d ? j : j - a.d] = sum;
}

// ---------------------------------------------------------------- launch rules
// The smallest (threads per row, chunks) that hold the row: one wavefront per row up to
// 4 chunks a lane, so small rows need no barrier, then 256 and 1024 threads.
struct NormPlan {
  int tpr, nch;  // nch = 0: the row does not fit registers
};
NormPlan norm_plan(int dtype, int d) {
  const int ch = dtype == 0 ? 4 : 8;
  static const int options[][2] = {{64, 1}, {64, 2}, {64, 4}, {256, 2}, {256, 4}, {1024, 2}};
  for (const auto& o : options)
    if ((long long)o[0] * o[1] * ch >= d) return NormPlan{o[0], o[1]};
  return NormPlan{1024, 0};
}

int norm_rows_per_block(const NormPlan& p) { return p.tpr < 256 ? 256 / p.tpr : 1; }

// Blocks of the forward (each takes rows in turn) and of the backward, whose
// every block also writes one partial row of 2d floats.
constexpr int kNormFwdBlocks = 2048, kNormBwdBlocks = 512;
unsigned norm_grid(const NormPlan& p, int T, int most) {
  const int rpb = norm_rows_per_block(p);
  return (unsigned)std::min<long long>(((long long)T + rpb - 1) / rpb, most);
}

template <class E, int TPR, int NCH, bool WHOLE>
hipError_t run_norm(bool bwd, bool dw, unsigned grid, const NormArgs& a, hipStream_t st) {
  const dim3 b(norm_threads<TPR>());
  if (!bwd) norm_fwd_kernel<E, TPR, NCH, WHOLE><<<grid, b, 0, st>>>(a);
  else if (dw) norm_bwd_kernel<E, TPR, NCH, WHOLE, true><<<grid, b, 0, st>>>(a);
  else norm_bwd_kernel<E, TPR, NCH, WHOLE, false><<<grid, b, 0, st>>>(a);
  return hipGetLastError();
}

template <class E, bool WHOLE>
hipError_t pick_norm(const NormPlan& p, bool bwd, bool dw, unsigned grid, const NormArgs& a,
                     hipStream_t st) {
  switch (p.tpr * 16 + p.nch) {
    case 64 * 16 + 1: return run_norm<E, 64, 1, WHOLE>(bwd, dw, grid, a, st);
    case 64 * 16 + 2: return run_norm<E, 64, 2, WHOLE>(bwd, dw, grid, a, st);
    case 64 * 16 + 4: return run_norm<E, 64, 4, WHOLE>(bwd, dw, grid, a, st);
    case 256 * 16 + 2: return run_norm<E, 256, 2, WHOLE>(bwd, dw, grid, a, st);
    case 256 * 16 + 4: return run_norm<E, 256, 4, WHOLE>(bwd, dw, grid, a, st);
    case 1024 * 16 + 2: return run_norm<E, 1024, 2, WHOLE>(bwd, dw, grid, a, st);
    default: return hipErrorInvalidValue;
  }
}

hipError_t run_plan(int dtype, const NormPlan& p, bool bwd, bool dw, unsigned grid,
                    const NormArgs& a, hipStream_t st) {
  if (dtype == 0)
    return a.d % ElemF32::kPerChunk == 0 ? pick_norm<ElemF32, true>(p, bwd, dw, grid, a, st)
                                         : pick_norm<ElemF32, false>(p, bwd, dw, grid, a, st);
  return a.d % ElemBF16::kPerChunk == 0 ? pick_norm<ElemBF16, true>(p, bwd, dw, grid, a, st)
                                        : pick_norm<ElemBF16, false>(p, bwd, dw, grid, a, st);
}

}  // namespace

hipError_t launch_layer_norm(int dtype, const NormArgs& a, hipStream_t st) {
  const NormPlan p = norm_plan(dtype, a.d);
  const unsigned grid = norm_grid(p, a.T, kNormFwdBlocks);
  if (p.nch != 0) return run_plan(dtype, p, false, false, grid, a, st);
  if (dtype == 0) norm_fwd_long_kernel<ElemF32><<<grid, 1024, 0, st>>>(a);
  else norm_fwd_long_kernel<ElemBF16><<<grid, 1024, 0, st>>>(a);
  return hipGetLastError();
}

int layer_norm_chunks(int dtype, int T, int d) {
  const NormPlan p = norm_plan(dtype, d);
  if (p.nch == 0) return T == 0 ? 0 : (T - 1) / long_rows(T) + 1;
  return (int)norm_grid(p, T, kNormBwdBlocks);
}

hipError_t launch_layer_norm_backward(int dtype, const NormArgs& a, hipStream_t st) {
  const NormPlan p = norm_plan(dtype, a.d);
  const bool dw = a.dweight != nullptr || a.dbias != nullptr;
  const int chunks = layer_norm_chunks(dtype, a.T, a.d);  // T = 0: none, so zero sums
  hipError_t e = hipSuccess;
  if (a.T == 0) {
  } else if (p.nch != 0) {
    e = run_plan(dtype, p, true, dw, norm_grid(p, a.T, kNormBwdBlocks), a, st);
  } else {
    const unsigned grid = norm_grid(p, a.T, kNormFwdBlocks);
    if (dtype == 0) norm_bwd_long_kernel<ElemF32><<<grid, 1024, 0, st>>>(a);
    else norm_bwd_long_kernel<ElemBF16><<<grid, 1024, 0, st>>>(a);
    e = hipGetLastError();
    if (e == hipSuccess && dw) {
      const dim3 g((a.d + 255) / 256, chunks);
      if (dtype == 0) norm_cols_long_kernel<ElemF32><<<g, 256, 0, st>>>(a);
      else norm_cols_long_kernel<ElemBF16><<<g, 256, 0, st>>>(a);
      e = hipGetLastError();
    }
  }
  if (e != hipSuccess || !dw) return e;
  norm_cols_kernel<<<(unsigned)((2LL * a.d + 31) / 32), 1024, 0, st>>>(a, chunks);
  return hipGetLastError();
}

}  // namespace moe
