// Root-mean-square norm with the residual's addition in front of it, forward and backward, and
// its output in 8 bits for products of 8-bit operands (gfx950):
//
//   h = x + residual (rounded to the storage type: the stream that the next layer reads)
//   rstd_t = 1 / sqrt((1/d) sum_j h_tj^2 + eps),  hh = h rstd,  y = hh w
//   g = dy w:  dx = rstd (g - hh mean_j(g hh)) + dh,  dw = sum_t dy hh
//
// dx is the gradient of x and of the residual alike; dh is what reaches h from later layers.
// An 8-bit y has one scale for each 128 columns of a row (f8.h), taken from the float32 values,
// which are rounded once, to 8 bits.
//
// Both directions are bound by HBM, each operand once in or out: a row stays in registers
// between its reduction and its output, TPR threads holding NCH chunks of 16 bytes each.  A
// block of 128 columns is 16 (bfloat16) or 32 (float32) neighbouring lanes' chunk, so its
// largest value needs no LDS.  The weight's gradient is added up in registers over the rows a
// block takes and joined from the blocks' partial rows in a fixed order by a second launch.
//
// Measured (a copy of 1 GiB runs at 5.1 TB/s here): 8192 x 2048 bfloat16 with residual to e4m3, h
// kept, 24.7 us (4.8 TB/s); 3001 x 1283 float32 12.4 us (5.0 TB/s); one row of 2048 4.5 us, which is
// a launch's own time; backward of 16384 x 4096 bfloat16 with dh 98.5 us (5.5 TB/s) and 4.7 for the
// 512 partial rows.  The rounding of h to the storage type is the one that the next layer reads;
// the sums are of that h, in float32, so that the backward finds the same values.
#include <algorithm>

#include "f8.h"
#include "ops_internal.h"
#include "row_chunks.h"

namespace moe {
namespace {

// Chunk c of this thread starts at column (c * TPR + i) * CH (i: the thread's index in
// its row).  A chunk's elements past the row's end are zeros.
template <class E, int TPR, int NCH, bool WHOLE, int Q>
__global__ __launch_bounds__(norm_threads<TPR>()) void rms_fwd_kernel(RmsArgs a) {
  using K = Chunk<E, WHOLE>;
  using T = typename E::T;
  constexpr int CH = K::CH, G = kF8Block / CH;
  __shared__ float s[2 * TPR / 64];
  constexpr int RPB = norm_threads<TPR>() / TPR;  // rows per block
  const int i = threadIdx.x % TPR, d = a.d;
  const float inv_d = 1.f / (float)d;
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
    u32x4 hv[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * TPR + i) * CH;
      hv[c] = j < d ? K::load(x, j, d) : u32x4{0u, 0u, 0u, 0u};
    }
    if (a.residual != nullptr) {
      const T* res = (const T*)a.residual + r * d;
      u32x4 rv[NCH];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int j = (c * TPR + i) * CH;
        rv[c] = j < d ? K::load(res, j, d) : u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        float f[CH], g[CH];
        K::unpack(hv[c], f);
        K::unpack(rv[c], g);
#pragma unroll
        for (int e = 0; e < CH; ++e) f[e] += g[e];
        hv[c] = K::pack(f);
      }
    }
    if (a.h != nullptr) {
      T* h = (T*)a.h + r * d;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int j = (c * TPR + i) * CH;
        float f[CH];
        K::unpack(hv[c], f);
        if (j < d) K::store(h, j, d, f);
      }
    }
    float sq = 0.f, zero = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float f[CH];
      K::unpack(hv[c], f);
#pragma unroll
      for (int e = 0; e < CH; ++e) sq += f[e] * f[e];
    }
    row_sum2<TPR>(sq, zero, s);
    const float rstd = 1.f / sqrtf(sq * inv_d + a.eps);
    if (i == 0 && a.rstd != nullptr) a.rstd[r] = rstd;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * TPR + i) * CH;
      float f[CH], w[CH];
      K::unpack(hv[c], f);
      K::unpack(wv[c], w);
#pragma unroll
      for (int e = 0; e < CH; ++e) f[e] = f[e] * rstd * w[e];
      if constexpr (Q == F8_NONE) {
        if (j < d) K::store((T*)a.out + r * d, j, d, f);
      } else {
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < CH; ++e) top = fmaxf(top, finite_abs(f[e]));
        const F8Scale sc = f8_scale<Q>(group_max<G>(top));
        if (j < d) {
          if (i % G == 0) a.scales[r * a.blocks + j / kF8Block] = sc.scale;
#pragma unroll
          for (int e = 0; e < CH; ++e) f[e] = f8_scaled(f[e], sc);
          f8_store<Q, CH>((uint8_t*)a.out + r * d, j, d, WHOLE, f);
        }
      }
    }
  }
}

// DW: also the block's partial weight gradient (part row blockIdx.x).
template <class E, int TPR, int NCH, bool WHOLE, bool DW>
__global__ __launch_bounds__(norm_threads<TPR>()) void rms_bwd_kernel(RmsArgs a) {
  using K = Chunk<E, WHOLE>;
  using T = typename E::T;
  constexpr int CH = K::CH;
  constexpr int RPB = norm_threads<TPR>() / TPR;
  __shared__ float s[2 * TPR / 64];
  __shared__ float s_col[(DW && RPB > 1) ? RPB * TPR * CH : 1];
  const int i = threadIdx.x % TPR, d = a.d;
  const float inv_d = 1.f / (float)d;
  float dw[DW ? NCH : 1][CH];
  if constexpr (DW) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int e = 0; e < CH; ++e) dw[c][e] = 0.f;
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
    u32x4 xv[NCH], yv[NCH], ev[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * TPR + i) * CH;
      xv[c] = j < d ? K::load(x, j, d) : u32x4{0u, 0u, 0u, 0u};
      yv[c] = j < d ? K::load(dy, j, d) : u32x4{0u, 0u, 0u, 0u};
      ev[c] = a.dh != nullptr && j < d ? K::load((const T*)a.dh + r * d, j, d)
                                       : u32x4{0u, 0u, 0u, 0u};
    }
    const float rstd = a.rstd[r];
    float c2 = 0.f, zero = 0.f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float f[CH], g[CH], w[CH];
      K::unpack(xv[c], f);
      K::unpack(yv[c], g);
      K::unpack(wv[c], w);
#pragma unroll
      for (int e = 0; e < CH; ++e) {  // (past the row's end dy = 0)
        const float xh = f[e] * rstd;
        c2 += g[e] * w[e] * xh;
        if constexpr (DW) dw[c][e] += g[e] * xh;
      }
    }
    row_sum2<TPR>(c2, zero, s);
    c2 *= inv_d;
    T* dx = (T*)a.out + r * d;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * TPR + i) * CH;
      if (j >= d) continue;
      float f[CH], g[CH], w[CH], more[CH];
      K::unpack(xv[c], f);
      K::unpack(yv[c], g);
      K::unpack(wv[c], w);
      K::unpack(ev[c], more);
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        const float v = rstd * (g[e] * w[e] - f[e] * rstd * c2);
        f[e] = v + more[e];
      }
      K::store(dx, j, d, f);
    }
  }
  if constexpr (DW) {
    float* part = a.part + (long long)blockIdx.x * d;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int j = (c * TPR + i) * CH;
      float f[CH];
#pragma unroll
      for (int e = 0; e < CH; ++e) f[e] = dw[c][e];
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
            *(f32x4*)(part + j + e) = f32x4{f[e], f[e + 1], f[e + 2], f[e + 3]};
        } else {
#pragma unroll
          for (int e = 0; e < CH; ++e)
            if (!WHOLE && j + e < d) part[j + e] = f[e];
        }
      }
    }
  }
}

// Rows too long for registers: one block of 1024 threads per row, the row read again from the
// caches (h, as the thread itself wrote it, which may be x's or the residual's place).
template <class E>
__device__ __forceinline__ float rms_h(const RmsArgs& a, long long at) {
  const float x = load_as_f32<E>((const typename E::T*)a.x + at);
  if (a.residual == nullptr) return x;
  typename E::T sum;
  store_from_f32<E>(&sum, x + load_as_f32<E>((const typename E::T*)a.residual + at));
  return load_as_f32<E>(&sum);
}
template <class E, int Q>
__global__ __launch_bounds__(1024) void rms_fwd_long_kernel(RmsArgs a) {
  using T = typename E::T;
  __shared__ float s[32];
  const int d = a.d, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const float inv_d = 1.f / (float)d;
  for (long long r = blockIdx.x; r < a.T; r += gridDim.x) {
    float sq = 0.f, zero = 0.f;
    // a wavefront's columns are whole blocks of 128, two columns a lane
    for (int j0 = wave * kF8Block; j0 < d; j0 += 16 * kF8Block)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = j0 + 64 * e + lane;
        if (j >= d) continue;
        const float f = rms_h<E>(a, r * d + j);
        if (a.h != nullptr) store_from_f32<E>((T*)a.h + r * d + j, f);
        sq += f * f;
      }
    row_sum2<1024>(sq, zero, s);
    const float rstd = 1.f / sqrtf(sq * inv_d + a.eps);
    if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[r] = rstd;
    for (int j0 = wave * kF8Block; j0 < d; j0 += 16 * kF8Block) {
      float y[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = j0 + 64 * e + lane;
        y[e] = 0.f;
        if (j >= d) continue;
        const float f = a.h != nullptr ? load_as_f32<E>((const T*)a.h + r * d + j)
                                       : rms_h<E>(a, r * d + j);
        y[e] = f * rstd * (a.weight != nullptr ? load_as_f32<E>((const T*)a.weight + j) : 1.f);
      }
      if constexpr (Q == F8_NONE) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = j0 + 64 * e + lane;
          if (j < d) store_from_f32<E>((T*)a.out + r * d + j, y[e]);
        }
      } else {
        const F8Scale sc =
            f8_scale<Q>(group_max<64>(fmaxf(finite_abs(y[0]), finite_abs(y[1]))));
        if (lane == 0) a.scales[r * a.blocks + j0 / kF8Block] = sc.scale;
        const uint32_t w = f8_pack4<Q>(f8_scaled(y[0], sc), f8_scaled(y[1], sc), 0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = j0 + 64 * e + lane;
          if (j < d) ((uint8_t*)a.out)[r * d + j] = (uint8_t)(w >> (8 * e));
        }
      }
    }
  }
}
template <class E>
__global__ __launch_bounds__(1024) void rms_bwd_long_kernel(RmsArgs a) {
  using T = typename E::T;
  __shared__ float s[32];
  const int d = a.d;
  const float inv_d = 1.f / (float)d;
  for (long long r = blockIdx.x; r < a.T; r += gridDim.x) {
    const T* x = (const T*)a.x + r * d;
    const T* dy = (const T*)a.dy + r * d;
    const float rstd = a.rstd[r];
    float c2 = 0.f, zero = 0.f;
    for (int j = threadIdx.x; j < d; j += 1024) {
      const float w = a.weight != nullptr ? load_as_f32<E>((const T*)a.weight + j) : 1.f;
      c2 += load_as_f32<E>(dy + j) * w * (load_as_f32<E>(x + j) * rstd);
    }
    row_sum2<1024>(c2, zero, s);
    c2 *= inv_d;
    for (int j = threadIdx.x; j < d; j += 1024) {
      const float w = a.weight != nullptr ? load_as_f32<E>((const T*)a.weight + j) : 1.f;
      const float more = a.dh != nullptr ? load_as_f32<E>((const T*)a.dh + r * d + j) : 0.f;
      const float v = rstd * (load_as_f32<E>(dy + j) * w - load_as_f32<E>(x + j) * rstd * c2);
      store_from_f32<E>((T*)a.out + r * d + j, v + more);
    }
  }
}
// Partial column sums of rms_long_rows(T) rows: one thread per column.
__host__ __device__ inline int rms_long_rows(int T) {
  return T <= 64 * 1024 ? 64 : (T - 1) / 1024 + 1;
}
template <class E>
__global__ __launch_bounds__(256) void rms_cols_long_kernel(RmsArgs a) {
  using T = typename E::T;
  const int j = blockIdx.x * 256 + threadIdx.x, d = a.d;
  if (j >= d) return;
  const int R = rms_long_rows(a.T), r0 = blockIdx.y * R, r1 = r0 + min(R, a.T - r0);
  float dw = 0.f;
  for (int r = r0; r < r1; ++r)
    dw += load_as_f32<E>((const T*)a.dy + (long long)r * d + j) *
          (load_as_f32<E>((const T*)a.x + (long long)r * d + j) * a.rstd[r]);
  a.part[(long long)blockIdx.y * d + j] = dw;
}

// dweight: column sums of the `chunks` partial rows, 32 columns per block, 32 threads a
// column over the rows, then the 32 sums in order.
__global__ __launch_bounds__(1024) void rms_cols_kernel(RmsArgs a, int chunks) {
  __shared__ float s[32][33];
  const int col = threadIdx.x & 31, g = threadIdx.x >> 5;
  const long long j = (long long)blockIdx.x * 32 + col;
  float sum = 0.f;
  if (j < a.d) {
#pragma unroll 8
    for (int p = g; p < chunks; p += 32) sum += a.part[(long long)p * a.d + j];
  }
  s[g][col] = sum;
  __syncthreads();
  if (g != 0 || j >= a.d) return;
  sum = 0.f;
#pragma unroll
  for (int q = 0; q < 32; ++q) sum += s[q][col];
  a.dweight[j] = sum;
}

// ---------------------------------------------------------------- launch rules
// The smallest (threads per row, chunks) that hold the row, as for layer norm.
struct RmsPlan {
  int tpr, nch;  // nch = 0: the row does not fit registers
};
RmsPlan rms_plan(int dtype, int d) {
  const int ch = dtype == 0 ? 4 : 8;
  static const int options[][2] = {{64, 1}, {64, 2}, {64, 4}, {256, 2}, {256, 4}, {1024, 2}};
  for (const auto& o : options)
    if ((long long)o[0] * o[1] * ch >= d) return RmsPlan{o[0], o[1]};
  return RmsPlan{1024, 0};
}

// Blocks of the forward (each takes rows in turn) and of the backward, whose every block
// also writes one partial row of d floats.
constexpr int kRmsFwdBlocks = 2048, kRmsBwdBlocks = 512;
unsigned rms_grid(const RmsPlan& p, int T, int most) {
  const int rpb = p.tpr < 256 ? 256 / p.tpr : 1;
  return (unsigned)std::min<long long>(((long long)T + rpb - 1) / rpb, most);
}

enum : int { RMS_FWD = 0, RMS_BWD = 1 };
template <class E, int TPR, int NCH, bool WHOLE>
hipError_t run_rms(int dir, int q, unsigned grid, const RmsArgs& a, hipStream_t st) {
  const dim3 b(norm_threads<TPR>());
  if (dir == RMS_BWD) {
    if (a.dweight != nullptr) rms_bwd_kernel<E, TPR, NCH, WHOLE, true><<<grid, b, 0, st>>>(a);
    else rms_bwd_kernel<E, TPR, NCH, WHOLE, false><<<grid, b, 0, st>>>(a);
  } else if (q == F8_NONE) rms_fwd_kernel<E, TPR, NCH, WHOLE, F8_NONE><<<grid, b, 0, st>>>(a);
  else if (q == F8_E4M3) rms_fwd_kernel<E, TPR, NCH, WHOLE, F8_E4M3><<<grid, b, 0, st>>>(a);
  else rms_fwd_kernel<E, TPR, NCH, WHOLE, F8_E5M2><<<grid, b, 0, st>>>(a);
  return hipGetLastError();
}
template <class E, bool WHOLE>
hipError_t pick_rms(const RmsPlan& p, int dir, int q, unsigned grid, const RmsArgs& a,
                    hipStream_t st) {
  switch (p.tpr * 16 + p.nch) {
    case 64 * 16 + 1: return run_rms<E, 64, 1, WHOLE>(dir, q, grid, a, st);
    case 64 * 16 + 2: return run_rms<E, 64, 2, WHOLE>(dir, q, grid, a, st);
    case 64 * 16 + 4: return run_rms<E, 64, 4, WHOLE>(dir, q, grid, a, st);
    case 256 * 16 + 2: return run_rms<E, 256, 2, WHOLE>(dir, q, grid, a, st);
    case 256 * 16 + 4: return run_rms<E, 256, 4, WHOLE>(dir, q, grid, a, st);
    case 1024 * 16 + 2: return run_rms<E, 1024, 2, WHOLE>(dir, q, grid, a, st);
    default: return hipErrorInvalidValue;
  }
}
hipError_t plan_rms(int dtype, const RmsPlan& p, int dir, int q, unsigned grid, const RmsArgs& a,
                    hipStream_t st) {
  if (dtype == 0)
    return a.d % ElemF32::kPerChunk == 0 ? pick_rms<ElemF32, true>(p, dir, q, grid, a, st)
                                         : pick_rms<ElemF32, false>(p, dir, q, grid, a, st);
  return a.d % ElemBF16::kPerChunk == 0 ? pick_rms<ElemBF16, true>(p, dir, q, grid, a, st)
                                        : pick_rms<ElemBF16, false>(p, dir, q, grid, a, st);
}
template <class E>
void long_rms(int q, unsigned grid, const RmsArgs& a, hipStream_t st) {
  if (q == F8_NONE) rms_fwd_long_kernel<E, F8_NONE><<<grid, 1024, 0, st>>>(a);
  else if (q == F8_E4M3) rms_fwd_long_kernel<E, F8_E4M3><<<grid, 1024, 0, st>>>(a);
  else rms_fwd_long_kernel<E, F8_E5M2><<<grid, 1024, 0, st>>>(a);
}

}  // namespace

hipError_t launch_rms_norm(int dtype, int f8, RmsArgs a, hipStream_t st) {
  const RmsPlan p = rms_plan(dtype, a.d);
  const unsigned grid = rms_grid(p, a.T, kRmsFwdBlocks);
  a.blocks = f8_blocks(a.d);
  if (p.nch != 0) return plan_rms(dtype, p, RMS_FWD, f8, grid, a, st);
  if (dtype == 0) long_rms<ElemF32>(f8, grid, a, st);
  else long_rms<ElemBF16>(f8, grid, a, st);
  return hipGetLastError();
}

int rms_norm_chunks(int dtype, int T, int d) {
  const RmsPlan p = rms_plan(dtype, d);
  if (p.nch == 0) return T == 0 ? 0 : (T - 1) / rms_long_rows(T) + 1;
  return (int)rms_grid(p, T, kRmsBwdBlocks);
}

hipError_t launch_rms_norm_backward(int dtype, const RmsArgs& a, hipStream_t st) {
  const RmsPlan p = rms_plan(dtype, a.d);
  const int chunks = rms_norm_chunks(dtype, a.T, a.d);  // T = 0: none, so zero sums
  hipError_t e = hipSuccess;
  if (a.T == 0) {
  } else if (p.nch != 0) {
    e = plan_rms(dtype, p, RMS_BWD, F8_NONE, rms_grid(p, a.T, kRmsBwdBlocks), a, st);
  } else {
    // the column sums first: dx may stand in dh's place, but never in x's or dy's
    if (a.dweight != nullptr) {
      const dim3 g((a.d + 255) / 256, chunks);
      if (dtype == 0) rms_cols_long_kernel<ElemF32><<<g, 256, 0, st>>>(a);
      else rms_cols_long_kernel<ElemBF16><<<g, 256, 0, st>>>(a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const unsigned grid = rms_grid(p, a.T, kRmsFwdBlocks);
    if (dtype == 0) rms_bwd_long_kernel<ElemF32><<<grid, 1024, 0, st>>>(a);
    else rms_bwd_long_kernel<ElemBF16><<<grid, 1024, 0, st>>>(a);
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.dweight == nullptr) return e;
  rms_cols_kernel<<<(unsigned)((a.d + 31LL) / 32), 1024, 0, st>>>(a, chunks);
  return hipGetLastError();
}

}  // namespace moe
