// Quantising to 8 bits with one float32 scale for each block of 128 (f8.h) and reading it back
// (gfx950): rows [T][d] with a scale for each 128 columns of a row, as the products of 8-bit
// operands take their rows, and matrices [E][n][k] with a scale for each 128 x 128, as they take
// an expert's weights (one scale then serves both contractions, over k and over n).
//
// Bound by HBM: every value is read once, held in registers until its block's largest is known,
// and written once.  A row's block is one 16-byte chunk of 16 (bfloat16) or 32 (float32) lanes;
// a matrix's block is a workgroup's 256 threads, each with its 16 (float32) or 8 chunks in flight.
// The rounding to 8 bits is the operator's own; scales and quotients are float32.
//
// Measured: 28672 x 896 bfloat16 rows to e5m2 16.5 us (4.7 TB/s; 15.1 with the launches of calls
// back to back overlapping); 64 matrices of 1408 x 2048 float32 160 us (5.8 TB/s: four of five bytes
// are reads, which run above a copy's rate); 28672 x 896 e4m3 rows read back to bfloat16 15.6 us (5.0 TB/s).
#include <algorithm>

#include "f8.h"
#include "ops_internal.h"
#include "row_chunks.h"

namespace moe {
namespace {

// Blocks of 128 columns, in order over the rows of `rows` rows (blocks * rows < 2^31).
template <class E, bool WHOLE, int Q>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const typename E::T* __restrict__ x,
                                                            int rows, int d, int blocks,
                                                            uint8_t* __restrict__ q,
                                                            float* __restrict__ scales) {
  using K = Chunk<E, WHOLE>;
  constexpr int CH = K::CH, G = kF8Block / CH, PER = 256 / G;
  const unsigned b = blockIdx.x * PER + threadIdx.x / G;
  const unsigned r = b / (unsigned)blocks;
  if (r >= (unsigned)rows) return;  // a group of G lanes leaves together
  const int j = (int)(b - r * blocks) * kF8Block + (threadIdx.x % G) * CH;
  float f[CH];
  K::unpack(j < d ? K::load(x + (size_t)r * d, j, d) : u32x4{0u, 0u, 0u, 0u}, f);
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < CH; ++e) top = fmaxf(top, finite_abs(f[e]));
  const F8Scale s = f8_scale<Q>(group_max<G>(top));
  if (threadIdx.x % G == 0) scales[b] = s.scale;
#pragma unroll
  for (int e = 0; e < CH; ++e) f[e] = f8_scaled(f[e], s);
  if (j < d) f8_store<Q, CH>(q + (size_t)r * d, j, d, WHOLE, f);
}

// One 128 x 128 block per workgroup; a thread holds the same columns of every RPP-th row.
template <class E, bool WHOLE, int Q>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const typename E::T* __restrict__ w,
                                                              int n, int k, int nb, int kb,
                                                              uint8_t* __restrict__ q,
                                                              float* __restrict__ scales) {
  using K = Chunk<E, WHOLE>;
  constexpr int CH = K::CH, G = kF8Block / CH, RPP = 256 / G, P = kF8Block / RPP;
  __shared__ float s_top[4];
  const unsigned block = blockIdx.x, m = block / (unsigned)kb;
  const int j = (int)(block - m * kb) * kF8Block + (threadIdx.x % G) * CH;
  const unsigned e = m / (unsigned)nb;
  const int i0 = (int)(m - e * nb) * kF8Block + threadIdx.x / G;
  const size_t first = (size_t)e * n;
  u32x4 v[P];
  float top = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i = i0 + p * RPP;
    v[p] = i < n && j < k ? K::load(w + (first + i) * k, j, k) : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float f[CH];
    K::unpack(v[p], f);
#pragma unroll
    for (int c = 0; c < CH; ++c) top = fmaxf(top, finite_abs(f[c]));
  }
  top = group_max<64>(top);
  if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top;
  __syncthreads();
  const F8Scale s =
      f8_scale<Q>(fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3])));
  if (threadIdx.x == 0) scales[block] = s.scale;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i = i0 + p * RPP;
    if (i >= n || j >= k) continue;
    float f[CH];
    K::unpack(v[p], f);
#pragma unroll
    for (int c = 0; c < CH; ++c) f[c] = f8_scaled(f[c], s);
    f8_store<Q, CH>(q + (first + i) * k, j, k, WHOLE, f);
  }
}

// Four columns a thread.
template <class E, int Q>
__global__ __launch_bounds__(256) void dequantize_rows_kernel(const uint8_t* __restrict__ q,
                                                              const float* __restrict__ scales,
                                                              int rows, int d, int blocks,
                                                              typename E::T* __restrict__ x) {
  const unsigned b = blockIdx.x * 8 + threadIdx.x / 32, r = b / (unsigned)blocks;
  if (r >= (unsigned)rows) return;
  const int j = (int)(b - r * blocks) * kF8Block + (threadIdx.x % 32) * 4;
  if (j >= d) return;
  const float s = scales[b];
  const uint8_t* from = q + (size_t)r * d;
  typename E::T* to = x + (size_t)r * d;
  if (d % 4 == 0) {
    const uint32_t v = *(const uint32_t*)(from + j);
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = f8_value<Q>((v >> (8 * e)) & 0xff) * s;
    if constexpr (sizeof(typename E::T) == 4) *(f32x4*)(to + j) = f32x4{f[0], f[1], f[2], f[3]};
    else *(uint2*)(to + j) = uint2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < d) store_from_f32<E>(to + j + e, f8_value<Q>(from[j + e]) * s);
  }
}

// Rows per launch, so that the blocks of 128 columns and the threads of a launch stay below
// 2^31 and 2^32.
int rows_per_launch(int T, int blocks) {
  return (int)std::max(1LL, std::min<long long>(T, (1LL << 26) / blocks));
}

template <class E, int Q>
void quantize_rows_of(const void* x, int rows, int d, int blocks, uint8_t* q, float* scales,
                      hipStream_t st) {
  constexpr int PER = 256 * E::kPerChunk / kF8Block;
  const unsigned grid = (unsigned)(((long long)rows * blocks + PER - 1) / PER);
  if (d % E::kPerChunk == 0)
    quantize_rows_kernel<E, true, Q>
        <<<grid, 256, 0, st>>>((const typename E::T*)x, rows, d, blocks, q, scales);
  else
    quantize_rows_kernel<E, false, Q>
        <<<grid, 256, 0, st>>>((const typename E::T*)x, rows, d, blocks, q, scales);
}
template <class E, int Q>
void quantize_blocks_of(const void* w, int E_, int n, int k, uint8_t* q, float* scales,
                        hipStream_t st) {
  const int nb = f8_blocks(n), kb = f8_blocks(k);
  const unsigned grid = (unsigned)((long long)E_ * nb * kb);
  if (k % E::kPerChunk == 0)
    quantize_blocks_kernel<E, true, Q>
        <<<grid, 256, 0, st>>>((const typename E::T*)w, n, k, nb, kb, q, scales);
  else
    quantize_blocks_kernel<E, false, Q>
        <<<grid, 256, 0, st>>>((const typename E::T*)w, n, k, nb, kb, q, scales);
}

template <class E, int Q>
void dequantize_rows_of(const uint8_t* q, const float* scales, int rows, int d, int blocks, void* x,
                        hipStream_t st) {
  const unsigned grid = (unsigned)(((long long)rows * blocks + 7) / 8);
  dequantize_rows_kernel<E, Q>
      <<<grid, 256, 0, st>>>(q, scales, rows, d, blocks, (typename E::T*)x);
}

}  // namespace

hipError_t launch_quantize_rows(int dtype, int f8, const void* x, int T, int d, void* q,
                                float* scales, hipStream_t st) {
  const int blocks = f8_blocks(d), most = rows_per_launch(T, blocks);
  const size_t es = dtype == 0 ? 4 : 2;
  const auto run = dtype == 0 ? (f8 == F8_E4M3 ? quantize_rows_of<ElemF32, F8_E4M3>
                                               : quantize_rows_of<ElemF32, F8_E5M2>)
                              : (f8 == F8_E4M3 ? quantize_rows_of<ElemBF16, F8_E4M3>
                                               : quantize_rows_of<ElemBF16, F8_E5M2>);
  for (int r = 0, rows; r < T; r += rows) {
    rows = std::min(most, T - r);
    run((const char*)x + (size_t)r * d * es, rows, d, blocks, (uint8_t*)q + (size_t)r * d,
        scales + (size_t)r * blocks, st);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_quantize_blocks(int dtype, int f8, const void* w, int E, int n, int k, void* q,
                                  float* scales, hipStream_t st) {
  const auto run = dtype == 0 ? (f8 == F8_E4M3 ? quantize_blocks_of<ElemF32, F8_E4M3>
                                               : quantize_blocks_of<ElemF32, F8_E5M2>)
                              : (f8 == F8_E4M3 ? quantize_blocks_of<ElemBF16, F8_E4M3>
                                               : quantize_blocks_of<ElemBF16, F8_E5M2>);
  run(w, E, n, k, (uint8_t*)q, scales, st);
  return hipGetLastError();
}

hipError_t launch_dequantize_rows(int f8, int dtype, const void* q, const float* scales, int T,
                                  int d, void* x, hipStream_t st) {
  const int blocks = f8_blocks(d), most = rows_per_launch(T, blocks);
  const size_t es = dtype == 0 ? 4 : 2;
  const auto run = dtype == 0 ? (f8 == F8_E4M3 ? dequantize_rows_of<ElemF32, F8_E4M3>
                                               : dequantize_rows_of<ElemF32, F8_E5M2>)
                              : (f8 == F8_E4M3 ? dequantize_rows_of<ElemBF16, F8_E4M3>
                                               : dequantize_rows_of<ElemBF16, F8_E5M2>);
  for (int r = 0, rows; r < T; r += rows) {
    rows = std::min(most, T - r);
    run((const uint8_t*)q + (size_t)r * d, scales + (size_t)r * blocks, rows, d, blocks,
        (char*)x + (size_t)r * d * es, st);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
