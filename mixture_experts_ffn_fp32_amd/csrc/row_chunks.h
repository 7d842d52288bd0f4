// Rows held in registers by the threads of a block, 16 bytes a thread and chunk: loads and
// stores of chunks at any width, and sums over a row's threads.  Shared by the norms and the
// quantising kernels (gfx950).
#pragma once

#include <type_traits>

#include "lds_dma.h"
#include "moe_internal.h"

namespace moe {
namespace {

// A 16-byte chunk of a row: CH elements as raw bits.  Rows of any width start at any
// element, so the accesses claim an element's alignment only (the hardware takes
// 16-byte accesses at any address; where the width is a whole number of chunks they are
// aligned anyway).  The row's last chunk is read and written element by element unless
// WHOLE says that the width is a multiple of a chunk (8192 x 2048 bfloat16: 15.2 ->
// 14.4 us without that branch).
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
template <class E, bool WHOLE>
struct Chunk {
  static constexpr int CH = E::kPerChunk;
  using T = typename E::T;
  using V = std::conditional_t<sizeof(T) == 4, u32x4_at4, u32x4_at2>;

  static __device__ __forceinline__ u32x4 load(const T* __restrict__ row, int j, int d) {
    if (WHOLE || j + CH <= d) return *(const V*)(row + j);
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < CH; ++e)
      if (j + e < d) {
        if constexpr (sizeof(T) == 4) v[e] = __float_as_uint(row[j + e]);
        else v[e >> 1] |= (uint32_t)row[j + e] << (16 * (e & 1));
      }
    return v;
  }
  static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[CH]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < CH; ++i) f[i] = __uint_as_float(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[CH]) {
    u32x4 v;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < CH; ++i) v[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
    return v;
  }
  static __device__ __forceinline__ void store(T* __restrict__ row, int j, int d,
                                               const float (&f)[CH]) {
    const u32x4 v = pack(f);
    if (WHOLE || j + CH <= d) {
      *(V*)(row + j) = v;
      return;
    }
#pragma unroll
    for (int e = 0; e < CH; ++e)
      if (j + e < d) {
        if constexpr (sizeof(T) == 4) row[j + e] = __uint_as_float(v[e]);
        else row[j + e] = (T)(v[e >> 1] >> (16 * (e & 1)));
      }
  }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
  return v;
}

// Sums of A and B over the TPR threads of a row (TPR = 64: one wavefront; else the
// block).  `s` holds two floats per wavefront; the two barriers let the caller
// reuse it at once.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& A, float& B, float* s) {
  A = wave_sum(A);
  B = wave_sum(B);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      s[2 * w] = A;
      s[2 * w + 1] = B;
    }
    __syncthreads();
    A = B = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      A += s[2 * i];
      B += s[2 * i + 1];
    }
    __syncthreads();
  }
}

template <int TPR>
constexpr int norm_threads() {
  return TPR < 256 ? 256 : TPR;
}

}  // namespace
}  // namespace moe
