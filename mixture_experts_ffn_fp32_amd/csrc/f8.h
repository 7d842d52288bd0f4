// 8-bit floating point with one float32 scale for each block of 128 values (gfx950):
//   scale = max |v| / most,  q = round(v / scale)      over the block's finite values,
// most being the type's largest value (e4m3 448, e5m2 57344); a block of zeros has scale 1.  A
// value that is not finite becomes NaN and takes no other value's scale.  Scales stay at or
// above 2^-126, so that 1 / scale and scale itself are normal float32 numbers.
#pragma once

#include <float.h>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kF8Block = 128;
enum : int { F8_NONE = 0, F8_E4M3 = 1, F8_E5M2 = 2 };

template <int Q>
__host__ __device__ constexpr float f8_most() {
  return Q == F8_E4M3 ? 448.f : 57344.f;
}
__host__ __device__ inline int f8_blocks(int n) { return n / kF8Block + (n % kF8Block != 0); }

// |v|, or 0 where v is not finite.
__device__ __forceinline__ float finite_abs(float v) {
  const float m = fabsf(v);
  return m <= FLT_MAX ? m : 0.f;
}

struct F8Scale {
  float scale, inv;
};
template <int Q>
__device__ __forceinline__ F8Scale f8_scale(float top) {
  F8Scale s;
  s.scale = top > 0.f ? fmaxf(top / f8_most<Q>(), FLT_MIN) : 1.f;
  s.inv = 1.f / s.scale;
  return s;
}
// v / scale as float32 division rounds it, before its rounding to 8 bits: the product with the
// rounded reciprocal, and its rest divided once more.  (The product alone is off by an ulp now
// and then, which moves values that lie between two of 8 bits, and bfloat16 values often do.)
// The block's largest value is `most` but for the scale's own rounding, which rounds back to it.
__device__ __forceinline__ float f8_scaled(float v, const F8Scale& s) {
  const float q = v * s.inv;
  return fabsf(v) <= FLT_MAX ? fmaf(fmaf(-q, s.scale, v), s.inv, q) : __builtin_nanf("");
}
// The value of a byte, exactly.
template <int Q>
__device__ __forceinline__ float f8_value(uint32_t byte) {
  if constexpr (Q == F8_E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
  else return __builtin_amdgcn_cvt_f32_bf8((int)byte, 0);
}
// Four values, rounded to nearest even, lowest byte first.
template <int Q>
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  int w = 0;
  if constexpr (Q == F8_E4M3) {
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  } else {
    w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
  }
  return (uint32_t)w;
}

// Largest of v over groups of G lanes (a power of two up to 64), in every lane of its group.
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int k = G / 2; k > 0; k >>= 1) v = fmaxf(v, __shfl_xor(v, k));
  return v;
}

// CH (4 or 8) consecutive values of a row of width d from column j, as bytes.  Rows of any
// width start at any byte; the row's last chunk is written byte by byte.
typedef uint32_t u32_at1 __attribute__((aligned(1)));
template <int Q, int CH>
__device__ __forceinline__ void f8_store(uint8_t* __restrict__ row, int j, int d, bool whole,
                                         const float (&v)[CH]) {
  uint32_t w[CH / 4];
#pragma unroll
  for (int i = 0; i < CH / 4; ++i)
    w[i] = f8_pack4<Q>(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  if (whole) {  // rows of whole chunks: aligned
    if constexpr (CH == 8) *(uint2*)(row + j) = uint2{w[0], w[1]};
    else *(uint32_t*)(row + j) = w[0];
  } else if (j + CH <= d) {
#pragma unroll
    for (int i = 0; i < CH / 4; ++i) *(u32_at1*)(row + j + 4 * i) = w[i];
  } else {
#pragma unroll
    for (int e = 0; e < CH; ++e)
      if (j + e < d) row[j + e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
  }
}

}  // namespace
}  // namespace moe
