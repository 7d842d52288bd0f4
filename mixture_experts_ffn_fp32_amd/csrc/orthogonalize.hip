// Orthogonalised update of weight gradients by Newton-Schulz products (gfx950),
// as the Muon optimiser applies it to each matrix parameter, here to every
// expert's block of the layer's weight gradients (DeepSeekMoE paper summary,
// papercache.org, sec. 3.2: W_gate, W_up, W_down per expert) in one call:
//
//   X_0 = G / (|G|_F + eps),  then `steps` times
//   A = X X^T,  P = a I + b A + c A^2,  X <- P X     (A = X^T X, X <- X P where
//                                                     G has more rows than columns)
//
// With the square completed, P = c S^2 + (a - c d^2) I, S = A + d I, d = b / (2 c): the
// first product's epilogue adds d to its diagonal and the second one needs no other
// operand (reading A again there cost as much time as the product itself).
//
// p(s) = a s + b s^3 + c s^5 acts on each singular value and drives it towards
// 1.  Bound by the matrix products: per step p^2 q + p^3 + 2 p^2 q flops (p the
// smaller side; A and A^2 are symmetric, so only tiles on and above the diagonal
// are computed and each is written to both places).
//
// Errors of an early step grow with the singular values they fall on (a factor
// of up to a per step), so single bfloat16 or float16 products lose what a
// float32 gradient holds.  X, A and P are kept as two float16 per value
// (tile_gemm.h) at fixed power-of-two scales that follow from bounds of p over
// the steps: float32 accuracy at three float16 products, and each product's
// epilogue writes the next one's operand directly.  The norm is summed in
// float64 (squares of small gradients leave float32's range).
//
// Measured, five steps: 64 float32 matrices of 1408 x 2048 14.9 to 15.9 ms (970 to 908 TFLOP/s of float16
// products, from card to card, of the 1415 that one dense product reaches here; X's product 1.46 ms, 1.32 times what
// that rate gives, the symmetric ones 0.82 ms, 1.77 times: their 21 tiles a matrix end unevenly and
// are written twice); 4 bfloat16 ones of 1280 x 896 428 to 470 us, where each of the 15
// products is about one tile per CU.
#include <math.h>

#include <algorithm>

#include "ops_internal.h"
#include "tile_gemm.h"

namespace moe {
namespace {

// The two kinds of product: a symmetric one, and the last one of a step.
enum : int { NS_SYM = 0, NS_APPLY = 1 };
constexpr int kNormParts = 64;  // partial norms per matrix

struct NsProduct {
  const uint8_t* A;
  const uint8_t* B;
  uint8_t* out;            // split rows
  void* last;              // APPLY, last step: the result instead
  long long stride_a, stride_b, stride_out, stride_last;  // bytes (last: elements) per matrix
  uint32_t pitch_a, pitch_b, pitch_out;
  int rows_a, rows_b;      // rows of the operands as they are stored
  int width_a, width_b;    // their padded widths (column layout)
  int M, N, K;             // output rows and columns, contraction
  int last_dtype;
  int count;               // matrices
  float scale;             // of the accumulators
  float diag;              // SYM: added on the diagonal
  int32_t* counters;       // tile claims (kTgCounters zeros), or NULL
};

template <class C, int KIND>
struct NsTiles {
  const NsProduct& p;
  struct Tile {
    TgOperand A, B;
    int m0, n0, steps, rows, cols, hint, i;
  };
  static constexpr bool SYM = KIND == NS_SYM;
  __device__ __forceinline__ bool tri(const Tile& t) const { return t.m0 == t.n0; }

  __device__ __forceinline__ int per_matrix() const {
    const int mt = (p.M + C::BM - 1) / C::BM;
    return SYM ? mt * (mt + 1) / 2 : mt * ((p.N + C::BN - 1) / C::BN);
  }
  __device__ __forceinline__ Tile tile(int L, int) const {
    Tile t;
    const int per = per_matrix(), mt = (p.M + C::BM - 1) / C::BM;
    t.i = L / per;
    int local = L - t.i * per;
    if (SYM) {  // row y of the upper triangle starts at tile y mt - y (y - 1) / 2
      int y = 0;
      while (local >= mt - y) {
        local -= mt - y;
        ++y;
      }
      t.m0 = y * C::BM;
      t.n0 = (y + local) * C::BN;
    } else {
      t.m0 = local % mt * C::BM;
      t.n0 = local / mt * C::BN;
    }
    t.hint = 0;
    t.rows = p.M - t.m0;
    t.cols = p.N - t.n0;
    t.A.p = p.A + (size_t)t.i * p.stride_a;
    t.A.pitch = p.pitch_a;
    t.A.rows = p.rows_a;
    t.A.width = p.width_a;
    t.B.p = p.B + (size_t)t.i * p.stride_b;
    t.B.pitch = p.pitch_b;
    t.B.rows = p.rows_b;
    t.B.width = p.width_b;
    t.steps = (p.K + C::KS - 1) / C::KS;
    return t;
  }

  __device__ __forceinline__ void store(const Tile& t, int wm, int wn, int lane,
                                        f32x16 (&acc)[C::FM][C::FN]) const {
    uint8_t* out = p.out + (size_t)t.i * p.stride_out;
    const int wide = (p.N + 31) & ~31;  // columns of an output row with its padding
    if constexpr (SYM) {
      // A lane holds rows m .. m + 3 (m = 8 q + 4 (lane / 32) in a fragment) of one
      // column n.  Written as columns m .. of row n (16-byte runs), and, four
      // lanes transposed among themselves, as columns n .. of rows m ...  A
      // diagonal tile (its lower left quarter not computed, only mirrored)
      // writes the second form, and the first of its upper right quarter.
      const bool diagonal = t.m0 == t.n0, quarters = diagonal && C::FM == 2 && t.rows > C::BM / 2;
#pragma unroll
      for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < C::FN; ++fn) {
          const bool lower = tg_skip<C, C::FM == 2>(fm, fn);
          const bool mirror = !diagonal || (quarters && fm < C::FM / 2 && fn >= C::FN / 2);
          if (lower && quarters) continue;
          const int n = t.n0 + tg_col<C>(wn, fn, lane, 0);
          const int m0 = t.m0 + tg_row<C>(wm, fm, 0, 0);  // the fragment's first row
          if (m0 >= wide || t.n0 + tg_col<C>(wn, fn, 0, 0) >= wide) continue;
          uint2 wh[4], wl[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int m = m0 + 8 * q + 4 * (lane >> 5);
            uint16_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v = acc[fm][fn][4 * q + e] * p.scale;
              if (m + e == n) v += p.diag;
              if (m + e >= p.M || n >= p.N) v = 0.f;
              split_f16(v, hi[e], lo[e]);
            }
            wh[q] = uint2{hi[0] | ((uint32_t)hi[1] << 16), hi[2] | ((uint32_t)hi[3] << 16)};
            wl[q] = uint2{lo[0] | ((uint32_t)lo[1] << 16), lo[2] | ((uint32_t)lo[3] << 16)};
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint2 h = tg_quad_transpose(wh[q], lane), l = tg_quad_transpose(wl[q], lane);
            const int m = m0 + 8 * q + 4 * (lane >> 5) + (lane & 3);
            if (m < p.M) {
              uint8_t* at = out + (size_t)m * p.pitch_out + split_at(n & ~3);
              *(uint2*)at = h;
              *(uint2*)(at + 64) = l;
            }
          }
          if (mirror && n < p.N) {
            u32x4 r0, r1;
            uint8_t* at = out + (size_t)n * p.pitch_out + split_at(m0 + 8 * (lane >> 5));
            tg_runs16(wh, r0, r1);
            *(u32x4*)at = r0;
            *(u32x4*)(at + 32) = r1;
            tg_runs16(wl, r0, r1);
            *(u32x4*)(at + 64) = r0;
            *(u32x4*)(at + 96) = r1;
          }
        }
    } else {
      const bool vec = p.N % 8 == 0;  // whole 16-byte runs of either type
#pragma unroll
      for (int fm = 0; fm < C::FM; ++fm) {
        const int m = t.m0 + tg_row<C>(wm, fm, lane, 0);
        if (m >= p.M) continue;
#pragma unroll
        for (int fn = 0; fn < C::FN; ++fn) {
          const int n0 = t.n0 + tg_col<C>(wn, fn, 0, 0);  // the fragment's first column
          if (n0 >= wide) continue;
          if (p.last == nullptr) {
            uint2 wh[4], wl[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int n = n0 + 8 * q + 4 * (lane >> 5);
              uint16_t hi[4], lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                split_f16(n + e < p.N ? acc[fm][fn][4 * q + e] * p.scale : 0.f, hi[e], lo[e]);
              wh[q] = uint2{hi[0] | ((uint32_t)hi[1] << 16), hi[2] | ((uint32_t)hi[3] << 16)};
              wl[q] = uint2{lo[0] | ((uint32_t)lo[1] << 16), lo[2] | ((uint32_t)lo[3] << 16)};
            }
            u32x4 r0, r1;
            uint8_t* at = out + (size_t)m * p.pitch_out + split_at(n0 + 8 * (lane >> 5));
            tg_runs16(wh, r0, r1);
            *(u32x4*)at = r0;
            *(u32x4*)(at + 32) = r1;
            tg_runs16(wl, r0, r1);
            *(u32x4*)(at + 64) = r0;
            *(u32x4*)(at + 96) = r1;
            continue;
          }
          const size_t row = (size_t)t.i * p.stride_last + (size_t)m * p.N;
          if (p.last_dtype == 0) {
            float* c = (float*)p.last + row;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int n = n0 + 8 * q + 4 * (lane >> 5);
              const f32x4 v = {acc[fm][fn][4 * q] * p.scale, acc[fm][fn][4 * q + 1] * p.scale,
                               acc[fm][fn][4 * q + 2] * p.scale, acc[fm][fn][4 * q + 3] * p.scale};
              if (vec) {
                if (n < p.N) *(f32x4*)(c + n) = v;
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (n + e < p.N) c[n + e] = v[e];
              }
            }
          } else {
            uint16_t* c = (uint16_t*)p.last + row;
            uint2 w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = uint2{pack_bf16x2(acc[fm][fn][4 * q] * p.scale, acc[fm][fn][4 * q + 1] * p.scale),
                           pack_bf16x2(acc[fm][fn][4 * q + 2] * p.scale, acc[fm][fn][4 * q + 3] * p.scale)};
            if (vec) {
              u32x4 r0, r1;
              tg_runs16(w, r0, r1);
              const int n = n0 + 8 * (lane >> 5);
              if (n < p.N) *(u32x4*)(c + n) = r0;
              if (n + 16 < p.N) *(u32x4*)(c + n + 16) = r1;
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int n = n0 + 8 * q + 4 * (lane >> 5);
                const uint32_t b[2] = {w[q].x, w[q].y};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (n + e < p.N) c[n + e] = (uint16_t)(b[e >> 1] >> (16 * (e & 1)));
              }
            }
          }
        }
      }
    }
  }
};

template <class C, int KIND>
__global__ __launch_bounds__(C::THREADS, C::WAVES_PER_SIMD) void ns_kernel(NsProduct p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::LDS];
  __shared__ int s_claim;
  const NsTiles<C, KIND> tiles{p};
  const int n = tiles.per_matrix() * p.count;
  if constexpr (C::SMALL) tg_run_small<C>(tiles, n, lds);
  else tg_run<C>(tiles, n, p.counters, lds, &s_claim);
}

// ---------------------------------------------------------------- the first iterate
// Partial sums of squares (and the products' claim counters zeroed): block (part, matrix) takes the part-th share of its values.
template <class E>
__global__ __launch_bounds__(256) void ns_norm_kernel(const void* __restrict__ x, long long stride,
                                                      long long per, double* __restrict__ part,
                                                      int32_t* __restrict__ counters, int claims) {
  __shared__ double s[4];
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < claims; i += 256) counters[i] = 0;
  const typename E::T* src = (const typename E::T*)x + (long long)blockIdx.y * stride;
  const long long chunks = (per + 7) / 8;
  const long long a = chunks * blockIdx.x / kNormParts, b = chunks * (blockIdx.x + 1) / kNormParts;
  const bool aligned = stride % E::kPerChunk == 0;
  double v = 0.0;
  for (long long i = a + threadIdx.x; i < b; i += 256) {
    float f[8];
    // (matrices back to back at an odd size are read element by element)
    if (aligned) load_chunk<E>(src, 8 * i, per, f);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 8 * i + e < per ? load_as_f32<E>(src + 8 * i + e) : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v += (double)f[e] * (double)f[e];
  }
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.y * kNormParts + blockIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
}

// X_0 in split rows (zeros in the padding), scaled by 2^ex; with `last` set (no
// steps), X_0 itself as the result.  One wavefront per row.
template <class E>
__global__ __launch_bounds__(256) void ns_start_kernel(const void* __restrict__ x, long long stride,
                                                       int m, int n, long long rows,
                                                       const double* __restrict__ part, float eps,
                                                       float scale, uint8_t* __restrict__ out,
                                                       uint32_t pitch, void* last,
                                                       long long last_stride, int last_dtype) {
  const int lane = threadIdx.x & 63;
  for (long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); r < rows; r += 4LL * gridDim.x) {
    const long long i = r / m, row = r % m;
    double sq = part[i * kNormParts + lane];
    static_assert(kNormParts == 64, "one partial norm per lane");
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) sq += __shfl_xor(sq, k);
    const double norm = sqrt(sq) + (double)eps;
    // an all-zero matrix stays zero
    const double f = norm == 0.0 ? 0.0 : (double)scale / norm;
    const typename E::T* src = (const typename E::T*)x + i * stride + row * n;
    if (last != nullptr) {
      for (int j = lane; j < n; j += 64) {
        const float v = (float)((double)load_as_f32<E>(src + j) * f);
        if (last_dtype == 0) ((float*)last)[i * last_stride + row * n + j] = v;
        else ((uint16_t*)last)[i * last_stride + row * n + j] = f32_to_bf16(v);
      }
      continue;
    }
    const int padded = (n + 31) & ~31;
    for (int j = 8 * lane; j < padded; j += 512) {
      float v[8];
      load_chunk<E>(src, j, n, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)((double)v[e] * f);
      store_chunk(v, out + r * pitch, j);
    }
  }
}

// ---------------------------------------------------------------- launch
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Exponent that keeps values up to `most` (in magnitude) below 2^15.
int scale_exponent(double most) { return 14 - (int)ceil(log2(std::max(most, 1e-30))); }

struct NsPlan {
  size_t x[2], a, p, part, counters, bytes;
  size_t stride_x, stride_a;
};
constexpr int kMaxSteps = 64;
NsPlan ns_plan(int B, int m, int n) {
  NsPlan l{};
  const int side = std::min(m, n);
  l.stride_x = (size_t)m * split_pitch(n);
  l.stride_a = (size_t)side * split_pitch(side);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = up256(at + bytes);
    return o;
  };
  l.x[0] = take(l.stride_x * B);
  l.x[1] = take(l.stride_x * B);
  l.a = take(l.stride_a * B);
  l.p = take(l.stride_a * B);
  l.part = take((size_t)B * kNormParts * 8);
  l.counters = take((size_t)kMaxSteps * 3 * kTgCounters * 4);
  l.bytes = at;
  return l;
}

template <class C, int KIND>
hipError_t run_ns(NsProduct p, hipStream_t st) {
  const long long mt = (p.M + C::BM - 1) / C::BM, nt = (p.N + C::BN - 1) / C::BN;
  const long long total = (KIND == NS_APPLY ? mt * nt : mt * (mt + 1) / 2) * p.count;
  const long long blocks = (long long)device_cu_count() * C::BPC;
  if (total <= blocks) p.counters = nullptr;  // one tile each
  ns_kernel<C, KIND><<<(unsigned)std::min(total, blocks), C::THREADS, 0, st>>>(p);
  return hipGetLastError();
}
// The largest tiles that give more than half of the CUs one (tile_gemm.h).
template <int KIND, bool AC, bool BC, bool SW>
hipError_t pick_ns(const NsProduct& p, hipStream_t st) {
  auto tiles = [&](long long b) {
    const long long mt = (p.M + b - 1) / b, nt = (p.N + b - 1) / b;
    return (KIND == NS_APPLY ? mt * nt : mt * (mt + 1) / 2) * p.count;
  };
  const int cus = device_cu_count();
  if (2 * tiles(256) > cus) return run_ns<TgConfig<TgBig, AC, BC, 2, SW>, KIND>(p, st);
  if (2 * tiles(128) > cus) return run_ns<TgConfig<TgMid, AC, BC, 2, SW>, KIND>(p, st);
  return run_ns<TgConfig<TgSmall, AC, BC, 2, SW>, KIND>(p, st);
}

}  // namespace

void ortho_bounds(int steps, float af, float bf, float cf, double* iterate, double* factor) {
  const double a = af, b = bf, c = cf;
  double s = 1.0, top = 1.0, f = 0.0;
  for (int k = 0; k < steps && top <= 1e30 && f <= 1e30; ++k) {
    // q = |a + b t + c t^2| and |u q(u^2)| = |a u + b u^3 + c u^5| over u in [0, s],
    // t = u^2: at the ends of the range and where their derivatives vanish
    const double end = s * s;
    double fac = fabs(a), next = 0.0;
    auto at = [&](double t) {
      if (!(t >= 0.0) || t > end) return;
      const double q = fabs(a + b * t + c * t * t);
      fac = std::max(fac, q);
      next = std::max(next, sqrt(t) * q);
    };
    at(end);
    if (c != 0.0) {
      at(-b / (2.0 * c));
      const double root = 9.0 * b * b - 20.0 * a * c;  // of a + 3 b t + 5 c t^2
      if (root >= 0.0) {
        at((-3.0 * b + sqrt(root)) / (10.0 * c));
        at((-3.0 * b - sqrt(root)) / (10.0 * c));
      }
    } else if (b != 0.0) {
      at(-a / (3.0 * b));
    }
    // (1.01: what the products' rounding adds, and that of these points)
    f = std::max(f, 1.01 * fac);
    s = 1.01 * next;
    top = std::max(top, s);
  }
  *iterate = top;
  *factor = f;
}

size_t ortho_workspace_bytes(int B, int m, int n) {
  // (no steps: the general path's norm and division, whatever the size)
  return std::max(ortho_small_fits(B, m, n) ? ortho_small_workspace_bytes(B, m, n) : 0,
                  ns_plan(B, m, n).bytes);
}

hipError_t launch_orthogonalize(const OrthoArgs& a, void* ws, hipStream_t st) {
  // d of the completed square; c = 0: the first product gives P = a I + b A itself
  const double d = a.c != 0.f ? (double)a.b / (2.0 * a.c) : 0.0;
  const int ex = scale_exponent(a.most_x), ea = scale_exponent(a.most_x * a.most_x + fabs(d)),
            ep = scale_exponent(a.most_p);
  OrthoScales sc{};
  sc.first = a.steps == 0 ? 1.f : ldexpf(1.f, ex);
  sc.s_scale = ldexpf(1.f, ea - 2 * ex);
  sc.s_diag = (float)ldexp(d, ea);
  sc.p_scale = a.c != 0.f ? ldexpf(a.c, ep - 2 * ea) : ldexpf(a.b, ep - 2 * ex);
  sc.p_diag = (float)ldexp(a.a - a.c * d * d, ep);
  sc.x_scale = ldexpf(1.f, -ep);
  sc.last_scale = ldexpf(1.f, -ep - ex);
  if (a.steps > 0 && ortho_small_fits(a.B, a.m, a.n))
    return launch_orthogonalize_small(a, sc, ws, st);
  const NsPlan l = ns_plan(a.B, a.m, a.n);
  uint8_t* w = (uint8_t*)ws;
  double* part = (double*)(w + l.part);
  const long long per = (long long)a.m * a.n, rows = (long long)a.B * a.m;
  int32_t* counters = (int32_t*)(w + l.counters);
  const int claims = a.steps * 3 * kTgCounters;
  const uint32_t px = (uint32_t)split_pitch(a.n), pa = (uint32_t)split_pitch(std::min(a.m, a.n));
  void* direct = a.steps == 0 ? a.out : nullptr;
  // (a launch holds fewer than 2^32 threads: past 2^20 blocks each takes further rows)
  const dim3 gn(kNormParts, a.B), gs((unsigned)std::min((rows + 3) / 4, 1LL << 20));
  if (a.dtype == 0) {
    ns_norm_kernel<ElemF32><<<gn, 256, 0, st>>>(a.x, a.x_stride, per, part,
                                                counters, claims);
    ns_start_kernel<ElemF32><<<gs, 256, 0, st>>>(a.x, a.x_stride, a.m, a.n, rows, part, a.eps, sc.first,
                                                 w + l.x[0], px, direct, a.out_stride, a.out_dtype);
  } else {
    ns_norm_kernel<ElemBF16><<<gn, 256, 0, st>>>(a.x, a.x_stride, per, part,
                                                counters, claims);
    ns_start_kernel<ElemBF16><<<gs, 256, 0, st>>>(a.x, a.x_stride, a.m, a.n, rows, part, a.eps, sc.first,
                                                  w + l.x[0], px, direct, a.out_stride, a.out_dtype);
  }
  hipError_t e = hipGetLastError();
  const bool tall = a.m > a.n;
  const int side = std::min(a.m, a.n), wide_x = (a.n + 31) & ~31, wide_a = (side + 31) & ~31;
  for (int k = 0; k < a.steps && e == hipSuccess; ++k) {
    const uint8_t* X = w + l.x[k & 1];
    int32_t* cnt = counters + k * 3 * kTgCounters;
    NsProduct g{};
    g.A = g.B = X;
    g.out = w + (a.c != 0.f ? l.a : l.p);
    g.stride_a = g.stride_b = l.stride_x;
    g.stride_out = l.stride_a;
    g.pitch_a = g.pitch_b = px;
    g.pitch_out = pa;
    g.rows_a = g.rows_b = a.m;
    g.width_a = g.width_b = wide_x;
    g.M = g.N = side;
    g.K = tall ? a.m : a.n;
    g.count = a.B;
    g.counters = cnt;
    g.scale = a.c != 0.f ? sc.s_scale : sc.p_scale;
    g.diag = a.c != 0.f ? sc.s_diag : sc.p_diag;
    e = tall ? pick_ns<NS_SYM, true, true, false>(g, st) : pick_ns<NS_SYM, false, false, false>(g, st);
    if (e != hipSuccess) break;
    if (a.c != 0.f) {
      NsProduct q{};
      q.A = q.B = w + l.a;
      q.out = w + l.p;
      q.stride_a = q.stride_b = q.stride_out = l.stride_a;
      q.pitch_a = q.pitch_b = q.pitch_out = pa;
      q.rows_a = q.rows_b = side;
      q.width_a = q.width_b = wide_a;
      q.M = q.N = q.K = side;
      q.count = a.B;
      q.counters = cnt + kTgCounters;
      q.scale = sc.p_scale;
      q.diag = sc.p_diag;
      e = pick_ns<NS_SYM, false, false, false>(q, st);
      if (e != hipSuccess) break;
    }
    NsProduct u{};
    u.out = w + l.x[(k + 1) & 1];
    u.stride_out = l.stride_x;
    u.pitch_out = px;
    u.M = a.m;
    u.N = a.n;
    u.K = side;
    u.count = a.B;
    u.counters = cnt + 2 * kTgCounters;
    u.scale = sc.x_scale;
    if (k + 1 == a.steps) {
      u.last = a.out;
      u.last_dtype = a.out_dtype;
      u.stride_last = a.out_stride;
      u.scale = sc.last_scale;
    }
    if (tall) {  // X P
      u.A = X;
      u.stride_a = l.stride_x;
      u.pitch_a = px;
      u.rows_a = a.m;
      u.width_a = wide_x;
      u.B = w + l.p;
      u.stride_b = l.stride_a;
      u.pitch_b = pa;
      u.rows_b = side;
      u.width_b = wide_a;
      e = pick_ns<NS_APPLY, false, false, true>(u, st);
    } else {  // P X
      u.A = w + l.p;
      u.stride_a = l.stride_a;
      u.pitch_a = pa;
      u.rows_a = side;
      u.width_a = wide_a;
      u.B = X;
      u.stride_b = l.stride_x;
      u.pitch_b = px;
      u.rows_b = a.m;
      u.width_b = wide_x;
      e = pick_ns<NS_APPLY, false, true, true>(u, st);
    }
  }
  return e;
}

}  // namespace moe
