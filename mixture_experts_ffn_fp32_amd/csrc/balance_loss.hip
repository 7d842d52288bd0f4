// Balance loss of the routing with its gradient, per batch or per sequence (DeepSeekMoE paper
// summary, papercache.org, sec. 3.3, expert-level and device-level balance losses), over the n
// rows of a sequence that are not masked:
//
//   count_i = #{(t, k) : idx[t][k] = i},  f_i = N count_i / (K n),  P_i = (1/n) sum_t s_ti
//   L_0 = alpha1 sum_i f_i P_i,  L_1 = alpha2 sum_g f'_g P'_g
//   f'_g = mean of f_i, P'_g = sum of P_i over the experts of device g
//
// The counts are whole numbers that no score's small change moves, so the losses are linear in
// the scores, with the same slopes in every row of a sequence:
//
//   dL_0 / ds_ti = alpha1 f_i / n,  dL_1 / ds_ti = alpha2 f'_{g(i)} / n
//
// and through the softmax  dlogits_ti = s_ti (c_i - sum_j s_tj c_j),  c = the slopes times the
// losses' own gradients.
//
// Small passes over the scores, bound by launches.  Forward: one launch for partial sums of
// kBlRows rows (float64, counts as whole numbers), one that joins a sequence's partial sums in
// order.  Backward: one launch, a wavefront per four rows.  Every sum has a fixed order.
//
// Measured: 4096 x 63 in one sequence 5.1, 4.5 and 5.2 us; 16384 x 128 in eight sequences (8 MB each
// way) 8.0, 5.7 and 8.3 us (with loads row by row, and a wavefront per row, 32 us for the three).
#include <algorithm>

#include "groups.h"
#include "ops_internal.h"

namespace moe {
namespace {

constexpr int kBlRows = 64;

// Partial sums of the chunks of kBlRows rows of the sequences, chunk b in partial row b: one chunk
// a block, and past kBlMostBlocks, as a launch holds fewer than 2^32 threads, each block takes
// further ones.  The loads of a thread's column (every 512 / NP-th row) are made eight at a time,
// whatever the mask says; a masked row's are left out of the sum.
constexpr int kBlThreads = 512;
constexpr long long kBlMostBlocks = 1 << 20;
__global__ __launch_bounds__(kBlThreads) void balance_loss_partial_kernel(BalanceLossArgs a) {
  __shared__ GroupTables t;
  __shared__ int cnt[256], valid[kBlRows];
  __shared__ double sum[kBlThreads];
  const int tid = threadIdx.x, N = a.N;
  group_tables<GR_FWD>(GroupDims{a.T, a.S, 0, 0}, a.offsets, kBlRows, t);
  const int chunks = uni(t.tiles[a.S]);
  for (int b = blockIdx.x; b < chunks; b += gridDim.x) {
    const int s = group_of(t.tiles, a.S, b, 0);
    const int t0 = t.off[s] + (b - t.tiles[s]) * kBlRows, rows = min(kBlRows, t.off[s + 1] - t0);
    if (tid < 256) cnt[tid] = 0;
    if (tid < kBlRows) valid[tid] = tid < rows && (a.mask == nullptr || a.mask[t0 + tid] != 0);
    __syncthreads();
    for (int j = tid; j < rows * a.K; j += kBlThreads) {
      const int e = a.idx[(size_t)t0 * a.K + j];
      if (valid[j / a.K] && (unsigned)e < (unsigned)N) atomicAdd(&cnt[e], 1);
    }
    // kBlThreads / NP rows at a time, NP columns each
    const int NP = N <= 64 ? 64 : N <= 128 ? 128 : 256, G = kBlThreads / NP;
    const int c = tid & (NP - 1), g = tid / NP;
    double p = 0.0;
    if (c < N) {
      const float* from = a.scores + (size_t)t0 * N + c;
      for (int r0 = g; r0 < rows; r0 += 8 * G) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = from[(size_t)min(r0 + i * G, rows - 1) * N];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (r0 + i * G < rows && valid[r0 + i * G]) p += (double)v[i];
      }
    }
    sum[tid] = p;
    __syncthreads();
    if (tid < N) {
      for (int q = NP; q < kBlThreads; q += NP) p += sum[q + tid];
      a.psum[(size_t)b * N + tid] = p;
      a.pcnt[(size_t)b * (N + 1) + tid] = cnt[tid];
    }
    if (tid < 64) {
      const int n = __popcll(__ballot(valid[tid] != 0));
      if (tid == 0) a.pcnt[(size_t)b * (N + 1) + N] = n;
    }
    __syncthreads();  // the next chunk's counts and rows
  }
}
static_assert(kBlRows == 64, "a wavefront counts a chunk's rows");

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
  return v;
}

// One block per sequence.
__global__ __launch_bounds__(1024) void balance_loss_final_kernel(BalanceLossArgs a) {
  __shared__ GroupTables t;
  __shared__ double sum[1024], l0[4], l1[4];
  __shared__ int cnt[1024], dev_cnt[256], dev_size[256], s_n;
  const int tid = threadIdx.x, N = a.N, s = blockIdx.x;
  group_tables<GR_FWD>(GroupDims{a.T, a.S, 0, 0}, a.offsets, kBlRows, t);
  const int b0 = t.tiles[s], b1 = t.tiles[s + 1];
  const int NP = N <= 64 ? 64 : N <= 128 ? 128 : 256, c = tid & (NP - 1), g = tid / NP;
  double p = 0.0;
  int n = 0;
  int of = -1;
  if (tid < N && a.device_of != nullptr) {
    of = a.device_of[tid];
    if ((unsigned)of >= (unsigned)a.D) of = -1;
  }
  if (c < N) {
    const int G = 1024 / NP;
    for (int b = b0 + g; b < b1; b += 4 * G) {
      double v[4];
      int k[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = min(b + i * G, b1 - 1);
        v[i] = a.psum[(size_t)q * N + c];
        k[i] = a.pcnt[(size_t)q * (N + 1) + c];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (b + i * G < b1) {
          p += v[i];
          n += k[i];
        }
    }
  }
  sum[tid] = p;
  cnt[tid] = n;
  if (tid < 256) dev_cnt[tid] = dev_size[tid] = 0;
  if (tid < 64) {
    int v = 0;
    for (int b = b0 + tid; b < b1; b += 64) v += a.pcnt[(size_t)b * (N + 1) + N];
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
    if (tid == 0) s_n = v;
  }
  __syncthreads();
  const double rows = s_n > 0 ? (double)s_n : 1.0;  // no rows: every sum is zero
  if (tid < N) {
    for (int q = NP; q < 1024; q += NP) {
      p += sum[q + tid];
      n += cnt[q + tid];
    }
    if (of >= 0) {
      atomicAdd(&dev_cnt[of], n);
      atomicAdd(&dev_size[of], 1);
    }
  }
  __syncthreads();
  double v0 = 0.0, v1 = 0.0;
  if (tid < N) {
    const double unit = (double)N / ((double)a.K * rows), P = p / rows;
    const double f = (double)a.alpha1 * unit * n;
    const double fd = of >= 0 ? (double)a.alpha2 * unit * dev_cnt[of] / dev_size[of] : 0.0;
    const size_t at = (size_t)s * N + tid;
    a.counts[at] = n;
    a.P[at] = (float)P;
    a.slopes[2 * (size_t)s * N + tid] = (float)(f / rows);
    a.slopes[(2 * (size_t)s + 1) * N + tid] = (float)(fd / rows);
    v0 = f * P;
    v1 = fd * P;
  }
  if (tid < 256) {
    v0 = wave_sum_f64(v0);
    v1 = wave_sum_f64(v1);
    if ((tid & 63) == 0) {
      l0[tid >> 6] = v0;
      l1[tid >> 6] = v1;
    }
  }
  __syncthreads();
  if (tid == 0) {
    a.losses[2 * s] = (float)(l0[0] + l0[1] + l0[2] + l0[3]);
    a.losses[2 * s + 1] = (float)(l1[0] + l1[1] + l1[2] + l1[3]);
  }
}

// One wavefront for kBlAtOnce neighbouring rows, PER columns of each a lane; rows of no sequence
// and masked ones are zeros.
constexpr int kBlAtOnce = 4;
template <int PER>
__global__ __launch_bounds__(256) void balance_loss_backward_kernel(BalanceLossArgs a) {
  __shared__ GroupTables t;
  const int lane = threadIdx.x & 63, N = a.N;
  group_tables<GR_FWD>(GroupDims{a.T, a.S, 0, 0}, a.offsets, kBlRows, t);
  const int first = t.off[0], last = t.off[a.S];
  int known = -1;  // the sequence whose slopes c holds
  float c[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) c[i] = 0.f;
  const long long stride = (long long)gridDim.x * 4 * kBlAtOnce;
  const long long r0 = ((long long)blockIdx.x * 4 + (threadIdx.x >> 6)) * kBlAtOnce;
  for (long long r = r0; r < a.T; r += stride) {
    float v[kBlAtOnce][PER], z[kBlAtOnce][PER], dot[kBlAtOnce];
    bool on[kBlAtOnce];
#pragma unroll
    for (int q = 0; q < kBlAtOnce; ++q) {
      const int row = uni((int)min(r + q, a.T - 1LL));
      on[q] = row >= first && row < last && (a.mask == nullptr || a.mask[row] != 0);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int j = lane + 64 * i;
        v[q][i] = j < N ? a.scores[(size_t)row * N + j] : 0.f;
      }
    }
#pragma unroll
    for (int q = 0; q < kBlAtOnce; ++q) {
      const int row = uni((int)min(r + q, a.T - 1LL));
      const int s = on[q] ? uni(group_of(t.off, a.S, row, max(known, 0))) : known;
      if (s != known) {
        known = s;
        const float d0 = a.dlosses != nullptr ? a.dlosses[2 * s] : 1.f;
        const float d1 = a.dlosses != nullptr ? a.dlosses[2 * s + 1] : 1.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int j = lane + 64 * i;
          const float* slopes = a.slopes + 2 * (size_t)s * N + j;
          c[i] = j < N ? d0 * slopes[0] + d1 * slopes[N] : 0.f;
        }
      }
      dot[q] = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        z[q][i] = c[i];
        dot[q] += v[q][i] * c[i];
      }
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1)
#pragma unroll
      for (int q = 0; q < kBlAtOnce; ++q) dot[q] += __shfl_xor(dot[q], k);
#pragma unroll
    for (int q = 0; q < kBlAtOnce; ++q)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int j = lane + 64 * i;
        if (r + q < a.T && j < N)
          a.dlogits[(size_t)(r + q) * N + j] = on[q] ? v[q][i] * (z[q][i] - dot[q]) : 0.f;
      }
  }
}

long long balance_loss_chunks(int T, int S) { return (T + (kBlRows - 1LL)) / kBlRows + S; }
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

size_t balance_loss_workspace_bytes(int T, int N, int S) {
  const size_t b = (size_t)balance_loss_chunks(T, S);
  return align256(b * N * 8) + b * (N + 1) * 4;
}

hipError_t launch_balance_loss(BalanceLossArgs a, void* ws, hipStream_t st) {
  const long long chunks = balance_loss_chunks(a.T, a.S);
  a.psum = (double*)ws;
  a.pcnt = (int32_t*)((char*)ws + align256((size_t)chunks * a.N * 8));
  if (a.T > 0) {
    const unsigned blocks = (unsigned)std::min(chunks, kBlMostBlocks);
    balance_loss_partial_kernel<<<blocks, kBlThreads, 0, st>>>(a);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  balance_loss_final_kernel<<<a.S, 1024, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const BalanceLossArgs& a, hipStream_t st) {
  const unsigned grid =
      (unsigned)std::min<long long>((a.T + 4LL * kBlAtOnce - 1) / (4 * kBlAtOnce), 2048);
  if (a.N <= 64) balance_loss_backward_kernel<1><<<grid, 256, 0, st>>>(a);
  else if (a.N <= 128) balance_loss_backward_kernel<2><<<grid, 256, 0, st>>>(a);
  else balance_loss_backward_kernel<4><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
