// Declarations shared by the operators beside the layer (norms, grouped products,
// orthogonalised update, 8-bit operands, balance loss) and their C-ABI host code.
#pragma once

#include "moe_internal.h"

namespace moe {

// The message moe_last_error() returns on this thread.
void set_last_error(const char* msg);

// ---------------------------------------------------------------- layer norm (norm.hip)
struct NormArgs {
  const void* x;       // [T][d]
  const void* weight;  // [d] or NULL (ones)
  const void* bias;    // [d] or NULL (zeros)
  const void* dy;      // [T][d]
  void* out;           // y or dx
  float* mean;         // [T]: written by the forward (may be NULL), read by the backward
  float* rstd;         // [T]
  float* part;         // [chunks][2][d] partial weight and bias gradients
  float* dweight;      // [d] or NULL
  float* dbias;        // [d] or NULL
  int T, d;
  float eps;
};
hipError_t launch_layer_norm(int dtype, const NormArgs& a, hipStream_t st);
// Rows of partial weight gradients the backward writes for these shapes.
int layer_norm_chunks(int dtype, int T, int d);
hipError_t launch_layer_norm_backward(int dtype, const NormArgs& a, hipStream_t st);

// ---------------------------------------------------------------- grouped products (grouped.hip)
struct GroupedArgs {
  const void* x;           // [M][k]
  const void* w;           // [E][n][k]
  const void* dy;          // [M][n]    (backward)
  const int32_t* offsets;  // [E+1]
  void* y;                 // [M][n]    (forward)
  void* dx;                // [M][k]    (backward, may be NULL)
  float* dw;               // [E][n][k] (backward, may be NULL)
  int M, E, n, k;
  int zero_rest;           // rows outside every group: 1 zeros, 0 left as they are
};
constexpr int kGroupedMaxE = 1024;
// Longest row (bytes, padded) whose 256-row tiles stay inside a 2 GiB buffer range.
constexpr long long kGroupedMaxRowBytes = 1 << 22;
size_t grouped_workspace_bytes(int dtype, int M, int E, int n, int k);
hipError_t launch_grouped(int dtype, const GroupedArgs& a, void* ws, hipStream_t st);
size_t grouped_backward_workspace_bytes(int dtype, int M, int E, int n, int k, bool dx, bool dw);
hipError_t launch_grouped_backward(int dtype, const GroupedArgs& a, void* ws, hipStream_t st);

// ---------------------------------------------------------------- orthogonalised update (orthogonalize.hip)
struct OrthoArgs {
  const void* x;
  void* out;
  long long x_stride, out_stride;  // elements from one matrix to the next
  int B, m, n, steps;
  int dtype, out_dtype;
  float eps, a, b, c;
  double most_x, most_p;  // ortho_bounds of these steps and coefficients
};
// Largest bounds of the iterate and of the polynomial factor over the steps, for
// coefficients (a, b, c) and a first iterate of Frobenius norm 1.
void ortho_bounds(int steps, float a, float b, float c, double* iterate, double* factor);
constexpr double kOrthoMaxBound = 1024.0;
size_t ortho_workspace_bytes(int B, int m, int n);
hipError_t launch_orthogonalize(const OrthoArgs& a, void* ws, hipStream_t st);

// Power-of-two scales and constants of the products (see launch_orthogonalize): X is
// held times 2^ex (`first`), S = A + d I times 2^ea, P times 2^ep; each product's
// accumulators times its scale are the next operand.
struct OrthoScales {
  float first, s_scale, s_diag, p_scale, p_diag, x_scale, last_scale;
};
// orthogonalize_small.hip: whether these matrices go there, and the launch.
bool ortho_small_fits(int B, int m, int n);
size_t ortho_small_workspace_bytes(int B, int m, int n);
hipError_t launch_orthogonalize_small(const OrthoArgs& a, const OrthoScales& s, void* ws,
                                      hipStream_t st);

// ---------------------------------------------------------------- RMS norm (rms_norm.hip)
struct RmsArgs {
  const void* x;         // [T][d] (backward: h)
  const void* residual;  // [T][d] or NULL
  const void* weight;    // [d] or NULL (ones)
  const void* dy;        // [T][d]
  const void* dh;        // [T][d] or NULL
  void* h;               // [T][d] or NULL; may be x or residual
  void* out;             // y, or dx (which may be dh)
  float* scales;         // [T][blocks], where y has 8 bits
  float* rstd;           // [T]: written by the forward (may be NULL), read by the backward
  float* part;           // [chunks][d] partial weight gradients
  float* dweight;        // [d] or NULL
  int T, d, blocks;
  float eps;
};
// f8: 0 the storage type, 1 e4m3, 2 e5m2 (y's type).
hipError_t launch_rms_norm(int dtype, int f8, RmsArgs a, hipStream_t st);
int rms_norm_chunks(int dtype, int T, int d);
hipError_t launch_rms_norm_backward(int dtype, const RmsArgs& a, hipStream_t st);

// ---------------------------------------------------------------- 8 bits (quantize.hip)
hipError_t launch_quantize_rows(int dtype, int f8, const void* x, int T, int d, void* q,
                                float* scales, hipStream_t st);
hipError_t launch_quantize_blocks(int dtype, int f8, const void* w, int E, int n, int k, void* q,
                                  float* scales, hipStream_t st);
hipError_t launch_dequantize_rows(int f8, int dtype, const void* q, const float* scales, int T,
                                  int d, void* x, hipStream_t st);

// ---------------------------------------------------------------- 8-bit grouped products (grouped_f8.hip)
struct GroupedF8Args {
  const void* x;           // [M][k] (dx: dy [M][n])
  const float* xs;         // [M][blocks of its columns]
  const void* w;           // [E][n][k]
  const float* ws;         // [E][blocks of n][blocks of k]
  const int32_t* offsets;  // [E+1], or NULL: one group of all rows
  void* out;               // [M][n] (dx: [M][k])
  int M, E, n, k;
  int zero_rest, out_f32;
};
size_t grouped_f8_workspace_bytes(int M, int E, int n, int k, bool dx);
hipError_t launch_grouped_f8(int f8, bool dx, const GroupedF8Args& a, void* ws, hipStream_t st);

// ---------------------------------------------------------------- balance loss (balance_loss.hip)
struct BalanceLossArgs {
  const float* scores;      // [T][N]
  const int32_t* idx;       // [T][K]
  const int32_t* offsets;   // [S+1], or NULL: one sequence of all rows
  const uint8_t* mask;      // [T] or NULL: rows that count (not zero)
  const int32_t* device_of; // [N] or NULL
  const float* dlosses;     // [S][2] or NULL (ones)
  int32_t* counts;          // [S][N]
  float* P;                 // [S][N]
  float* losses;            // [S][2]
  float* slopes;            // [S][2][N]: written by the forward, read by the backward
  float* dlogits;           // [T][N]
  double* psum;             // [chunks][N]
  int32_t* pcnt;            // [chunks][N + 1]
  int T, N, K, S, D;
  float alpha1, alpha2;
};
size_t balance_loss_workspace_bytes(int T, int N, int S);
hipError_t launch_balance_loss(BalanceLossArgs a, void* ws, hipStream_t st);
hipError_t launch_balance_loss_backward(const BalanceLossArgs& a, hipStream_t st);

int device_cu_count();

}  // namespace moe
