// Host code of the operators for 8-bit experts and of the balance loss under sanitizers: every
// validation path and workspace plan, none of which reaches a GPU.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>

#include "moe.h"

static int failures = 0;
#define WANT(call, status)                                                              \
  do {                                                                                  \
    const int got = (call);                                                             \
    if (got != (status) || (got != MOE_OK && strlen(moe_last_error()) == 0)) {          \
      printf("line %d: status %d, expected %d (%s)\n", __LINE__, got, (status),         \
             moe_last_error());                                                         \
      ++failures;                                                                       \
    }                                                                                   \
  } while (0)

static void* at(uintptr_t v) { return (void*)v; }

int main() {
  size_t bytes = 0;
  const int F = MOE_DTYPE_F32, B = MOE_DTYPE_BF16, Q = MOE_DTYPE_E4M3, R = MOE_DTYPE_E5M2;
  const uintptr_t far = (uintptr_t)1 << 44;
  float* f1 = (float*)at((uintptr_t)1 << 40);
  float* f2 = (float*)at((uintptr_t)1 << 41);
  // RMS norm
  WANT(moe_rms_norm(at(16), 0, 0, -1, 8, 0.f, F, F, 0, at(far), 0, 0, 0), MOE_ERR_INVALID_ARG);
  WANT(moe_rms_norm(at(16), 0, 0, 1, 8, NAN, F, F, 0, at(far), 0, 0, 0), MOE_ERR_INVALID_ARG);
  WANT(moe_rms_norm(at(16), 0, 0, 1, 8, 0.f, F, B, 0, at(far), 0, 0, 0), MOE_ERR_UNSUPPORTED);
  WANT(moe_rms_norm(at(16), 0, 0, 1, 8, 0.f, F, Q, 0, at(far), 0, 0, 0), MOE_ERR_INVALID_ARG);
  WANT(moe_rms_norm(at(16), 0, 0, 1, 8, 0.f, F, F, 0, at(far), f1, 0, 0), MOE_ERR_INVALID_ARG);
  WANT(moe_rms_norm(at(16), at(18), 0, 1, 8, 0.f, F, F, 0, at(far), 0, 0, 0), MOE_ERR_ALIGNMENT);
  WANT(moe_rms_norm(at(16), 0, 0, 1, 8, 0.f, F, F, at(32), at(far), 0, 0, 0), MOE_ERR_INVALID_ARG);
  WANT(moe_rms_norm(at(16), 0, 0, 2147483647, 1 << 24, 0.f, F, R, at(16), at(far), f1, 0, 0),
       MOE_ERR_INVALID_ARG);  // sizes past 2^55 overlap whatever lies there
  WANT(moe_rms_norm(0, 0, 0, 0, 8, 0.f, F, F, 0, 0, 0, 0, 0), MOE_OK);
  for (int T : {0, 1, 7, 4096, 2147483647})
    for (int d : {1, 64, 1283, 8192, 20000, 1 << 24})
      for (int dt : {F, B}) WANT(moe_rms_norm_backward_workspace_size(T, d, dt, &bytes), MOE_OK);
  WANT(moe_rms_norm_backward_workspace_size(4, 64, Q, &bytes), MOE_ERR_UNSUPPORTED);
  WANT(moe_rms_norm_backward(at(16), at(1 << 20), 0, f1, 0, 4, 64, F, at(far), f2, 0, 0, 0),
       MOE_ERR_INVALID_ARG);
  WANT(moe_rms_norm_backward(at(16), at(1 << 20), 0, f1, 0, 4, 64, F, at(far), f2, at(1 << 24), 4, 0),
       MOE_ERR_WORKSPACE);
  // 8 bits
  WANT(moe_quantize_rows(at(16), 4, 64, F, F, at(far), f1, 0), MOE_ERR_UNSUPPORTED);
  WANT(moe_quantize_rows(at(16), 2147483647, 1 << 24, F, Q, at(far), f1, 0), MOE_ERR_INVALID_ARG);
  WANT(moe_quantize_blocks(at(16), 2147483647, 1, 1, F, Q, at(far), f1, 0), MOE_ERR_UNSUPPORTED);
  WANT(moe_quantize_blocks(at(16), 1, 1 << 20, 1 << 20, F, Q, at(far), f1, 0), MOE_ERR_UNSUPPORTED);
  WANT(moe_quantize_blocks(at(16), 3, 200, 100, F, Q, at(32), f1, 0), MOE_ERR_INVALID_ARG);
  WANT(moe_dequantize_rows(at(16), f1, 4, 64, B, F, at(far), 0), MOE_ERR_UNSUPPORTED);
  WANT(moe_dequantize_rows(at(16), f1, 4, 64, Q, F, at(16), 0), MOE_ERR_INVALID_ARG);
  // products
  for (int M : {0, 1, 300, 1 << 20, 2147483647})
    for (int E : {1, 64, 1024})
      for (int n : {1, 16, 267, 2048, 1 << 20})
        for (int k : {1, 16, 267, 2048, 1 << 20}) {
          size_t a = 0, b = 0;
          const int s = moe_grouped_matmul_quantized_workspace_size(M, E, n, k, &a);
          if (s != MOE_OK && s != MOE_ERR_UNSUPPORTED) ++failures;
          if (moe_grouped_matmul_quantized_dx_workspace_size(M, E, n, k, &b) != s) ++failures;
          if (s == MOE_OK && M > 0 && k % 16 == 0 && (a != 0 || (n % 16 == 0 && b != 0))) ++failures;
        }
  WANT(moe_grouped_matmul_quantized(at(16), f1, at(1 << 20), f2, 0, 4, 2, 8, 8, Q, F, 1, at(far), 0, 0, 0),
       MOE_ERR_INVALID_ARG);
  WANT(moe_grouped_matmul_quantized(at(16), f1, at(1 << 20), f2, 0, 20000, 1, 8, 8, Q, F, 1, at(far),
                                    at(64), 1, 0),
       MOE_ERR_WORKSPACE);  // (fewer rows need none: odd ones are read where they are)
  WANT(moe_grouped_matmul_quantized_dx(at(16), f1, at(1 << 20), f2, 0, 4, 1, 8, 8, F, F, 1, at(far), 0, 0, 0),
       MOE_ERR_UNSUPPORTED);
  WANT(moe_grouped_matmul_quantized_dx(at(16), f1, at(1 << 20), f2, 0, 0, 1, 8, 8, R, F, 1, 0, 0, 0, 0),
       MOE_OK);
  // balance loss
  for (int T : {0, 1, 100000, 2147483647})
    for (int N : {1, 63, 256})
      for (int S : {1, 1024}) WANT(moe_balance_loss_workspace_size(T, N, S, &bytes), MOE_OK);
  int32_t* i1 = (int32_t*)at((uintptr_t)1 << 42);
  float* f3 = (float*)at((uintptr_t)1 << 43);
  WANT(moe_balance_loss(f1, i1, 0, 0, 0, 2147483647, 256, 2, 1, 0, 1.f, 1.f, i1, f2, f3, f3, at(far),
                        (size_t)-1, 0),
       MOE_ERR_UNSUPPORTED);
  WANT(moe_balance_loss(f1, i1, 0, 0, i1, 8, 8, 2, 1, 0, 1.f, 1.f, i1, f2, f3, f3, at(far), (size_t)-1, 0),
       MOE_ERR_INVALID_ARG);
  WANT(moe_balance_loss(f1, i1, 0, 0, 0, 8, 8, 2, 1, 0, 1.f, INFINITY, i1, f2, f3, f3, at(far),
                        (size_t)-1, 0),
       MOE_ERR_INVALID_ARG);
  WANT(moe_balance_loss_backward(f1, f2, 0, 0, 0, 8, 8, 1, f2, 0), MOE_ERR_INVALID_ARG);
  WANT(moe_balance_loss_backward(0, 0, 0, 0, 0, 0, 8, 1, 0, 0), MOE_OK);
  if (failures == 0) printf("ALL OK\n");
  return failures != 0;
}
