// Calls the operators' entry points with arguments that validation rejects (or
// that leave nothing to do), host code built with sanitizers.  No HIP call is
// reached.  Prints ALL OK.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "moe.h"

static int bad = 0;
#define WANT(expr, status)                                                        \
  do {                                                                            \
    const moe_status_t got = (expr);                                              \
    if (got != (status)) {                                                        \
      printf("%s: got %d, want %d (%s)\n", #expr, (int)got, (int)(status),       \
             moe_last_error());                                                   \
      ++bad;                                                                      \
    }                                                                             \
  } while (0)

static void* at(uint64_t a) { return (void*)(uintptr_t)a; }

int main() {
  const uint64_t K = 1ull << 30;
  size_t n = 0;
  float* f1 = (float*)at(3 * K);
  float* f2 = (float*)at(4 * K);
  const int32_t* off = (const int32_t*)at(16);
  // sizes: small, large, at and past every limit
  const int dims[] = {-1, 0, 1, 7, 64, 2048, 20000, 1 << 20, (1 << 20) + 1, 1 << 24, 0x7fffffff};
  for (int dt = -1; dt <= 2; ++dt)
    for (int a : dims)
      for (int b : dims) {
        (void)moe_layer_norm_backward_workspace_size(a, b, dt, &n);
        (void)moe_orthogonalize_workspace_size(a, b, b, &n);
        (void)moe_orthogonalize_workspace_size(1, a, b, &n);
        for (int e : {0, 1, 64, 1024, 1025}) {
          (void)moe_grouped_matmul_workspace_size(a, e, b, b, dt, &n);
          (void)moe_grouped_matmul_workspace_size(b, e, a, 64, dt, &n);
          for (int want = 0; want < 4; ++want)
            (void)moe_grouped_matmul_backward_workspace_size(b, e, a, 33, dt, want & 1, want >> 1, &n);
        }
      }
  WANT(moe_layer_norm(at(K), at(16), at(K / 2), 4, 0, 1e-5f, 1, at(2 * K), f1, f2, nullptr), MOE_ERR_INVALID_ARG);
  WANT(moe_layer_norm(at(K), at(16), at(K / 2), 4, 64, NAN, 1, at(2 * K), f1, f2, nullptr), MOE_ERR_INVALID_ARG);
  WANT(moe_layer_norm(at(K), at(16), at(K / 2), 4, 64, 0.f, 1, at(K + 64), f1, f2, nullptr), MOE_ERR_INVALID_ARG);
  WANT(moe_layer_norm(at(K), at(16), at(K / 2), 4, 64, 0.f, 1, at(2 * K + 2), f1, f2, nullptr), MOE_ERR_ALIGNMENT);
  WANT(moe_layer_norm(nullptr, nullptr, nullptr, 0, 64, 0.f, 0, nullptr, nullptr, nullptr, nullptr), MOE_OK);
  WANT(moe_layer_norm_backward(at(K), at(2 * K), nullptr, f1, f2, 4, 64, 0, at(5 * K), f1, nullptr, at(6 * K),
                               1 << 20, nullptr), MOE_ERR_INVALID_ARG);
  WANT(moe_layer_norm_backward(at(K), at(2 * K), nullptr, f1, f2, 4, 64, 0, at(5 * K), (float*)at(6 * K), nullptr,
                               at(7 * K), 16, nullptr), MOE_ERR_WORKSPACE);
  WANT(moe_grouped_matmul(at(K), at(2 * K), off, 8, 2, 16, 16, 0, 1, at(K), at(5 * K), K, nullptr), MOE_ERR_INVALID_ARG);
  WANT(moe_grouped_matmul(at(K), at(2 * K), nullptr, 8, 2, 16, 16, 0, 1, at(3 * K), at(5 * K), K, nullptr), MOE_ERR_INVALID_ARG);
  WANT(moe_grouped_matmul(at(K), at(2 * K), off, 8, 2, 16, 16, 0, 1, at(3 * K), at(5 * K), 1, nullptr), MOE_ERR_WORKSPACE);
  WANT(moe_grouped_matmul(nullptr, nullptr, nullptr, 0, 2, 16, 16, 0, 1, nullptr, nullptr, 0, nullptr), MOE_OK);
  WANT(moe_grouped_matmul_backward(at(K), at(2 * K), off, at(7 * K), 8, 2, 16, 16, 1, 1, nullptr, nullptr, at(5 * K), K,
                                   nullptr), MOE_ERR_INVALID_ARG);
  WANT(moe_grouped_matmul_backward(at(K), at(2 * K), off, at(7 * K), 8, 2, 16, 16, 1, 1, at(7 * K), f1, at(5 * K), K,
                                   nullptr), MOE_ERR_INVALID_ARG);
  WANT(moe_grouped_matmul_backward(nullptr, nullptr, nullptr, nullptr, 0, 2, 16, 16, 1, 1, at(7 * K), nullptr, nullptr,
                                   0, nullptr), MOE_OK);
  for (float c : {0.f, 1e-30f, 2.0315f, -2.f, 3e38f, INFINITY, NAN})
    for (float b : {0.f, -4.775f, 1e19f, -3e38f, NAN})
      for (float a : {0.f, 3.4445f, -100.f, 3e38f, -INFINITY})
        for (int steps : {0, 1, 5, 64, 65})
          // no workspace: refused, whatever the coefficients are
          if (moe_orthogonalize(at(K), 64, 1, 8, 8, 0, steps, 1e-7f, a, b, c, at(2 * K), 64, 0, nullptr, 0, nullptr) == MOE_OK)
            ++bad;
  WANT(moe_orthogonalize(at(K), INT64_MAX, 1, 8, 8, 0, 5, 0.f, 1.5f, -.5f, 0.f, at(2 * K), -7, 0, at(3 * K), 0, nullptr),
       MOE_ERR_WORKSPACE);
  WANT(moe_orthogonalize(at(K), -64, 2, 8, 8, 0, 5, 0.f, 1.5f, -.5f, 0.f, at(2 * K), 64, 0, at(3 * K), 0, nullptr),
       MOE_ERR_INVALID_ARG);
  WANT(moe_orthogonalize(at(K), INT64_MAX, 2, 8, 8, 0, 5, 0.f, 1.5f, -.5f, 0.f, at(2 * K), 64, 0, at(3 * K), K, nullptr),
       MOE_ERR_INVALID_ARG);
  if (bad == 0) printf("ALL OK\n");
  return bad != 0;
}
