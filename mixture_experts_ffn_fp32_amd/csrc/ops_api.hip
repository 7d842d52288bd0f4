// C ABI of the operators beside the layer: argument validation, workspace
// checks and launches.  As in the layer's own entry points, validation runs
// before any HIP call, no device memory is allocated and nothing waits.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <string>

#include "moe.h"
#include "ops_internal.h"

namespace {

moe_status_t fail(moe_status_t s, const std::string& msg) {
  moe::set_last_error(msg.c_str());
  return s;
}
moe_status_t ok() {
  moe::set_last_error("");
  return MOE_OK;
}
moe_status_t launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(MOE_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return ok();
}

moe_status_t check_dtype(const char* name, int dtype) {
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)
    return fail(MOE_ERR_UNSUPPORTED,
                std::string(name) + " must be MOE_DTYPE_F32 (0) or MOE_DTYPE_BF16 (1)");
  return MOE_OK;
}
moe_status_t check_ptr(const char* name, const void* p, bool required) {
  if (p == nullptr) {
    if (required) return fail(MOE_ERR_INVALID_ARG, std::string(name) + " is NULL");
    return MOE_OK;
  }
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0)
    return fail(MOE_ERR_ALIGNMENT, std::string(name) + " is not 16-byte aligned");
  return MOE_OK;
}
moe_status_t check_workspace(const void* ws, size_t have, size_t need, const char* query) {
  if (need == 0) return MOE_OK;
  moe_status_t s = check_ptr("workspace", ws, true);
  if (s != MOE_OK) return s;
  if (have < need) return fail(MOE_ERR_WORKSPACE, std::string("workspace smaller than ") + query);
  return MOE_OK;
}
size_t elem_size(int dtype) { return dtype == MOE_DTYPE_BF16 ? 2 : 4; }

// 8-bit types, as the kernels name them (f8.h); 0: another type.
int f8_of(int dtype) {
  return dtype == MOE_DTYPE_E4M3 ? 1 : dtype == MOE_DTYPE_E5M2 ? 2 : 0;
}
moe_status_t check_f8(const char* name, int dtype) {
  if (f8_of(dtype) == 0)
    return fail(MOE_ERR_UNSUPPORTED,
                std::string(name) + " must be MOE_DTYPE_E4M3 (2) or MOE_DTYPE_E5M2 (3)");
  return MOE_OK;
}
size_t blocks_of(int n) { return ((size_t)n + 127) / 128; }

// A buffer of a call: an output must not overlap any other one.
struct Span {
  const char* name;
  const void* p;
  size_t bytes;
  bool written;
};
moe_status_t check_overlaps(const Span* s, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j) {
      if (i == j || !s[i].written || (s[j].written && j < i)) continue;
      if (s[i].p == nullptr || s[j].p == nullptr || s[i].bytes == 0 || s[j].bytes == 0) continue;
      const uintptr_t a = (uintptr_t)s[i].p, b = (uintptr_t)s[j].p;
      if (a < b + s[j].bytes && b < a + s[i].bytes)
        return fail(MOE_ERR_INVALID_ARG, std::string(s[i].name) + " overlaps " + s[j].name);
    }
  return MOE_OK;
}

// ---------------------------------------------------------------- layer norm
moe_status_t check_norm(int T, int d, int dtype) {
  moe_status_t s = check_dtype("dtype", dtype);
  if (s != MOE_OK) return s;
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T must be >= 0");
  if (d < 1) return fail(MOE_ERR_INVALID_ARG, "d must be positive");
  if (d > (1 << 24)) return fail(MOE_ERR_UNSUPPORTED, "d > 2^24 is not supported");
  return MOE_OK;
}
size_t norm_bwd_bytes(int T, int d, int dtype) {
  return T == 0 ? 0 : (size_t)moe::layer_norm_chunks(dtype, T, d) * 2 * d * 4;
}

// ---------------------------------------------------------------- grouped products
moe_status_t check_grouped(int M, int E, int n, int k, int dtype) {
  moe_status_t s = check_dtype("dtype", dtype);
  if (s != MOE_OK) return s;
  if (M < 0) return fail(MOE_ERR_INVALID_ARG, "M must be >= 0");
  if (E < 1) return fail(MOE_ERR_INVALID_ARG, "E must be >= 1");
  if (E > moe::kGroupedMaxE)
    return fail(MOE_ERR_UNSUPPORTED, "E > " + std::to_string(moe::kGroupedMaxE) + " groups is not supported");
  if (n < 1) return fail(MOE_ERR_INVALID_ARG, "n must be positive");
  if (k < 1) return fail(MOE_ERR_INVALID_ARG, "k must be positive");
  // rows are addressed as 32-bit byte offsets from a tile's first row
  const long long row = 4 * (((long long)std::max(n, k) + 63) / 64 * 64);
  if (row > moe::kGroupedMaxRowBytes)
    return fail(MOE_ERR_UNSUPPORTED, "n and k must stay at or below " +
                                         std::to_string(moe::kGroupedMaxRowBytes / 4));
  const long long tiles = ((long long)M / 64 + 1 + E) * ((std::max(n, k) + 63LL) / 64);
  const long long wtiles = (long long)E * ((n + 63LL) / 64) * ((k + 63LL) / 64);
  if (std::max(tiles, wtiles) > 0x3fffffffLL || (long long)E * n > 0x7fffffffLL)
    return fail(MOE_ERR_UNSUPPORTED, "M, E, n, k give too many tiles");
  return MOE_OK;
}

// ---------------------------------------------------------------- orthogonalised update
moe_status_t check_ortho(int B, int m, int n) {
  if (B < 0) return fail(MOE_ERR_INVALID_ARG, "B must be >= 0");
  if (B > 65535) return fail(MOE_ERR_UNSUPPORTED, "B > 65535 matrices is not supported");
  if (m < 1 || n < 1) return fail(MOE_ERR_INVALID_ARG, "m and n must be positive");
  if (m > (1 << 20) || n > (1 << 20))
    return fail(MOE_ERR_UNSUPPORTED, "m and n must stay at or below 2^20");
  const long long mt = (m + 63LL) / 64, nt = (n + 63LL) / 64;
  if (mt * nt * std::max(B, 1) > 0x3fffffffLL || (long long)B * m > 0x7fffffffLL)
    return fail(MOE_ERR_UNSUPPORTED, "B, m, n give too many tiles");
  return MOE_OK;
}

// ---------------------------------------------------------------- RMS norm
size_t rms_bwd_bytes(int T, int d, int dtype) {
  return T == 0 ? 0 : (size_t)moe::rms_norm_chunks(dtype, T, d) * d * 4;
}

// ---------------------------------------------------------------- 8-bit grouped products
moe_status_t grouped_f8_size(bool dx, int M, int E, int n, int k, size_t* bytes) {
  moe_status_t s = check_grouped(M, E, n, k, MOE_DTYPE_F32);
  if (s != MOE_OK) return s;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = M == 0 ? 0 : moe::grouped_f8_workspace_bytes(M, E, n, k, dx);
  return ok();
}
moe_status_t grouped_f8(bool dx, const void* x, const float* xs, const void* w, const float* ws,
                        const int32_t* offsets, int M, int E, int n, int k, int x_dtype,
                        int out_dtype, int zero_rest, void* out, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  moe_status_t s = check_grouped(M, E, n, k, MOE_DTYPE_F32);
  if (s != MOE_OK) return s;
  if ((s = check_f8(dx ? "dy_dtype" : "x_dtype", x_dtype)) != MOE_OK) return s;
  if ((s = check_dtype("out_dtype", out_dtype)) != MOE_OK) return s;
  if (M == 0) return ok();
  if ((s = check_ptr(dx ? "dy" : "x", x, true)) != MOE_OK) return s;
  if ((s = check_ptr(dx ? "dys" : "xs", xs, true)) != MOE_OK) return s;
  if ((s = check_ptr("w", w, true)) != MOE_OK) return s;
  if ((s = check_ptr("ws", ws, true)) != MOE_OK) return s;
  if ((s = check_ptr("offsets", offsets, E > 1)) != MOE_OK) return s;
  if ((s = check_ptr(dx ? "dx" : "y", out, true)) != MOE_OK) return s;
  const size_t need = moe::grouped_f8_workspace_bytes(M, E, n, k, dx);
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           dx ? "moe_grouped_matmul_quantized_dx_workspace_size()"
                              : "moe_grouped_matmul_quantized_workspace_size()")) != MOE_OK)
    return s;
  const int in = dx ? n : k, width = dx ? k : n;
  const Span spans[] = {{dx ? "dy" : "x", x, (size_t)M * in, false},
                        {dx ? "dys" : "xs", xs, (size_t)M * blocks_of(in) * 4, false},
                        {"w", w, (size_t)E * n * k, false},
                        {"ws", ws, E * blocks_of(n) * blocks_of(k) * 4, false},
                        {"offsets", offsets, (size_t)(E + 1) * 4, false},
                        {dx ? "dx" : "y", out, (size_t)M * width * elem_size(out_dtype), true},
                        {"workspace", workspace, need, true}};
  if ((s = check_overlaps(spans, 7)) != MOE_OK) return s;
  moe::GroupedF8Args a{};
  a.x = x;
  a.xs = xs;
  a.w = w;
  a.ws = ws;
  a.offsets = offsets;
  a.out = out;
  a.M = M;
  a.E = E;
  a.n = n;
  a.k = k;
  a.zero_rest = zero_rest != 0;
  a.out_f32 = out_dtype == MOE_DTYPE_F32;
  return launched(moe::launch_grouped_f8(f8_of(x_dtype), dx, a, workspace, stream),
                  "8-bit grouped product launch");
}

// ---------------------------------------------------------------- balance loss
moe_status_t check_balance_loss(int T, int N, int S) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T must be >= 0");
  if (N < 1) return fail(MOE_ERR_INVALID_ARG, "N must be >= 1");
  if (N > 256) return fail(MOE_ERR_UNSUPPORTED, "N > 256 routed experts is not supported");
  if (S < 1) return fail(MOE_ERR_INVALID_ARG, "S must be >= 1");
  if (S > moe::kGroupedMaxE)
    return fail(MOE_ERR_UNSUPPORTED,
                "S > " + std::to_string(moe::kGroupedMaxE) + " sequences is not supported");
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_layer_norm(const void* x, const void* weight, const void* bias, int T, int d,
                            float eps, int dtype, void* y, float* mean, float* rstd,
                            void* stream) {
  moe_status_t s = check_norm(T, d, dtype);
  if (s != MOE_OK) return s;
  if (!(eps >= 0.f) || isinf(eps)) return fail(MOE_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (T == 0) return ok();
  if ((s = check_ptr("x", x, true)) != MOE_OK) return s;
  if ((s = check_ptr("weight", weight, false)) != MOE_OK) return s;
  if ((s = check_ptr("bias", bias, false)) != MOE_OK) return s;
  if ((s = check_ptr("y", y, true)) != MOE_OK) return s;
  if ((s = check_ptr("mean", mean, false)) != MOE_OK) return s;
  if ((s = check_ptr("rstd", rstd, false)) != MOE_OK) return s;
  const size_t es = elem_size(dtype), act = (size_t)T * d * es, vec = (size_t)d * es;
  const Span spans[] = {{"x", x, act, false},        {"weight", weight, vec, false},
                        {"bias", bias, vec, false},  {"y", y, act, true},
                        {"mean", mean, (size_t)T * 4, true}, {"rstd", rstd, (size_t)T * 4, true}};
  if ((s = check_overlaps(spans, 6)) != MOE_OK) return s;
  moe::NormArgs a{};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.out = y;
  a.mean = mean;
  a.rstd = rstd;
  a.T = T;
  a.d = d;
  a.eps = eps;
  return launched(moe::launch_layer_norm(dtype, a, (hipStream_t)stream), "layer norm launch");
}

moe_status_t moe_layer_norm_backward_workspace_size(int T, int d, int dtype, size_t* bytes) {
  moe_status_t s = check_norm(T, d, dtype);
  if (s != MOE_OK) return s;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = norm_bwd_bytes(T, d, dtype);
  return ok();
}

moe_status_t moe_layer_norm_backward(const void* dy, const void* x, const void* weight,
                                     const float* mean, const float* rstd, int T, int d, int dtype,
                                     void* dx, float* dweight, float* dbias, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  moe_status_t s = check_norm(T, d, dtype);
  if (s != MOE_OK) return s;
  if ((s = check_ptr("dy", dy, T > 0)) != MOE_OK) return s;
  if ((s = check_ptr("x", x, T > 0)) != MOE_OK) return s;
  if ((s = check_ptr("weight", weight, false)) != MOE_OK) return s;
  if ((s = check_ptr("mean", mean, T > 0)) != MOE_OK) return s;
  if ((s = check_ptr("rstd", rstd, T > 0)) != MOE_OK) return s;
  if ((s = check_ptr("dx", dx, T > 0)) != MOE_OK) return s;
  if ((s = check_ptr("dweight", dweight, false)) != MOE_OK) return s;
  if ((s = check_ptr("dbias", dbias, false)) != MOE_OK) return s;
  const size_t need = dweight != nullptr || dbias != nullptr ? norm_bwd_bytes(T, d, dtype) : 0;
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "moe_layer_norm_backward_workspace_size()")) != MOE_OK)
    return s;
  const size_t es = elem_size(dtype), act = (size_t)T * d * es;
  const Span spans[] = {{"dy", dy, act, false},
                        {"x", x, act, false},
                        {"weight", weight, d * es, false},
                        {"mean", mean, (size_t)T * 4, false},
                        {"rstd", rstd, (size_t)T * 4, false},
                        {"dx", dx, act, true},
                        {"dweight", dweight, (size_t)d * 4, true},
                        {"dbias", dbias, (size_t)d * 4, true},
                        {"workspace", workspace, need, true}};
  if ((s = check_overlaps(spans, 9)) != MOE_OK) return s;
  moe::NormArgs a{};
  a.x = x;
  a.weight = weight;
  a.dy = dy;
  a.out = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.part = (float*)workspace;
  a.dweight = dweight;
  a.dbias = dbias;
  a.T = T;
  a.d = d;
  return launched(moe::launch_layer_norm_backward(dtype, a, (hipStream_t)stream),
                  "layer norm backward launch");
}

moe_status_t moe_grouped_matmul_workspace_size(int M, int E, int n, int k, int dtype,
                                               size_t* bytes) {
  moe_status_t s = check_grouped(M, E, n, k, dtype);
  if (s != MOE_OK) return s;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = M == 0 ? 0 : moe::grouped_workspace_bytes(dtype, M, E, n, k);
  return ok();
}

moe_status_t moe_grouped_matmul(const void* x, const void* w, const int32_t* offsets, int M, int E,
                                int n, int k, int dtype, int zero_rest, void* y, void* workspace,
                                size_t workspace_bytes, void* stream) {
  moe_status_t s = check_grouped(M, E, n, k, dtype);
  if (s != MOE_OK) return s;
  if (M == 0) return ok();
  if ((s = check_ptr("x", x, true)) != MOE_OK) return s;
  if ((s = check_ptr("w", w, true)) != MOE_OK) return s;
  if ((s = check_ptr("offsets", offsets, true)) != MOE_OK) return s;
  if ((s = check_ptr("y", y, true)) != MOE_OK) return s;
  const size_t need = moe::grouped_workspace_bytes(dtype, M, E, n, k);
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "moe_grouped_matmul_workspace_size()")) != MOE_OK)
    return s;
  const size_t es = elem_size(dtype);
  const Span spans[] = {{"x", x, (size_t)M * k * es, false},
                        {"w", w, (size_t)E * n * k * es, false},
                        {"offsets", offsets, (size_t)(E + 1) * 4, false},
                        {"y", y, (size_t)M * n * es, true},
                        {"workspace", workspace, need, true}};
  if ((s = check_overlaps(spans, 5)) != MOE_OK) return s;
  moe::GroupedArgs a{};
  a.x = x;
  a.w = w;
  a.offsets = offsets;
  a.y = y;
  a.M = M;
  a.E = E;
  a.n = n;
  a.k = k;
  a.zero_rest = zero_rest != 0;
  return launched(moe::launch_grouped(dtype, a, workspace, (hipStream_t)stream),
                  "grouped product launch");
}

moe_status_t moe_grouped_matmul_backward_workspace_size(int M, int E, int n, int k, int dtype,
                                                        int want_dx, int want_dw, size_t* bytes) {
  moe_status_t s = check_grouped(M, E, n, k, dtype);
  if (s != MOE_OK) return s;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = moe::grouped_backward_workspace_bytes(dtype, M, E, n, k, want_dx != 0, want_dw != 0);
  return ok();
}

moe_status_t moe_grouped_matmul_backward(const void* x, const void* w, const int32_t* offsets,
                                         const void* dy, int M, int E, int n, int k, int dtype,
                                         int zero_rest, void* dx, float* dw, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  moe_status_t s = check_grouped(M, E, n, k, dtype);
  if (s != MOE_OK) return s;
  // (without rows dx has no elements, and its pointer may be NULL)
  if (M == 0 && dw == nullptr) return ok();
  if (dx == nullptr && dw == nullptr)
    return fail(MOE_ERR_INVALID_ARG, "dx and dw are both NULL: nothing to compute");
  if ((s = check_ptr("x", x, M > 0 && dw != nullptr)) != MOE_OK) return s;
  if ((s = check_ptr("w", w, M > 0 && dx != nullptr)) != MOE_OK) return s;
  if ((s = check_ptr("offsets", offsets, true)) != MOE_OK) return s;
  if ((s = check_ptr("dy", dy, M > 0)) != MOE_OK) return s;
  if ((s = check_ptr("dx", dx, false)) != MOE_OK) return s;
  if ((s = check_ptr("dw", dw, false)) != MOE_OK) return s;
  const bool want_dx = dx != nullptr && M > 0;
  const size_t need =
      moe::grouped_backward_workspace_bytes(dtype, M, E, n, k, want_dx, dw != nullptr);
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "moe_grouped_matmul_backward_workspace_size()")) != MOE_OK)
    return s;
  const size_t es = elem_size(dtype);
  const Span spans[] = {{"x", x, (size_t)M * k * es, false},
                        {"w", w, (size_t)E * n * k * es, false},
                        {"offsets", offsets, (size_t)(E + 1) * 4, false},
                        {"dy", dy, (size_t)M * n * es, false},
                        {"dx", dx, (size_t)M * k * es, true},
                        {"dw", dw, (size_t)E * n * k * 4, true},
                        {"workspace", workspace, need, true}};
  if ((s = check_overlaps(spans, 7)) != MOE_OK) return s;
  moe::GroupedArgs a{};
  a.x = x;
  a.w = w;
  a.dy = dy;
  a.offsets = offsets;
  a.dx = want_dx ? dx : nullptr;
  a.dw = dw;
  a.M = M;
  a.E = E;
  a.n = n;
  a.k = k;
  a.zero_rest = zero_rest != 0;
  return launched(moe::launch_grouped_backward(dtype, a, workspace, (hipStream_t)stream),
                  "grouped product backward launch");
}

moe_status_t moe_orthogonalize_workspace_size(int B, int m, int n, size_t* bytes) {
  moe_status_t s = check_ortho(B, m, n);
  if (s != MOE_OK) return s;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = B == 0 ? 0 : moe::ortho_workspace_bytes(B, m, n);
  return ok();
}

moe_status_t moe_orthogonalize(const void* x, int64_t x_stride, int B, int m, int n, int dtype,
                               int steps, float eps, float a, float b, float c, void* out,
                               int64_t out_stride, int out_dtype, void* workspace,
                               size_t workspace_bytes, void* stream) {
  moe_status_t s = check_ortho(B, m, n);
  if (s != MOE_OK) return s;
  if ((s = check_dtype("dtype", dtype)) != MOE_OK) return s;
  if ((s = check_dtype("out_dtype", out_dtype)) != MOE_OK) return s;
  if (steps < 0 || steps > 64)
    return fail(MOE_ERR_INVALID_ARG, "steps must satisfy 0 <= steps <= 64");
  if (!(eps >= 0.f) || isinf(eps)) return fail(MOE_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!isfinite(a) || !isfinite(b) || !isfinite(c))
    return fail(MOE_ERR_INVALID_ARG, "the coefficients must be finite");
  double iterate = 0.0, factor = 0.0;
  moe::ortho_bounds(steps, a, b, c, &iterate, &factor);
  if (!(iterate * iterate <= moe::kOrthoMaxBound) || !(factor <= moe::kOrthoMaxBound))
    return fail(MOE_ERR_UNSUPPORTED,
                "the coefficients let the iterate grow past the range its products are held in");
  // P comes from the completed square, which cancels b^2 / (4 c) against a
  if (c != 0.f && !((double)b * b <= 64.0 * fabs((double)c)))
    return fail(MOE_ERR_UNSUPPORTED, "the coefficients must satisfy c == 0 or b * b <= 64 |c|");
  if (B == 0) return ok();
  const int64_t per = (int64_t)m * n;
  if (B > 1 && (x_stride < per || out_stride < per))
    return fail(MOE_ERR_INVALID_ARG, "x_stride and out_stride must be at least m * n");
  if (B > 1 && std::max(x_stride, out_stride) > INT64_MAX / 8 / B)
    return fail(MOE_ERR_INVALID_ARG, "x_stride and out_stride reach past the address space");
  const size_t es = elem_size(dtype), eo = elem_size(out_dtype);
  if (B > 1 && ((x_stride * es) % 16 != 0 || (out_stride * eo) % 16 != 0) &&
      (x_stride != per || out_stride != per))
    return fail(MOE_ERR_ALIGNMENT, "matrices that are not back to back must start 16-byte aligned");
  if ((s = check_ptr("x", x, true)) != MOE_OK) return s;
  if ((s = check_ptr("out", out, true)) != MOE_OK) return s;
  const size_t need = moe::ortho_workspace_bytes(B, m, n);
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "moe_orthogonalize_workspace_size()")) != MOE_OK)
    return s;
  const size_t xb = ((size_t)(B - 1) * x_stride + per) * es,
               ob = ((size_t)(B - 1) * out_stride + per) * eo;
  // in place: the same matrices, read whole before the first result is written
  const bool in_place = x == out && dtype == out_dtype && (B == 1 || x_stride == out_stride);
  const Span spans[] = {{"x", in_place ? nullptr : x, xb, false},
                        {"out", out, ob, true},
                        {"workspace", workspace, need, true},
                        {"x", x, xb, false}};
  if ((s = check_overlaps(spans, 3)) != MOE_OK) return s;
  if ((s = check_overlaps(spans + 2, 2)) != MOE_OK) return s;
  moe::OrthoArgs o{};
  o.x = x;
  o.out = out;
  o.x_stride = B > 1 ? x_stride : per;
  o.out_stride = B > 1 ? out_stride : per;
  o.B = B;
  o.m = m;
  o.n = n;
  o.steps = steps;
  o.dtype = dtype;
  o.out_dtype = out_dtype;
  o.eps = eps;
  o.a = a;
  o.b = b;
  o.c = c;
  o.most_x = iterate;
  o.most_p = factor;
  return launched(moe::launch_orthogonalize(o, workspace, (hipStream_t)stream),
                  "orthogonalise launch");
}

moe_status_t moe_rms_norm(const void* x, const void* residual, const void* weight, int T, int d,
                          float eps, int dtype, int y_dtype, void* h, void* y, float* scales,
                          float* rstd, void* stream) {
  moe_status_t s = check_norm(T, d, dtype);
  if (s != MOE_OK) return s;
  const int f8 = f8_of(y_dtype);
  if (f8 == 0 && y_dtype != dtype)
    return fail(MOE_ERR_UNSUPPORTED, "y_dtype must be dtype, MOE_DTYPE_E4M3 or MOE_DTYPE_E5M2");
  if (!(eps >= 0.f) || isinf(eps)) return fail(MOE_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (f8 == 0 && scales != nullptr)
    return fail(MOE_ERR_INVALID_ARG, "scales belong to an 8-bit y only");
  if (T == 0) return ok();
  if ((s = check_ptr("x", x, true)) != MOE_OK) return s;
  if ((s = check_ptr("residual", residual, false)) != MOE_OK) return s;
  if ((s = check_ptr("weight", weight, false)) != MOE_OK) return s;
  if ((s = check_ptr("h", h, false)) != MOE_OK) return s;
  if ((s = check_ptr("y", y, true)) != MOE_OK) return s;
  if ((s = check_ptr("scales", scales, f8 != 0)) != MOE_OK) return s;
  if ((s = check_ptr("rstd", rstd, false)) != MOE_OK) return s;
  const size_t es = elem_size(dtype), act = (size_t)T * d * es;
  // h may stand in x's or the residual's place: a thread reads its elements of a row before it
  // writes them
  const Span spans[] = {{"x", h == x ? nullptr : x, act, false},
                        {"residual", h == residual ? nullptr : residual, act, false},
                        {"weight", weight, (size_t)d * es, false},
                        {"h", h, act, true},
                        {"y", y, (size_t)T * d * (f8 != 0 ? 1 : es), true},
                        {"scales", scales, (size_t)T * blocks_of(d) * 4, true},
                        {"rstd", rstd, (size_t)T * 4, true}};
  if ((s = check_overlaps(spans, 7)) != MOE_OK) return s;
  moe::RmsArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.h = h;
  a.out = y;
  a.scales = scales;
  a.rstd = rstd;
  a.T = T;
  a.d = d;
  a.eps = eps;
  return launched(moe::launch_rms_norm(dtype, f8, a, (hipStream_t)stream), "RMS norm launch");
}

moe_status_t moe_rms_norm_backward_workspace_size(int T, int d, int dtype, size_t* bytes) {
  moe_status_t s = check_norm(T, d, dtype);
  if (s != MOE_OK) return s;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = rms_bwd_bytes(T, d, dtype);
  return ok();
}

moe_status_t moe_rms_norm_backward(const void* dy, const void* h, const void* weight,
                                   const float* rstd, const void* dh, int T, int d, int dtype,
                                   void* dx, float* dweight, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  moe_status_t s = check_norm(T, d, dtype);
  if (s != MOE_OK) return s;
  if ((s = check_ptr("dy", dy, T > 0)) != MOE_OK) return s;
  if ((s = check_ptr("h", h, T > 0)) != MOE_OK) return s;
  if ((s = check_ptr("weight", weight, false)) != MOE_OK) return s;
  if ((s = check_ptr("rstd", rstd, T > 0)) != MOE_OK) return s;
  if ((s = check_ptr("dh", dh, false)) != MOE_OK) return s;
  if ((s = check_ptr("dx", dx, T > 0)) != MOE_OK) return s;
  if ((s = check_ptr("dweight", dweight, false)) != MOE_OK) return s;
  const size_t need = dweight != nullptr ? rms_bwd_bytes(T, d, dtype) : 0;
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "moe_rms_norm_backward_workspace_size()")) != MOE_OK)
    return s;
  const size_t es = elem_size(dtype), act = (size_t)T * d * es;
  const Span spans[] = {{"dy", dy, act, false},
                        {"h", h, act, false},
                        {"weight", weight, d * es, false},
                        {"rstd", rstd, (size_t)T * 4, false},
                        {"dh", dh == dx ? nullptr : dh, act, false},
                        {"dx", dx, act, true},
                        {"dweight", dweight, (size_t)d * 4, true},
                        {"workspace", workspace, need, true}};
  if ((s = check_overlaps(spans, 8)) != MOE_OK) return s;
  moe::RmsArgs a{};
  a.x = h;
  a.weight = weight;
  a.dy = dy;
  a.dh = dh;
  a.out = dx;
  a.rstd = const_cast<float*>(rstd);
  a.part = (float*)workspace;
  a.dweight = dweight;
  a.T = T;
  a.d = d;
  return launched(moe::launch_rms_norm_backward(dtype, a, (hipStream_t)stream),
                  "RMS norm backward launch");
}

moe_status_t moe_quantize_rows(const void* x, int T, int d, int dtype, int q_dtype, void* q,
                               float* scales, void* stream) {
  moe_status_t s = check_norm(T, d, dtype);
  if (s != MOE_OK) return s;
  if ((s = check_f8("q_dtype", q_dtype)) != MOE_OK) return s;
  if (T == 0) return ok();
  if ((s = check_ptr("x", x, true)) != MOE_OK) return s;
  if ((s = check_ptr("q", q, true)) != MOE_OK) return s;
  if ((s = check_ptr("scales", scales, true)) != MOE_OK) return s;
  const Span spans[] = {{"x", x, (size_t)T * d * elem_size(dtype), false},
                        {"q", q, (size_t)T * d, true},
                        {"scales", scales, T * blocks_of(d) * 4, true}};
  if ((s = check_overlaps(spans, 3)) != MOE_OK) return s;
  return launched(
      moe::launch_quantize_rows(dtype, f8_of(q_dtype), x, T, d, q, scales, (hipStream_t)stream),
      "quantise launch");
}

moe_status_t moe_quantize_blocks(const void* w, int E, int n, int k, int dtype, int q_dtype,
                                 void* q, float* scales, void* stream) {
  moe_status_t s = check_dtype("dtype", dtype);
  if (s != MOE_OK) return s;
  if ((s = check_f8("q_dtype", q_dtype)) != MOE_OK) return s;
  if (E < 0) return fail(MOE_ERR_INVALID_ARG, "E must be >= 0");
  if (n < 1 || k < 1) return fail(MOE_ERR_INVALID_ARG, "n and k must be positive");
  if (n > (1 << 20) || k > (1 << 20))
    return fail(MOE_ERR_UNSUPPORTED, "n and k must stay at or below 2^20");
  const size_t blocks = blocks_of(n) * blocks_of(k);
  if ((size_t)E * blocks > (size_t)1 << 23)
    return fail(MOE_ERR_UNSUPPORTED, "more than 2^23 blocks of 128 x 128 are not supported");
  if (E == 0) return ok();
  if ((s = check_ptr("w", w, true)) != MOE_OK) return s;
  if ((s = check_ptr("q", q, true)) != MOE_OK) return s;
  if ((s = check_ptr("scales", scales, true)) != MOE_OK) return s;
  const size_t all = (size_t)E * n * k;
  const Span spans[] = {{"w", w, all * elem_size(dtype), false},
                        {"q", q, all, true},
                        {"scales", scales, E * blocks * 4, true}};
  if ((s = check_overlaps(spans, 3)) != MOE_OK) return s;
  return launched(moe::launch_quantize_blocks(dtype, f8_of(q_dtype), w, E, n, k, q, scales,
                                              (hipStream_t)stream),
                  "quantise launch");
}

moe_status_t moe_dequantize_rows(const void* q, const float* scales, int T, int d, int q_dtype,
                                 int dtype, void* x, void* stream) {
  moe_status_t s = check_norm(T, d, dtype);
  if (s != MOE_OK) return s;
  if ((s = check_f8("q_dtype", q_dtype)) != MOE_OK) return s;
  if (T == 0) return ok();
  if ((s = check_ptr("q", q, true)) != MOE_OK) return s;
  if ((s = check_ptr("scales", scales, true)) != MOE_OK) return s;
  if ((s = check_ptr("x", x, true)) != MOE_OK) return s;
  const Span spans[] = {{"q", q, (size_t)T * d, false},
                        {"scales", scales, T * blocks_of(d) * 4, false},
                        {"x", x, (size_t)T * d * elem_size(dtype), true}};
  if ((s = check_overlaps(spans, 3)) != MOE_OK) return s;
  return launched(
      moe::launch_dequantize_rows(f8_of(q_dtype), dtype, q, scales, T, d, x, (hipStream_t)stream),
      "dequantise launch");
}

moe_status_t moe_grouped_matmul_quantized_workspace_size(int M, int E, int n, int k,
                                                         size_t* bytes) {
  return grouped_f8_size(false, M, E, n, k, bytes);
}

moe_status_t moe_grouped_matmul_quantized(const void* x, const float* xs, const void* w,
                                          const float* ws, const int32_t* offsets, int M, int E,
                                          int n, int k, int x_dtype, int out_dtype, int zero_rest,
                                          void* y, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  return grouped_f8(false, x, xs, w, ws, offsets, M, E, n, k, x_dtype, out_dtype, zero_rest, y,
                    workspace, workspace_bytes, (hipStream_t)stream);
}

moe_status_t moe_grouped_matmul_quantized_dx_workspace_size(int M, int E, int n, int k,
                                                            size_t* bytes) {
  return grouped_f8_size(true, M, E, n, k, bytes);
}

moe_status_t moe_grouped_matmul_quantized_dx(const void* dy, const float* dys, const void* w,
                                             const float* ws, const int32_t* offsets, int M, int E,
                                             int n, int k, int dy_dtype, int out_dtype,
                                             int zero_rest, void* dx, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  return grouped_f8(true, dy, dys, w, ws, offsets, M, E, n, k, dy_dtype, out_dtype, zero_rest, dx,
                    workspace, workspace_bytes, (hipStream_t)stream);
}

moe_status_t moe_balance_loss_workspace_size(int T, int N, int S, size_t* bytes) {
  moe_status_t s = check_balance_loss(T, N, S);
  if (s != MOE_OK) return s;
  if (bytes == nullptr) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = T == 0 ? 0 : moe::balance_loss_workspace_bytes(T, N, S);
  return ok();
}

moe_status_t moe_balance_loss(const float* scores, const int32_t* idx, const int32_t* offsets,
                              const uint8_t* mask, const int32_t* device_of, int T, int N, int K,
                              int S, int D, float alpha1, float alpha2, int32_t* counts, float* P,
                              float* losses, float* slopes, void* workspace,
                              size_t workspace_bytes, void* stream) {
  moe_status_t s = check_balance_loss(T, N, S);
  if (s != MOE_OK) return s;
  if (K < 1 || K > N) return fail(MOE_ERR_INVALID_ARG, "K must satisfy 1 <= K <= N");
  if ((long long)T * K > 0x7fffffffLL)
    return fail(MOE_ERR_UNSUPPORTED, "T * K must stay below 2^31");
  if (D < 0) return fail(MOE_ERR_INVALID_ARG, "D must be >= 0");
  if (D > 256) return fail(MOE_ERR_UNSUPPORTED, "D > 256 devices is not supported");
  if (device_of != nullptr && D == 0)
    return fail(MOE_ERR_INVALID_ARG, "device_of needs the number of devices D");
  if (!isfinite(alpha1) || !isfinite(alpha2))
    return fail(MOE_ERR_INVALID_ARG, "alpha1 and alpha2 must be finite");
  if ((s = check_ptr("scores", scores, T > 0)) != MOE_OK) return s;
  if ((s = check_ptr("idx", idx, T > 0)) != MOE_OK) return s;
  if ((s = check_ptr("offsets", offsets, S > 1)) != MOE_OK) return s;
  if ((s = check_ptr("mask", mask, false)) != MOE_OK) return s;
  if ((s = check_ptr("device_of", device_of, false)) != MOE_OK) return s;
  if ((s = check_ptr("counts", counts, true)) != MOE_OK) return s;
  if ((s = check_ptr("P", P, true)) != MOE_OK) return s;
  if ((s = check_ptr("losses", losses, true)) != MOE_OK) return s;
  if ((s = check_ptr("slopes", slopes, true)) != MOE_OK) return s;
  const size_t need = T == 0 ? 0 : moe::balance_loss_workspace_bytes(T, N, S);
  if ((s = check_workspace(workspace, workspace_bytes, need,
                           "moe_balance_loss_workspace_size()")) != MOE_OK)
    return s;
  const size_t per = (size_t)S * N * 4;
  const Span spans[] = {{"scores", scores, (size_t)T * N * 4, false},
                        {"idx", idx, (size_t)T * K * 4, false},
                        {"offsets", offsets, (size_t)(S + 1) * 4, false},
                        {"mask", mask, (size_t)T, false},
                        {"device_of", device_of, (size_t)N * 4, false},
                        {"counts", counts, per, true},
                        {"P", P, per, true},
                        {"losses", losses, (size_t)S * 8, true},
                        {"slopes", slopes, 2 * per, true},
                        {"workspace", workspace, need, true}};
  if ((s = check_overlaps(spans, 10)) != MOE_OK) return s;
  moe::BalanceLossArgs a{};
  a.scores = scores;
  a.idx = idx;
  a.offsets = offsets;
  a.mask = mask;
  a.device_of = device_of;
  a.counts = counts;
  a.P = P;
  a.losses = losses;
  a.slopes = slopes;
  a.T = T;
  a.N = N;
  a.K = K;
  a.S = S;
  a.D = D;
  a.alpha1 = alpha1;
  a.alpha2 = alpha2;
  return launched(moe::launch_balance_loss(a, workspace, (hipStream_t)stream),
                  "balance loss launch");
}

moe_status_t moe_balance_loss_backward(const float* scores, const float* slopes,
                                       const float* dlosses, const int32_t* offsets,
                                       const uint8_t* mask, int T, int N, int S, float* dlogits,
                                       void* stream) {
  moe_status_t s = check_balance_loss(T, N, S);
  if (s != MOE_OK) return s;
  if (T == 0) return ok();
  if ((s = check_ptr("scores", scores, true)) != MOE_OK) return s;
  if ((s = check_ptr("slopes", slopes, true)) != MOE_OK) return s;
  if ((s = check_ptr("dlosses", dlosses, false)) != MOE_OK) return s;
  if ((s = check_ptr("offsets", offsets, S > 1)) != MOE_OK) return s;
  if ((s = check_ptr("mask", mask, false)) != MOE_OK) return s;
  if ((s = check_ptr("dlogits", dlogits, true)) != MOE_OK) return s;
  const Span spans[] = {{"scores", scores, (size_t)T * N * 4, false},
                        {"slopes", slopes, (size_t)S * N * 8, false},
                        {"dlosses", dlosses, (size_t)S * 8, false},
                        {"offsets", offsets, (size_t)(S + 1) * 4, false},
                        {"mask", mask, (size_t)T, false},
                        {"dlogits", dlogits, (size_t)T * N * 4, true}};
  if ((s = check_overlaps(spans, 6)) != MOE_OK) return s;
  moe::BalanceLossArgs a{};
  a.scores = scores;
  a.slopes = const_cast<float*>(slopes);
  a.dlosses = dlosses;
  a.offsets = offsets;
  a.mask = mask;
  a.dlogits = dlogits;
  a.T = T;
  a.N = N;
  a.S = S;
  return launched(moe::launch_balance_loss_backward(a, (hipStream_t)stream),
                  "balance loss backward launch");
}

}  // extern "C"
