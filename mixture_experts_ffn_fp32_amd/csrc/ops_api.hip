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

}  // extern "C"
