// Launch code of the operators beside the layer under sanitizers, on the CPU: their host objects
// are linked with the few runtime calls below, which take a launch's sizes and run nothing.  Every
// launch has to hold fewer than 2^32 threads along each of its sides (beyond, blocks are left
// out without an error).
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>
#include <string>

#include "groups.h"
#include "moe.h"

static int failures = 0;
static std::string what, error;
static long long launches = 0;
static dim3 grid, block;

namespace moe {
void set_last_error(const char* msg) { error = msg; }
}  // namespace moe

extern "C" {
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t, hipStream_t) {
  grid = g;
  block = b;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* g, dim3* b, size_t* shared, hipStream_t* st) {
  *g = grid;
  *b = block;
  *shared = 0;
  *st = nullptr;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 g, dim3 b, void**, size_t, hipStream_t) {
  ++launches;
  const uint64_t n[3] = {(uint64_t)g.x * b.x, (uint64_t)g.y * b.y, (uint64_t)g.z * b.z};
  if (n[0] == 0 || n[1] == 0 || n[2] == 0 || (n[0] | n[1] | n[2]) >> 32 != 0 || g.y > 65535 || g.z > 65535 ||
      b.x * b.y * b.z > 1024) {
    printf("%s: %u x %u x %u blocks of %u x %u x %u threads\n", what.c_str(), g.x, g.y, g.z, b.x, b.y, b.z);
    ++failures;
  }
  return hipSuccess;
}
void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, dim3*, dim3*, int*) {}
hipError_t hipGetLastError(void) { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return ""; }
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
  *v = 256;
  return hipSuccess;
}
}

// Buffers of up to 2^40 bytes.
static void* at(int i) { return (void*)((uintptr_t)(i + 1) << 40); }
static float* fl(int i) { return (float*)at(i); }
static int32_t* in(int i) { return (int32_t*)at(i); }

static void took(int status, const std::string& call) {
  if (status != MOE_OK) {
    printf("%s: status %d (%s)\n", call.c_str(), status, error.c_str());
    ++failures;
  }
}
#define RUN(name, call)                                        \
  do {                                                         \
    what = name;                                               \
    const long long before = launches;                         \
    took(call, what);                                          \
    if (launches == before) {                                  \
      printf("%s: nothing was launched\n", what.c_str());      \
      ++failures;                                              \
    }                                                          \
  } while (0)

static const size_t kRoom = (size_t)1 << 40;
static const int kMost = 2147483647;
static std::string of(const char* name, std::initializer_list<long long> v) {
  std::string s = name;
  for (long long x : v) s += " " + std::to_string(x);
  return s;
}

// Tiles of a group of any number of rows: none is lost, none too many.
static void tiles() {
  for (int bm : {32, 64, 128, 256})
    for (long long rows : {0LL, 1LL, bm - 1LL, (long long)bm, bm + 1LL, kMost - 256LL, kMost - 255LL, kMost - 63LL,
                           kMost - 1LL, (long long)kMost}) {
      const int got = moe::group_tiles<moe::GR_FWD>(moe::GroupDims{kMost, 1, 16, 16}, (int)rows, bm);
      if (got != (rows + bm - 1) / bm) {
        printf("%lld rows in tiles of %d: %d\n", rows, bm, got);
        ++failures;
      }
      const int w = moe::group_tiles<moe::GR_DW>(moe::GroupDims{kMost, 1, 1 << 20, 16}, (int)rows, bm);
      if (w != (rows > 0 ? (1 << 20) / bm : 0)) ++failures;
    }
}

static void balance() {
  for (int T : {1, 64, 65, 1 << 29, kMost - 64, kMost - 63, kMost - 1, kMost})
    for (int S : {1, 1024}) {
      size_t bytes = 0;
      took(moe_balance_loss_workspace_size(T, 3, S, &bytes), of("balance loss size", {T, S}));
      const size_t chunks = ((size_t)T + 63) / 64 + S;
      if (bytes < chunks * 40 || bytes > chunks * 40 + 256) {
        printf("balance loss %d %d: %zu bytes for %zu chunks\n", T, S, bytes, chunks);
        ++failures;
      }
    }
  for (int T : {1, 64, 1 << 20, 1 << 26, (1 << 29) - 64, 1 << 29, kMost - 63, kMost})
    for (int S : {1, 1024}) {
      RUN(of("balance loss", {T, S}), moe_balance_loss(fl(0), in(1), in(2), 0, 0, T, 3, 1, S, 0, 1.f, 1.f, in(3), fl(4),
                                                       fl(5), fl(6), at(7), kRoom, 0));
      RUN(of("its gradient", {T, S}),
          moe_balance_loss_backward(fl(0), fl(6), 0, in(2), 0, T, 3, S, fl(8), 0));
    }
}

static void products() {
  const int Q = MOE_DTYPE_E4M3, R = MOE_DTYPE_E5M2, F = MOE_DTYPE_F32, B = MOE_DTYPE_BF16;
  struct Shape {
    int M, E, n, k;
    size_t copy;  // bytes of the operands' copies: w's rows, for y
  };
  const Shape shapes[] = {{1, 1, 1, 1, 256 + 256}, {1, 1, 2048, 2048, 0}, {1021, 16, 136, 267, 0},
                          {20000, 1, 8, 8, 20000 * 16 + 256}, {49152, 64, 1408, 2048, 0},
                          {9000, 2, 1100, 267, 9000 * 272 + 2 * 1100 * 272}, {kMost, 1, 16, 16, 0},
                          {kMost, 1024, 16, 16, 0}, {kMost, 1, 17, 17, 0}, {1 << 20, 1024, 64, 48, 0},
                          {3, 1, 1 << 20, 1 << 20, 0}, {64, 1024, 1 << 20, 1, 0}};
  for (const Shape& s : shapes)
    for (int dx : {0, 1})
      for (int x : {Q, R})
        for (int out : {F, B}) {
          const std::string name = of(dx ? "8-bit dx" : "8-bit y", {s.M, s.E, s.n, s.k});
          size_t bytes = 0;
          took(dx ? moe_grouped_matmul_quantized_dx_workspace_size(s.M, s.E, s.n, s.k, &bytes)
                  : moe_grouped_matmul_quantized_workspace_size(s.M, s.E, s.n, s.k, &bytes), name);
          // none for whole 16 bytes; else up to both operands' rows of whole 16 bytes
          const int into = dx ? s.n : s.k;
          const size_t most = (into % 16 ? (size_t)s.M * ((into + 15) / 16 * 16) + 255 : 0) +
                              (s.k % 16 ? (size_t)s.E * s.n * ((s.k + 15) / 16 * 16) + 255 : 0);
          if (bytes > most || (!dx && s.copy != 0 && bytes < s.copy - 512)) {
            printf("%s: workspace of %zu bytes\n", name.c_str(), bytes);
            ++failures;
          }
          if (bytes > kRoom) continue;
          RUN(name, dx ? moe_grouped_matmul_quantized_dx(at(0), fl(1), at(2), fl(3), in(4), s.M, s.E, s.n, s.k, x, out, 1,
                                                         at(5), at(6), kRoom, 0)
                       : moe_grouped_matmul_quantized(at(0), fl(1), at(2), fl(3), in(4), s.M, s.E, s.n, s.k, x, out, 1,
                                                      at(5), at(6), kRoom, 0));
        }
  for (const Shape& s : shapes)
    for (int dt : {F, B}) {
      const std::string name = of("grouped", {s.M, s.E, s.n, s.k, dt});
      size_t bytes = 0;
      took(moe_grouped_matmul_workspace_size(s.M, s.E, s.n, s.k, dt, &bytes), name);
      if (bytes > kRoom || (size_t)s.E * s.n * s.k * 4 > kRoom) continue;
      RUN(name, moe_grouped_matmul(at(0), at(1), in(2), s.M, s.E, s.n, s.k, dt, 1, at(3), at(4), kRoom, 0));
      took(moe_grouped_matmul_backward_workspace_size(s.M, s.E, s.n, s.k, dt, 1, 1, &bytes), name);
      if (bytes > kRoom) continue;
      RUN(name + " gradients", moe_grouped_matmul_backward(at(0), at(1), in(2), at(3), s.M, s.E, s.n, s.k, dt, 1, at(4),
                                                           fl(5), at(6), kRoom, 0));
    }
}

static void rows() {
  const int F = MOE_DTYPE_F32, B = MOE_DTYPE_BF16;
  struct Shape {
    int T, d;
  };
  for (const Shape& s : {Shape{1, 1}, {1, 1 << 24}, {4096, 8192}, {3001, 1283}, {70000, 20000}, {kMost, 1}, {kMost, 8},
                         {kMost, 128}, {1 << 20, 1 << 17}, {(1 << 24) + 5, 2049}})
    for (int dt : {F, B}) {
      for (int q : {dt, (int)MOE_DTYPE_E4M3, (int)MOE_DTYPE_E5M2})
        RUN(of("RMS norm", {s.T, s.d, dt, q}), moe_rms_norm(at(0), at(1), at(2), s.T, s.d, 0.f, dt, q, at(3), at(4),
                                                            q == dt ? nullptr : fl(5), fl(6), 0));
      RUN(of("RMS norm gradients", {s.T, s.d, dt}),
          moe_rms_norm_backward(at(0), at(1), at(2), fl(3), at(4), s.T, s.d, dt, at(5), fl(6), at(7), kRoom, 0));
      RUN(of("layer norm", {s.T, s.d, dt}), moe_layer_norm(at(0), at(1), at(2), s.T, s.d, 0.f, dt, at(3), fl(4), fl(5), 0));
      RUN(of("layer norm gradients", {s.T, s.d, dt}),
          moe_layer_norm_backward(at(0), at(1), at(2), fl(3), fl(4), s.T, s.d, dt, at(5), fl(6), fl(7), at(8), kRoom, 0));
      for (int q : {MOE_DTYPE_E4M3, MOE_DTYPE_E5M2}) {
        RUN(of("quantise", {s.T, s.d, dt}), moe_quantize_rows(at(0), s.T, s.d, dt, q, at(1), fl(2), 0));
        RUN(of("read back", {s.T, s.d, dt}), moe_dequantize_rows(at(0), fl(1), s.T, s.d, q, dt, at(2), 0));
      }
    }
  for (int T : {0, 1, 64 * 1024, 64 * 1024 + 1, kMost - 1023, kMost - 1, kMost})
    for (int d : {1, 16384, 16385, 1 << 24})
      for (int dt : {F, B}) {
        size_t r = 0, l = 0;
        took(moe_rms_norm_backward_workspace_size(T, d, dt, &r), of("RMS norm size", {T, d, dt}));
        took(moe_layer_norm_backward_workspace_size(T, d, dt, &l), of("layer norm size", {T, d, dt}));
        // partial rows of d (2 d) floats: none without rows, at most 1024
        const size_t row = (size_t)d * 4;
        if ((r == 0) != (T == 0) || r % row != 0 || r > 1024 * row || (l == 0) != (T == 0) || l % (2 * row) != 0 ||
            l > 1024 * 2 * row) {
          printf("partial rows of %d x %d: %zu and %zu bytes\n", T, d, r, l);
          ++failures;
        }
      }
  for (int q : {MOE_DTYPE_E4M3, MOE_DTYPE_E5M2})
    for (int dt : {F, B}) {
      RUN("quantise matrices", moe_quantize_blocks(at(0), 1 << 23, 1, 1, dt, q, at(1), fl(2), 0));
      RUN("quantise matrices", moe_quantize_blocks(at(0), 1, 1 << 20, 1 << 17, dt, q, at(1), fl(2), 0));
      RUN("quantise matrices", moe_quantize_blocks(at(0), 64, 1408, 2047, dt, q, at(1), fl(2), 0));
    }
}

int main(int argc, char** argv) {
  for (int i = 1; i < argc; ++i) {
    if (!strcmp(argv[i], "tiles")) tiles();
    if (!strcmp(argv[i], "balance")) balance();
    if (!strcmp(argv[i], "products")) products();
    if (!strcmp(argv[i], "rows")) rows();
  }
  if (failures == 0) printf("ALL OK\n");
  return failures != 0;
}
