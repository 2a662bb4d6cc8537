// The layer operators' C ABI (mx_layer_api.cpp) on the host alone: launcher
// stubs record their calls, and every check here ends before or at a stub.
// Run under AddressSanitizer and UndefinedBehaviorSanitizer, and under
// ThreadSanitizer with several threads at once.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <thread>
#include <vector>

#include "mx_internal.h"
#include "mx_layer.h"

static thread_local int g_calls = 0;
static thread_local bool g_fail = false;
static hipError_t hit() {
  g_calls++;
  return g_fail ? hipErrorInvalidValue : hipSuccess;
}
extern "C" const char *hipGetErrorString(hipError_t) { return "stubbed launch failure"; }

mx_status_t mxi_record_hip_error(hipError_t) { return MX_ERR_HIP; }
hipError_t mxi_launch_rmsnorm(const void *, const void *, const void *, int, int64_t, int64_t, float,
                              int, uint8_t *, uint8_t *, void *, hipStream_t) { return hit(); }
int64_t mxi_rmsnorm_partials(int64_t rows, int64_t) { return rows < 64 ? rows : 64; }
hipError_t mxi_launch_rmsnorm_backward(const void *, const void *, const void *, const void *, int,
                                       int64_t, int64_t, float, void *, float *, float *,
                                       hipStream_t) { return hit(); }
hipError_t mxi_launch_quantize8_blocks(const void *, int, int64_t, int64_t, int, uint8_t *,
                                       uint8_t *, uint8_t *, uint8_t *, hipStream_t) { return hit(); }
size_t mxi_matmul8_workspace(int64_t m, int64_t n, int64_t k, int, int) {
  return k > 4096 ? (size_t)(m * n * 8) : 0;
}
hipError_t mxi_launch_matmul8(const uint8_t *, const uint8_t *, const uint8_t *, const uint8_t *,
                              int64_t, int64_t, int64_t, int, int, void *, void *,
                              hipStream_t) { return hit(); }
hipError_t mxi_launch_kv_append(const void *, const void *, int, int64_t, int64_t,
                                const mx_kv_cache_t &, const mx_kv_batch_t &, hipStream_t) {
  return hit();
}
size_t mxi_kv_attention_workspace(int64_t tokens, int, int, int, int, int64_t max_length) {
  return max_length > 512 ? (size_t)tokens * 64 : 0;
}
hipError_t mxi_launch_kv_attention(const void *, int64_t, int, const mx_kv_cache_t &,
                                   const mx_kv_batch_t &, int64_t, float, void *, void *,
                                   hipStream_t) { return hit(); }

#define CHECK(x)                                                    \
  do {                                                              \
    if (!(x)) {                                                     \
      printf("%s:%d: %s\n", __FILE__, __LINE__, #x);                \
      exit(1);                                                      \
    }                                                               \
  } while (0)

template <typename T>
static T *at(uint64_t a) {
  return reinterpret_cast<T *>(static_cast<uintptr_t>(a) << 32);
}

static void run() {
  auto X = at<uint8_t>(1), C = at<uint8_t>(2), S = at<uint8_t>(3), W = at<uint8_t>(4);
  auto H = at<uint8_t>(5), R = at<uint8_t>(6), CT = at<uint8_t>(7), ST = at<uint8_t>(8);
  const mx_dtype_t bf = MX_BF16;

  // quantizer
  int calls = g_calls;
  CHECK(mx_quantize_mxfp8_blocks(X, (mx_dtype_t)3, 4, 64, 32, C, S, CT, ST, nullptr) == MX_ERR_DTYPE);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, 4, 64, 64, C, S, CT, ST, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, 4, 48, 32, C, S, CT, ST, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, -1, 64, 32, C, S, CT, ST, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, (int64_t)1 << 32, 64, 32, C, S, CT, ST, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, 1, (int64_t)1 << 40, 32, C, S, CT, ST, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, 4, 64, 32, nullptr, nullptr, nullptr, nullptr, nullptr) == MX_ERR_NULL);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, 4, 64, 32, C, nullptr, CT, ST, nullptr) == MX_ERR_NULL);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, 4, 64, 32, C, S, nullptr, ST, nullptr) == MX_ERR_NULL);
  CHECK(mx_quantize_mxfp8_blocks(X + 4, bf, 4, 64, 32, C, S, CT, ST, nullptr) == MX_ERR_ALIGN);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, 4, 64, 32, C, S, CT, ST + 8, nullptr) == MX_ERR_ALIGN);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, 4, 64, 32, X + 16, S, CT, ST, nullptr) == MX_ERR_ALIAS);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, 4, 64, 32, C, S, C + 16, ST, nullptr) == MX_ERR_ALIAS);
  // padded columns: 64 x 32 bytes, although there are only 4 rows
  CHECK(mx_quantize_mxfp8_blocks(X, bf, 4, 64, 32, C, CT + 2032, CT, ST, nullptr) == MX_ERR_ALIAS);
  CHECK(g_calls == calls);
  CHECK(mx_quantize_mxfp8_blocks(nullptr, bf, 0, 64, 32, nullptr, nullptr, nullptr, nullptr, nullptr) == MX_OK);
  CHECK(g_calls == calls);
  CHECK(mx_quantize_mxfp8_blocks(X, bf, 4, 64, 32, C, S, nullptr, nullptr, nullptr) == MX_OK);
  CHECK(g_calls == calls + 1);

  // norm
  calls = g_calls;
  CHECK(mx_rmsnorm_mxfp8(X, R, W, (mx_dtype_t)9, 4, 64, 1e-5f, 32, C, S, H, nullptr) == MX_ERR_DTYPE);
  CHECK(mx_rmsnorm_mxfp8(X, R, W, bf, 4, 65568, 1e-5f, 32, C, S, H, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_rmsnorm_mxfp8(X, R, W, bf, 4, 40, 1e-5f, 32, C, S, H, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_rmsnorm_mxfp8(X, R, W, bf, 4, 64, -1.0f, 32, C, S, H, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_rmsnorm_mxfp8(X, R, W, bf, 4, 64, NAN, 32, C, S, H, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_rmsnorm_mxfp8(X, R, W, bf, 4, 64, 1e-5f, 16, C, S, H, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_rmsnorm_mxfp8(X, nullptr, W, bf, 4, 64, 1e-5f, 32, C, S, H, nullptr) == MX_ERR_NULL);
  CHECK(mx_rmsnorm_mxfp8(X, R, nullptr, bf, 4, 64, 1e-5f, 32, C, S, H, nullptr) == MX_ERR_NULL);
  CHECK(mx_rmsnorm_mxfp8(X, R + 8, W, bf, 4, 64, 1e-5f, 32, C, S, H, nullptr) == MX_ERR_ALIGN);
  CHECK(mx_rmsnorm_mxfp8(X, R, W, bf, 4, 64, 1e-5f, 32, C, S, X + 16, nullptr) == MX_ERR_ALIAS);
  CHECK(mx_rmsnorm_mxfp8(X, R, W, bf, 4, 64, 1e-5f, 32, X, S, H, nullptr) == MX_ERR_ALIAS);
  CHECK(mx_rmsnorm_mxfp8(X, R, W, bf, 4, 64, 1e-5f, 32, C, S, W, nullptr) == MX_ERR_ALIAS);
  CHECK(g_calls == calls);
  CHECK(mx_rmsnorm_mxfp8(X, R, W, bf, 4, 64, 1e-5f, 32, C, S, X, nullptr) == MX_OK);
  CHECK(mx_rmsnorm_mxfp8(X, R, W, bf, 4, 64, 0.0f, 128, C, S, R, nullptr) == MX_OK);
  CHECK(mx_rmsnorm_mxfp8(nullptr, nullptr, nullptr, bf, 0, 64, 0.0f, 128, nullptr, nullptr, nullptr, nullptr) == MX_OK);
  CHECK(g_calls == calls + 2);

  // its gradient
  const size_t ws = mx_rmsnorm_backward_workspace_size(4, 64);
  CHECK(ws == 4 * 64 * 4 && mx_rmsnorm_backward_workspace_size(4, 63) == 0);
  float *dw = reinterpret_cast<float *>(ST);
  calls = g_calls;
  CHECK(mx_rmsnorm_backward(X, H, W, R, bf, 4, 64, 1e-5f, C, dw, CT, ws - 1, nullptr) == MX_ERR_WORKSPACE);
  CHECK(mx_rmsnorm_backward(X, H, W, R, bf, 4, 64, 1e-5f, C, dw, nullptr, ws, nullptr) == MX_ERR_WORKSPACE);
  CHECK(mx_rmsnorm_backward(X, H, W, R, bf, 4, 64, 1e-5f, C, dw, CT + 4, ws, nullptr) == MX_ERR_WORKSPACE);
  CHECK(mx_rmsnorm_backward(X, H, W, R, bf, 4, 64, 1e-5f, nullptr, dw, CT, ws, nullptr) == MX_ERR_NULL);
  CHECK(mx_rmsnorm_backward(X, H, W, R, bf, 4, 64, 1e-5f, C, nullptr, CT, ws, nullptr) == MX_ERR_NULL);
  CHECK(mx_rmsnorm_backward(X, H, W, R, bf, 4, 64, 1e-5f, X + 32, dw, CT, ws, nullptr) == MX_ERR_ALIAS);
  CHECK(mx_rmsnorm_backward(X, H, W, R, bf, 4, 64, 1e-5f, W, dw, CT, ws, nullptr) == MX_ERR_ALIAS);
  CHECK(mx_rmsnorm_backward(X, H, W, R, bf, 4, 64, 1e-5f, C, dw, C, ws, nullptr) == MX_ERR_ALIAS);
  CHECK(mx_rmsnorm_backward(X, H, W, R, bf, 4, 64, 1e-5f, C, dw, dw, ws, nullptr) == MX_ERR_ALIAS);
  CHECK(g_calls == calls);
  for (uint8_t *o : {X, H, R, C})
    CHECK(mx_rmsnorm_backward(X, H, W, R, bf, 4, 64, 1e-5f, o, dw, CT, ws, nullptr) == MX_OK);
  CHECK(mx_rmsnorm_backward(nullptr, nullptr, nullptr, nullptr, bf, 0, 64, 0, nullptr, dw, nullptr, 0, nullptr) == MX_OK);
  CHECK(g_calls == calls + 5);

  // product
  calls = g_calls;
  CHECK(mx_matmul_mxfp8(X, S, C, ST, 4, 4, 64, 32, (mx_dtype_t)7, H, nullptr, 0, nullptr) == MX_ERR_DTYPE);
  CHECK(mx_matmul_mxfp8(X, S, C, ST, 4, 4, 0, 32, bf, H, nullptr, 0, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_matmul_mxfp8(X, S, C, ST, 4, 4, 48, 32, bf, H, nullptr, 0, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_matmul_mxfp8(X, S, C, ST, 4, 4, 64, 256, bf, H, nullptr, 0, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_matmul_mxfp8(X, S, C, ST, 4, 4, (1 << 20) + 32, 32, bf, H, nullptr, 0, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_matmul_mxfp8(X, S, C, ST, -4, 4, 64, 32, bf, H, nullptr, 0, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_matmul_mxfp8(X, S, C, ST, INT32_MAX, INT32_MAX, 64, 32, bf, H, nullptr, 0, nullptr) == MX_ERR_SHAPE);
  CHECK(mx_matmul_mxfp8(X, nullptr, C, ST, 4, 4, 64, 32, bf, H, nullptr, 0, nullptr) == MX_ERR_NULL);
  CHECK(mx_matmul_mxfp8(X, S + 4, C, ST, 4, 4, 64, 32, bf, H, nullptr, 0, nullptr) == MX_ERR_ALIGN);
  CHECK(mx_matmul_mxfp8(X, S, C, ST, 4, 4, 64, 32, bf, C + 16, nullptr, 0, nullptr) == MX_ERR_ALIAS);
  CHECK(mx_matmul_mxfp8(X, S, C, ST, 4, 4, 8192, 32, bf, H, nullptr, 0, nullptr) == MX_ERR_WORKSPACE);
  CHECK(mx_matmul_mxfp8(X, S, C, ST, 4, 4, 8192, 32, bf, H, X, 128, nullptr) == MX_ERR_ALIAS);
  CHECK(g_calls == calls);
  CHECK(mx_matmul_mxfp8(X, S, X, S, 4, 4, 64, 32, bf, H, nullptr, 0, nullptr) == MX_OK);
  CHECK(mx_matmul_mxfp8(X, S, C, ST, 4, 4, 8192, 32, MX_F32, H, CT, 128, nullptr) == MX_OK);
  CHECK(mx_matmul_mxfp8(nullptr, nullptr, nullptr, nullptr, 0, 4, 64, 32, bf, nullptr, nullptr, 0, nullptr) == MX_OK);
  CHECK(g_calls == calls + 2);
  CHECK(mx_matmul_mxfp8_workspace_size(4, 4, 8192, 32, bf) == 128);
  CHECK(mx_matmul_mxfp8_workspace_size(4, 4, 8200, 32, bf) == 0);

  // cache
  auto I = at<int32_t>(9);
  const mx_kv_cache_t good = {C, S, CT, ST, 10, 2, 64, 32};
  const mx_kv_batch_t batch = {I, I + 64, I + 128, 5, 3, 4};
  calls = g_calls;
  auto app = [&](const mx_kv_cache_t *c, const mx_kv_batch_t *b, int64_t ks = 128, int64_t vs = 128) {
    return mx_kv_append(X, H, bf, ks, vs, c, b, nullptr);
  };
  auto att = [&](const mx_kv_cache_t *c, const mx_kv_batch_t *b, int qh = 4, float sc = 0.1f,
                 int64_t longest = 0, int64_t qs = 1024, void *w = nullptr, size_t n = 0) {
    return mx_kv_attention(X, qs, qh, c, b, longest, sc, H, w, n, nullptr);
  };
  CHECK(app(nullptr, &batch) == MX_ERR_NULL && app(&good, nullptr) == MX_ERR_NULL);
  for (int what = 0; what < 8; what++) {
    mx_kv_cache_t c = good;
    if (what == 0) c.dim = 96;
    if (what == 1) c.page = 48;
    if (what == 2) c.page = 16;
    if (what == 3) c.page = 512;
    if (what == 4) c.heads = 0;
    if (what == 5) c.pages = 0;
    if (what == 6) c.pages = (int64_t)1 << 32;
    if (what == 7) c.heads = 70000;
    CHECK(app(&c, &batch) == MX_ERR_SHAPE && att(&c, &batch) == MX_ERR_SHAPE);
  }
  for (int what = 0; what < 5; what++) {
    mx_kv_batch_t b = batch;
    if (what == 0) b.batch = 0;
    if (what == 1) b.width = 0;
    if (what == 2) b.tokens = -1;
    if (what == 3) b.tokens = INT32_MAX;
    if (what == 4) b.width = 1 << 27;
    CHECK(app(&good, &b) == MX_ERR_SHAPE && att(&good, &b) == MX_ERR_SHAPE);
  }
  for (int what = 0; what < 3; what++) {
    mx_kv_cache_t c = good;
    mx_kv_batch_t b = batch;
    if (what == 0) c.v_scales = nullptr;
    if (what == 1) b.cu = nullptr;
    if (what == 2) b.table = nullptr;
    CHECK(app(&c, &b) == MX_ERR_NULL && att(&c, &b) == MX_ERR_NULL);
  }
  CHECK(app(&good, &batch, 127) == MX_ERR_SHAPE && app(&good, &batch, 132) == MX_ERR_ALIGN);
  CHECK(app(&good, &batch, 128, 120) == MX_ERR_SHAPE);
  CHECK(mx_kv_append(X, H, (mx_dtype_t)4, 128, 128, &good, &batch, nullptr) == MX_ERR_DTYPE);
  CHECK(mx_kv_append(X, C, bf, 128, 128, &good, &batch, nullptr) == MX_ERR_ALIAS);
  CHECK(att(&good, &batch, 3) == MX_ERR_SHAPE && att(&good, &batch, 0) == MX_ERR_SHAPE);
  CHECK(att(&good, &batch, 512) == MX_ERR_SHAPE);
  CHECK(att(&good, &batch, 4, 0.0f) == MX_ERR_SHAPE && att(&good, &batch, 4, -1.0f) == MX_ERR_SHAPE);
  CHECK(att(&good, &batch, 4, NAN) == MX_ERR_SHAPE && att(&good, &batch, 4, INFINITY) == MX_ERR_SHAPE);
  CHECK(att(&good, &batch, 4, 0.1f, -1) == MX_ERR_SHAPE);
  CHECK(att(&good, &batch, 4, 0.1f, 0, 200) == MX_ERR_SHAPE);
  CHECK(att(&good, &batch, 4, 0.1f, 0, 260) == MX_ERR_ALIGN);
  CHECK(mx_kv_attention(X, 1024, 4, &good, &batch, 0, 0.1f, X, nullptr, 0, nullptr) == MX_ERR_ALIAS);
  {
    mx_kv_batch_t b = batch;
    b.width = 100;  // room for 3200 tokens: the stub asks for a workspace
    CHECK(att(&good, &b) == MX_ERR_WORKSPACE);
    CHECK(att(&good, &b, 4, 0.1f, 0, 1024, R + 8, 1 << 20) == MX_ERR_WORKSPACE);
    CHECK(att(&good, &b, 4, 0.1f, 0, 1024, C, 1 << 20) == MX_ERR_ALIAS);
  }
  CHECK(g_calls == calls);
  CHECK(app(&good, &batch) == MX_OK && att(&good, &batch) == MX_OK);
  mx_kv_batch_t none = batch;
  none.tokens = 0;
  CHECK(app(&good, &none) == MX_OK && att(&good, &none) == MX_OK);
  CHECK(g_calls == calls + 2);
  CHECK(mx_kv_attention_workspace_size(5, 3, 4, 2, 64, 3200) == 320);
  CHECK(mx_kv_attention_workspace_size(5, 3, 5, 2, 64, 3200) == 0);

  g_fail = true;
  CHECK(app(&good, &batch) == MX_ERR_HIP && att(&good, &batch) == MX_ERR_HIP);
  g_fail = false;
}

int main() {
  run();
  std::vector<std::thread> ts;
  for (int i = 0; i < 8; i++) ts.emplace_back([] { for (int j = 0; j < 50; j++) run(); });
  for (auto &t : ts) t.join();
  printf("layer ABI checks passed\n");
  return 0;
}
