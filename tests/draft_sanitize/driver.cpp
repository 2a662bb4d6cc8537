// The C ABI of positions and drafted tokens (mx_draft_api.cpp) on the host alone:
// launcher stubs record their calls, and every check here ends before or at a
// stub. Run under AddressSanitizer and UndefinedBehaviorSanitizer, and under
// ThreadSanitizer with several threads at once.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

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

mx_status_t mxi_record_hip_error(hipError_t) { return MX_ERR_HIP; }
hipError_t mxi_launch_norm_rotate(const mx_heads_t &, const mx_heads_t *, int, int64_t, int, float,
                                  const mx_rotary_t &, hipStream_t) { return hit(); }
int64_t mxi_norm_rotate_partials(int64_t tokens) { return 2 * (tokens < 64 ? tokens : 64); }
hipError_t mxi_launch_norm_rotate_backward(const mx_heads_grad_t &, const mx_heads_grad_t *, int,
                                           int64_t, int, float, const mx_rotary_t &, float *,
                                           hipStream_t) { return hit(); }
hipError_t mxi_launch_kv_append_rotary(const void *, const void *, int, int64_t, int64_t, const void *,
                                       float, const mx_rotary_t &, const mx_kv_cache_t &,
                                       const mx_kv_batch_t &, hipStream_t) { return hit(); }
size_t mxi_kv_attention_tree_workspace(int64_t tokens, int, int, int, int, int64_t max_length) {
  return max_length > 512 ? (size_t)tokens * 64 : 0;
}
hipError_t mxi_launch_kv_attention_tree(const void *, int64_t, int, const mx_kv_cache_t &,
                                        const mx_kv_batch_t &, const uint32_t *, int, int64_t, float,
                                        void *, void *, hipStream_t) { return hit(); }
size_t mxi_verify_workspace(int64_t tokens, int, int64_t) { return (size_t)tokens * 64; }
hipError_t mxi_launch_verify(const void *, const void *, int, const int32_t *, const int32_t *,
                             const int32_t *, const float *, int64_t, int, int64_t, int, int32_t *,
                             int32_t *, int32_t *, void *, hipStream_t) { return hit(); }
hipError_t mxi_launch_kv_keep(const mx_kv_cache_t &, const mx_kv_batch_t &, const int32_t *, int,
                              const int32_t *, hipStream_t) { return hit(); }

#define CHECK(x)                                                    \
  do {                                                              \
    if (!(x)) {                                                     \
      printf("%s:%d: %s\n", __FILE__, __LINE__, #x);                \
      exit(1);                                                      \
    }                                                               \
  } while (0)

template <typename T>
static T *at(uint64_t a) {
  return reinterpret_cast<T *>(static_cast<uintptr_t>(a) << 36);
}
template <typename T, typename F>
static T with(T x, F f) {
  f(x);
  return x;
}

static void rotate() {
  const mx_dtype_t bf = MX_BF16;
  const mx_rotary_t r = {at<float>(1), at<int32_t>(2), 100, 64, 0};
  const mx_heads_t q = {at<uint8_t>(3), 4 * 64, at<uint8_t>(4), at<uint8_t>(5), 4 * 64, 4};
  const mx_heads_t k = {at<uint8_t>(6), 2 * 64, at<uint8_t>(7), at<uint8_t>(8), 2 * 64, 2};
  auto call = [&](mx_heads_t a, mx_heads_t b, mx_rotary_t t, int64_t tokens = 10, int dim = 64,
                  float eps = 0.0f, int dtype = MX_BF16) {
    return mx_norm_rotate(&a, &b, (mx_dtype_t)dtype, tokens, dim, eps, &t, nullptr);
  };
  int calls = g_calls;
  CHECK(mx_norm_rotate(nullptr, &k, bf, 10, 64, 0, &r, nullptr) == MX_ERR_NULL);
  CHECK(call(q, k, r, 10, 64, 0, 2) == MX_ERR_DTYPE);
  CHECK(call(q, k, r, -1) == MX_ERR_SHAPE);
  CHECK(call(q, k, r, (int64_t)1 << 31) == MX_ERR_SHAPE);
  for (int dim : {0, 32, 96, 512, -64}) CHECK(call(q, k, r, 10, dim) == MX_ERR_SHAPE);
  CHECK(call(q, k, r, 10, 64, -1.0f) == MX_ERR_SHAPE);
  CHECK(call(q, k, r, 10, 64, NAN) == MX_ERR_SHAPE);
  CHECK(call(q, k, r, 10, 64, INFINITY) == MX_ERR_SHAPE);
  for (int heads : {0, -1, 65536}) {
    CHECK(call(with(q, [&](auto &h) { h.heads = heads; }), k, r) == MX_ERR_SHAPE);
    CHECK(call(q, with(k, [&](auto &h) { h.heads = heads; }), r) == MX_ERR_SHAPE);
  }
  for (int rot : {-16, 8, 24, 80}) CHECK(call(q, k, with(r, [&](auto &t) { t.rot = rot; })) == MX_ERR_SHAPE);
  CHECK(call(q, k, with(r, [](auto &t) { t.length = 0; })) == MX_ERR_SHAPE);
  CHECK(call(q, k, with(r, [](auto &t) { t.length = INT64_MAX; })) == MX_ERR_SHAPE);
  CHECK(call(with(q, [](auto &h) { h.x_stride = 255; }), k, r) == MX_ERR_SHAPE);
  CHECK(call(with(q, [](auto &h) { h.y_stride = (int64_t)1 << 31; }), k, r) == MX_ERR_SHAPE);
  CHECK(call(q, with(k, [](auto &h) { h.x_stride = INT32_MAX; }), r, INT32_MAX) == MX_ERR_SHAPE);
  CHECK(call(with(q, [](auto &h) { h.x = nullptr; }), k, r) == MX_ERR_NULL);
  CHECK(call(q, with(k, [](auto &h) { h.y = nullptr; }), r) == MX_ERR_NULL);
  CHECK(call(q, k, with(r, [](auto &t) { t.table = nullptr; })) == MX_ERR_NULL);
  CHECK(call(q, k, with(r, [](auto &t) { t.positions = nullptr; })) == MX_ERR_NULL);
  CHECK(call(with(q, [](auto &h) { h.x = at<uint8_t>(3) + 8; }), k, r) == MX_ERR_ALIGN);
  CHECK(call(with(q, [](auto &h) { h.weight = at<uint8_t>(4) + 2; }), k, r) == MX_ERR_ALIGN);
  CHECK(call(with(q, [](auto &h) { h.x_stride = 260; }), k, r) == MX_ERR_ALIGN);
  CHECK(call(q, with(k, [](auto &h) { h.y_stride = 132; }), r) == MX_ERR_ALIGN);
  CHECK(call(q, k, with(r, [](auto &t) { t.table = at<float>(1) + 1; })) == MX_ERR_ALIGN);
  CHECK(call(q, k, with(r, [](auto &t) { t.positions = reinterpret_cast<int32_t *>(at<uint8_t>(2) + 2); })) == MX_ERR_ALIGN);
  // outputs on inputs, weights, the rotation, each other
  CHECK(call(with(q, [&](auto &h) { h.y = at<uint8_t>(3) + 512; }), k, r) == MX_ERR_ALIAS);
  CHECK(call(with(q, [&](auto &h) { h.y = at<uint8_t>(3); h.y_stride = 512; }), k, r) == MX_ERR_ALIAS);
  CHECK(call(with(q, [&](auto &h) { h.y = at<uint8_t>(6); }), k, r) == MX_ERR_ALIAS);
  CHECK(call(with(q, [&](auto &h) { h.y = at<uint8_t>(8); }), k, r) == MX_ERR_ALIAS);
  CHECK(call(with(q, [&](auto &h) { h.y = at<uint8_t>(4); }), k, r) == MX_ERR_ALIAS);
  CHECK(call(with(q, [&](auto &h) { h.y = at<uint8_t>(7); }), k, r) == MX_ERR_ALIAS);
  CHECK(call(with(q, [&](auto &h) { h.y = at<uint8_t>(1) + 16; }), k, r) == MX_ERR_ALIAS);
  CHECK(call(q, with(k, [&](auto &h) { h.y = at<uint8_t>(2) + 32; }), r) == MX_ERR_ALIAS);
  CHECK(g_calls == calls);
  CHECK(call(q, k, r, 0) == MX_OK && g_calls == calls);
  CHECK(call(q, k, r) == MX_OK && g_calls == ++calls);
  CHECK(mx_norm_rotate(&q, nullptr, bf, 10, 64, 0, nullptr, nullptr) == MX_OK && g_calls == ++calls);
  // without a rotation its pointers do not count
  CHECK(call(q, k, mx_rotary_t{nullptr, nullptr, 0, 0, 0}) == MX_OK && g_calls == ++calls);
  // in place, and both parts of one projection's rows in place
  CHECK(call(with(q, [&](auto &h) { h.y = const_cast<void *>(h.x); }), k, r) == MX_OK && g_calls == ++calls);
  uint8_t *rows = at<uint8_t>(9);
  mx_heads_t a = {rows, 8 * 64, nullptr, rows, 8 * 64, 4}, b = {rows + 512, 8 * 64, nullptr, rows + 512, 8 * 64, 2};
  CHECK(call(a, b, r) == MX_OK && g_calls == ++calls);
  b.y = rows + 384;  // k's output over q's last head
  CHECK(call(a, b, r) == MX_ERR_ALIAS);
  b.y = rows + 896;  // over the next row's begin
  CHECK(call(a, b, r) == MX_ERR_ALIAS);
  g_fail = true;
  CHECK(call(q, k, r) == MX_ERR_HIP);
  g_fail = false;
}

static void rotate_backward() {
  const mx_rotary_t r = {at<float>(1), at<int32_t>(2), 100, 64, 1};
  const mx_heads_grad_t q = {at<uint8_t>(3), 256, at<uint8_t>(4), 256, at<uint8_t>(5), at<uint8_t>(6), 256, at<float>(7), 4};
  const mx_heads_grad_t k = {at<uint8_t>(8), 128, at<uint8_t>(9), 128, at<uint8_t>(10), at<uint8_t>(11), 128, at<float>(12), 2};
  uint8_t *ws = at<uint8_t>(13);
  const size_t size = mx_norm_rotate_backward_workspace_size(10, 64);
  CHECK(size == 10 * 2 * 64 * 4);
  CHECK(mx_norm_rotate_backward_workspace_size(-1, 64) == 0 && mx_norm_rotate_backward_workspace_size(10, 96) == 0);
  auto call = [&](mx_heads_grad_t a, mx_heads_grad_t b, int64_t tokens = 10, void *w = at<uint8_t>(13), size_t n = 1 << 20,
                  int dim = 64, int dtype = MX_BF16) {
    return mx_norm_rotate_backward(&a, &b, (mx_dtype_t)dtype, tokens, dim, 0.0f, &r, w, n, nullptr);
  };
  int calls = g_calls;
  CHECK(mx_norm_rotate_backward(nullptr, &k, MX_BF16, 10, 64, 0, &r, ws, size, nullptr) == MX_ERR_NULL);
  CHECK(call(q, k, 10, ws, size, 64, 7) == MX_ERR_DTYPE);
  CHECK(call(q, k, 10, ws, size, 32) == MX_ERR_SHAPE);
  CHECK(call(with(q, [](auto &h) { h.heads = 0; }), k) == MX_ERR_SHAPE);
  CHECK(call(with(q, [](auto &h) { h.dy_stride = 100; }), k) == MX_ERR_SHAPE);
  CHECK(call(with(q, [](auto &h) { h.dx_stride = 100; }), k) == MX_ERR_SHAPE);
  CHECK(call(q, with(k, [](auto &h) { h.x_stride = 100; })) == MX_ERR_SHAPE);
  CHECK(call(with(q, [](auto &h) { h.dweight = nullptr; }), k) == MX_ERR_NULL);
  CHECK(call(with(q, [](auto &h) { h.dy = nullptr; }), k) == MX_ERR_NULL);
  CHECK(call(with(q, [](auto &h) { h.x = nullptr; }), k) == MX_ERR_NULL);
  CHECK(call(q, with(k, [](auto &h) { h.dx = nullptr; })) == MX_ERR_NULL);
  CHECK(call(with(q, [](auto &h) { h.dweight = at<float>(7) + 1; }), k) == MX_ERR_ALIGN);
  CHECK(call(with(q, [](auto &h) { h.dx = at<uint8_t>(6) + 4; }), k) == MX_ERR_ALIGN);
  CHECK(call(with(q, [](auto &h) { h.x_stride = 260; }), k) == MX_ERR_ALIGN);
  CHECK(call(q, k, 10, nullptr, 0) == MX_ERR_WORKSPACE);
  CHECK(call(q, k, 10, ws + 8, 1 << 20) == MX_ERR_WORKSPACE);
  CHECK(call(q, k, 10, ws, size - 1) == MX_ERR_WORKSPACE);
  CHECK(call(with(q, [](auto &h) { h.dweight = at<float>(12); }), k) == MX_ERR_ALIAS);
  CHECK(call(with(q, [](auto &h) { h.dweight = at<float>(8) + 16; }), k) == MX_ERR_ALIAS);
  CHECK(call(with(q, [](auto &h) { h.dx = at<uint8_t>(3) + 512; }), k) == MX_ERR_ALIAS);
  CHECK(call(with(q, [](auto &h) { h.dx = at<uint8_t>(9); }), k) == MX_ERR_ALIAS);
  CHECK(call(with(q, [](auto &h) { h.dx = at<uint8_t>(11); }), k) == MX_ERR_ALIAS);
  CHECK(call(with(q, [](auto &h) { h.dx = at<uint8_t>(1); }), k) == MX_ERR_ALIAS);
  CHECK(call(q, k, 10, at<uint8_t>(4)) == MX_ERR_ALIAS);
  CHECK(call(q, k, 10, at<uint8_t>(12)) == MX_ERR_ALIAS);
  CHECK(call(q, k, 10, at<uint8_t>(2)) == MX_ERR_ALIAS);
  CHECK(g_calls == calls);
  CHECK(call(q, k) == MX_OK && g_calls == ++calls);
  CHECK(call(q, k, 0, nullptr, 0) == MX_OK && g_calls == ++calls);  // zeros to the dweights
  CHECK(call(with(q, [](auto &h) { h.dx = const_cast<void *>(h.dy); }), k) == MX_OK && g_calls == ++calls);
  CHECK(call(with(q, [](auto &h) { h.dx = const_cast<void *>(h.x); }), k) == MX_OK && g_calls == ++calls);
  // without weights neither x nor scratch is wanted
  auto bare = [](auto &h) { h.weight = nullptr; h.x = nullptr; h.dweight = nullptr; h.x_stride = 0; };
  CHECK(call(with(q, bare), with(k, bare), 10, nullptr, 0) == MX_OK && g_calls == ++calls);
}

static void cache_calls() {
  const mx_kv_cache_t c = {at<uint8_t>(1), at<uint8_t>(2), at<uint8_t>(3), at<uint8_t>(4), 10, 2, 64, 32};
  const mx_kv_batch_t b = {at<int32_t>(5), at<int32_t>(6), at<int32_t>(7), 8, 2, 4};
  const mx_rotary_t r = {at<float>(8), nullptr, 100, 64, 0};
  uint8_t *k = at<uint8_t>(9), *v = at<uint8_t>(10), *w = at<uint8_t>(11);
  auto append = [&](mx_kv_cache_t cc, mx_kv_batch_t bb, mx_rotary_t rr, const void *kk, int64_t stride = 128, float eps = 0.0f,
                    const void *weight = at<uint8_t>(11), int dtype = MX_BF16) {
    return mx_kv_append_rotary(kk, v, (mx_dtype_t)dtype, stride, 128, weight, eps, &rr, &cc, &bb, nullptr);
  };
  int calls = g_calls;
  CHECK(mx_kv_append_rotary(k, v, MX_BF16, 128, 128, w, 0, &r, nullptr, &b, nullptr) == MX_ERR_NULL);
  CHECK(mx_kv_append_rotary(k, v, MX_BF16, 128, 128, w, 0, &r, &c, nullptr, nullptr) == MX_ERR_NULL);
  CHECK(append(c, b, r, k, 128, 0, w, 9) == MX_ERR_DTYPE);
  CHECK(append(c, b, r, k, 127) == MX_ERR_SHAPE);
  CHECK(append(c, b, r, k, 128, -1.0f) == MX_ERR_SHAPE);
  CHECK(append(c, b, r, k, 128, INFINITY) == MX_ERR_SHAPE);
  CHECK(append(c, b, with(r, [](auto &t) { t.rot = 80; }), k) == MX_ERR_SHAPE);
  CHECK(append(c, b, with(r, [](auto &t) { t.length = 0; }), k) == MX_ERR_SHAPE);
  CHECK(append(with(c, [](auto &x) { x.dim = 256; }), b, r, k) == MX_ERR_SHAPE);
  CHECK(append(with(c, [](auto &x) { x.page = 48; }), b, r, k) == MX_ERR_SHAPE);
  CHECK(append(c, with(b, [](auto &x) { x.width = INT32_MAX; }), r, k) == MX_ERR_SHAPE);
  CHECK(append(c, b, r, nullptr) == MX_ERR_NULL);
  CHECK(append(c, b, with(r, [](auto &t) { t.table = nullptr; }), k) == MX_ERR_NULL);
  CHECK(append(c, with(b, [](auto &x) { x.lengths = nullptr; }), r, k) == MX_ERR_NULL);
  CHECK(append(c, b, r, k + 8) == MX_ERR_ALIGN);
  CHECK(append(c, b, r, k, 132) == MX_ERR_ALIGN);
  CHECK(append(c, b, r, k, 128, 0, w + 4) == MX_ERR_ALIGN);
  CHECK(append(c, b, with(r, [](auto &t) { t.positions = reinterpret_cast<int32_t *>(at<uint8_t>(12) + 1); }), k) == MX_ERR_ALIGN);
  CHECK(append(c, b, r, c.v_codes) == MX_ERR_ALIAS);
  CHECK(append(c, b, r, k, 128, 0, c.k_codes) == MX_ERR_ALIAS);
  CHECK(append(c, b, with(r, [&](auto &t) { t.table = reinterpret_cast<float *>(c.k_codes); }), k) == MX_ERR_ALIAS);
  CHECK(append(c, b, with(r, [&](auto &t) { t.positions = reinterpret_cast<int32_t *>(c.v_scales); }), k) == MX_ERR_ALIAS);
  CHECK(g_calls == calls);
  CHECK(append(c, with(b, [](auto &x) { x.tokens = 0; }), r, nullptr) == MX_OK && g_calls == calls);
  CHECK(append(c, b, r, k) == MX_OK && g_calls == ++calls);
  CHECK(mx_kv_append_rotary(k, v, MX_F32, 128, 128, nullptr, 0, nullptr, &c, &b, nullptr) == MX_OK && g_calls == ++calls);

  uint32_t *m = at<uint32_t>(13);
  uint8_t *q = at<uint8_t>(14), *out = at<uint8_t>(15), *ws = at<uint8_t>(16);
  auto attend = [&](mx_kv_cache_t cc, mx_kv_batch_t bb, const uint32_t *mask, int words = 1, int q_heads = 4, float scale = 1.0f,
                    const void *qq = at<uint8_t>(14), int64_t stride = 256, void *o = at<uint8_t>(15)) {
    return mx_kv_attention_tree(qq, stride, q_heads, &cc, &bb, mask, words, 128, scale, o, nullptr, 0, nullptr);
  };
  CHECK(mx_kv_attention_tree(q, 256, 4, nullptr, &b, m, 1, 128, 1, out, nullptr, 0, nullptr) == MX_ERR_NULL);
  CHECK(attend(c, b, nullptr) == MX_ERR_NULL);
  CHECK(attend(c, b, m, 0) == MX_ERR_SHAPE);
  CHECK(attend(c, b, m, 65536) == MX_ERR_SHAPE);
  CHECK(attend(c, b, m, 1, 3) == MX_ERR_SHAPE);
  CHECK(attend(c, b, m, 1, 4, 0.0f) == MX_ERR_SHAPE);
  CHECK(attend(c, b, m, 1, 4, INFINITY) == MX_ERR_SHAPE);
  CHECK(attend(c, b, m, 1, 4, 1, q, 255) == MX_ERR_SHAPE);
  CHECK(attend(c, b, m, 1, 4, 1, nullptr) == MX_ERR_NULL);
  CHECK(attend(c, b, m, 1, 4, 1, q + 2) == MX_ERR_ALIGN);
  CHECK(attend(c, b, m, 1, 4, 1, q, 260) == MX_ERR_ALIGN);
  CHECK(attend(c, b, reinterpret_cast<uint32_t *>(at<uint8_t>(13) + 2)) == MX_ERR_ALIGN);
  CHECK(attend(c, b, m, 1, 4, 1, q, 256, q) == MX_ERR_ALIAS);
  CHECK(attend(c, b, m, 1, 4, 1, q, 256, m) == MX_ERR_ALIAS);
  CHECK(mx_kv_attention_tree(q, 256, 4, &c, &(const mx_kv_batch_t &)with(b, [](auto &x) { x.width = 40; }), m, 1, 0, 1, out,
                             nullptr, 0, nullptr) == MX_ERR_WORKSPACE);
  CHECK(mx_kv_attention_tree(q, 256, 4, &c, &(const mx_kv_batch_t &)with(b, [](auto &x) { x.width = 40; }), m, 1, 0, 1, out,
                             ws + 8, 1 << 20, nullptr) == MX_ERR_WORKSPACE);
  CHECK(g_calls == calls);
  CHECK(attend(c, with(b, [](auto &x) { x.tokens = 0; }), nullptr) == MX_OK && g_calls == calls);
  CHECK(attend(c, b, m) == MX_OK && g_calls == ++calls);
  CHECK(mx_kv_attention_tree(q, 256, 4, &c, &(const mx_kv_batch_t &)with(b, [](auto &x) { x.width = 40; }), m, 65535, 0, 1, out,
                             ws, 1 << 20, nullptr) == MX_OK && g_calls == ++calls);

  int32_t *path = at<int32_t>(17), *count = at<int32_t>(18);
  auto keep = [&](mx_kv_cache_t cc, mx_kv_batch_t bb, const int32_t *p, int width = 5, const int32_t *n = at<int32_t>(18)) {
    return mx_kv_keep(&cc, &bb, p, width, n, nullptr);
  };
  const mx_kv_batch_t kb = {at<int32_t>(5), nullptr, at<int32_t>(7), -7, 2, 4};  // cu and tokens do not count
  CHECK(mx_kv_keep(nullptr, &kb, path, 5, count, nullptr) == MX_ERR_NULL);
  CHECK(mx_kv_keep(&c, nullptr, path, 5, count, nullptr) == MX_ERR_NULL);
  CHECK(keep(c, kb, nullptr) == MX_ERR_NULL);
  CHECK(keep(c, kb, path, 5, nullptr) == MX_ERR_NULL);
  CHECK(keep(c, kb, path, 0) == MX_ERR_SHAPE);
  CHECK(keep(c, kb, path, INT32_MAX) == MX_ERR_SHAPE);
  CHECK(keep(c, with(kb, [](auto &x) { x.batch = -1; }), path) == MX_ERR_SHAPE);
  CHECK(keep(c, with(kb, [](auto &x) { x.width = 0; }), path) == MX_ERR_SHAPE);
  CHECK(keep(c, with(kb, [](auto &x) { x.width = INT32_MAX; }), path) == MX_ERR_SHAPE);
  CHECK(keep(with(c, [](auto &x) { x.pages = 0; }), kb, path) == MX_ERR_SHAPE);
  CHECK(keep(c, with(kb, [](auto &x) { x.table = nullptr; }), path) == MX_ERR_NULL);
  CHECK(keep(with(c, [](auto &x) { x.k_codes = at<uint8_t>(1) + 4; }), kb, path) == MX_ERR_ALIGN);
  CHECK(keep(c, kb, reinterpret_cast<int32_t *>(at<uint8_t>(17) + 2)) == MX_ERR_ALIGN);
  CHECK(keep(c, kb, reinterpret_cast<int32_t *>(c.k_codes)) == MX_ERR_ALIAS);
  CHECK(g_calls == calls);
  CHECK(keep(c, with(kb, [](auto &x) { x.batch = 0; }), nullptr) == MX_OK && g_calls == calls);
  CHECK(keep(c, kb, path) == MX_OK && g_calls == ++calls);
}

static void verify() {
  uint8_t *t = at<uint8_t>(1), *d = at<uint8_t>(2), *ws = at<uint8_t>(3);
  int32_t *ids = at<int32_t>(4), *up = at<int32_t>(5), *cu = at<int32_t>(6);
  float *u = at<float>(7);
  int32_t *path = at<int32_t>(8), *count = at<int32_t>(9), *token = at<int32_t>(10);
  struct Call {
    const void *target, *draft;
    int dtype;
    const int32_t *ids, *up, *cu;
    const float *u;
    int64_t tokens;
    int batch;
    int64_t vocab;
    int width;
    int32_t *path, *count, *token;
    void *ws;
    size_t size;
  };
  const Call ok = {t, d, MX_F32, ids, up, cu, u, 10, 3, 1000, 4, path, count, token, ws, 1 << 20};
  auto call = [](const Call &c) {
    return mx_verify_drafts(c.target, c.draft, (mx_dtype_t)c.dtype, c.ids, c.up, c.cu, c.u, c.tokens, c.batch, c.vocab,
                            c.width, c.path, c.count, c.token, c.ws, c.size, nullptr);
  };
  auto bad = [&](auto f, mx_status_t want) { CHECK(call(with(ok, f)) == want); };
  int calls = g_calls;
  bad([](Call &c) { c.dtype = 5; }, MX_ERR_DTYPE);
  bad([](Call &c) { c.tokens = -1; }, MX_ERR_SHAPE);
  bad([](Call &c) { c.tokens = (int64_t)1 << 31; }, MX_ERR_SHAPE);
  bad([](Call &c) { c.batch = -1; }, MX_ERR_SHAPE);
  bad([](Call &c) { c.batch = 0; }, MX_ERR_SHAPE);
  bad([](Call &c) { c.batch = 65536; }, MX_ERR_SHAPE);
  bad([](Call &c) { c.vocab = 0; }, MX_ERR_SHAPE);
  bad([](Call &c) { c.vocab = (int64_t)1 << 31; }, MX_ERR_SHAPE);
  bad([](Call &c) { c.vocab = INT32_MAX; c.tokens = INT32_MAX; }, MX_ERR_SHAPE);
  bad([](Call &c) { c.vocab = INT32_MAX; c.batch = 65535; }, MX_ERR_SHAPE);
  bad([](Call &c) { c.width = 0; }, MX_ERR_SHAPE);
  bad([](Call &c) { c.width = 1025; }, MX_ERR_SHAPE);
  bad([](Call &c) { c.target = nullptr; }, MX_ERR_NULL);
  bad([](Call &c) { c.ids = nullptr; }, MX_ERR_NULL);
  bad([](Call &c) { c.up = nullptr; }, MX_ERR_NULL);
  bad([](Call &c) { c.cu = nullptr; }, MX_ERR_NULL);
  bad([](Call &c) { c.u = nullptr; }, MX_ERR_NULL);
  bad([](Call &c) { c.path = nullptr; }, MX_ERR_NULL);
  bad([](Call &c) { c.count = nullptr; }, MX_ERR_NULL);
  bad([](Call &c) { c.token = nullptr; }, MX_ERR_NULL);
  bad([](Call &c) { c.target = at<uint8_t>(1) + 4; }, MX_ERR_ALIGN);
  bad([](Call &c) { c.draft = at<uint8_t>(2) + 4; }, MX_ERR_ALIGN);
  bad([](Call &c) { c.ids = reinterpret_cast<int32_t *>(at<uint8_t>(4) + 1); }, MX_ERR_ALIGN);
  bad([](Call &c) { c.path = reinterpret_cast<int32_t *>(at<uint8_t>(8) + 1); }, MX_ERR_ALIGN);
  bad([](Call &c) { c.ws = nullptr; }, MX_ERR_WORKSPACE);
  bad([](Call &c) { c.ws = at<uint8_t>(3) + 4; }, MX_ERR_WORKSPACE);
  bad([](Call &c) { c.size = 10 * 64 - 1; }, MX_ERR_WORKSPACE);
  bad([](Call &c) { c.path = at<int32_t>(9); }, MX_ERR_ALIAS);
  bad([](Call &c) { c.token = at<int32_t>(4); }, MX_ERR_ALIAS);
  bad([](Call &c) { c.count = at<int32_t>(1); }, MX_ERR_ALIAS);
  bad([](Call &c) { c.ws = at<uint8_t>(2); }, MX_ERR_ALIAS);
  bad([](Call &c) { c.ws = at<uint8_t>(7); }, MX_ERR_ALIAS);
  CHECK(g_calls == calls);
  CHECK(call(ok) == MX_OK && g_calls == ++calls);
  CHECK(call(with(ok, [](Call &c) { c.draft = nullptr; c.dtype = MX_BF16; })) == MX_OK && g_calls == ++calls);
  // no tokens: outputs alone; no sequences: nothing
  CHECK(call(with(ok, [](Call &c) { c.tokens = 0; c.target = c.draft = nullptr; c.ws = nullptr; c.size = 0; })) == MX_OK &&
        g_calls == ++calls);
  CHECK(call(with(ok, [](Call &c) { c.tokens = 0; c.batch = 0; c.path = nullptr; })) == MX_OK && g_calls == calls);
  CHECK(mx_verify_drafts_workspace_size(10, 3, 1000) == 640);
  CHECK(mx_verify_drafts_workspace_size(10, 0, 1000) == 0 && mx_verify_drafts_workspace_size(0, 3, 1000) == 0 &&
        mx_verify_drafts_workspace_size(10, 3, 0) == 0);
}

int main() {
  std::vector<std::thread> threads;
  for (int i = 0; i < 4; i++)
    threads.emplace_back([] {
      for (int n = 0; n < 20; n++) {
        rotate();
        rotate_backward();
        cache_calls();
        verify();
      }
    });
  for (auto &t : threads) t.join();
  printf("draft ABI checks passed\n");
  return 0;
}
