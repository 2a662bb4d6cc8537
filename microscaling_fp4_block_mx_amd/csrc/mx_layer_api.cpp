// mx_layer_api.cpp - C ABI of the transformer-layer operators: synchronous
// host-side argument validation, then asynchronous launches on the caller's
// stream. Every check runs before any HIP call.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "mx_internal.h"
#include "mx_layer.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dtype_ok(int d) { return d == MX_F32 || d == MX_BF16; }
int64_t elem_bytes(int d) { return d == MX_F32 ? 4 : 2; }
bool block_ok(int b) { return b == 32 || b == 128; }
int64_t blocks(int64_t k, int block) { return (k + block - 1) / block; }

// rows (< 2^31) x k (a positive multiple of 32) elements.
mx_status_t check_rows(int64_t rows, int64_t k, int64_t most_k) {
  if (rows < 0 || rows > INT32_MAX || k <= 0 || k % 32 != 0 || k > most_k) return MX_ERR_SHAPE;
  return MX_OK;
}

struct Range {
  const void *p;
  int64_t n;
};
bool overlap(const Range &a, const Range &b) {
  if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  return pa < pb + (uintptr_t)b.n && pb < pa + (uintptr_t)a.n;
}
// Any output against any input or a later output.
template <int O, int I>
bool clash(const Range (&out)[O], const Range (&in)[I]) {
  for (int i = 0; i < O; i++) {
    for (int j = 0; j < I; j++)
      if (overlap(out[i], in[j])) return true;
    for (int j = i + 1; j < O; j++)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

mx_status_t finish(hipError_t e) { return e == hipSuccess ? MX_OK : mxi_record_hip_error(e); }

hipStream_t stream_of(void *s) { return static_cast<hipStream_t>(s); }

constexpr int64_t kMaxColumns = 65535LL * 128;  // tiles of 128 in one grid dimension
constexpr int64_t kMaxProductK = 1 << 20;       // 32-bit offsets inside a tile of rows
constexpr int64_t kMaxLength = INT32_MAX - 2047;

mx_status_t check_cache(const mx_kv_cache_t *c, const mx_kv_batch_t *b) {
  if (!c || !b) return MX_ERR_NULL;
  if (c->dim != 64 && c->dim != 128) return MX_ERR_SHAPE;
  if (c->page < 32 || c->page > 256 || (c->page & (c->page - 1))) return MX_ERR_SHAPE;
  if (c->heads < 1 || c->heads > 65535 || c->pages < 0 || c->pages > INT32_MAX) return MX_ERR_SHAPE;
  if (b->tokens < 0 || b->tokens > INT32_MAX / 2 || b->batch < 0 || b->batch > (1 << 24) ||
      b->width < 0)
    return MX_ERR_SHAPE;
  // lengths and positions are 32-bit, those of the tiles that are asked for ahead too
  if ((int64_t)b->width * c->page > kMaxLength) return MX_ERR_SHAPE;
  if (b->tokens > 0 && (b->batch < 1 || b->width < 1 || c->pages < 1)) return MX_ERR_SHAPE;
  // workgroups of one launch: at most two pages more than whole ones per sequence
  if (b->tokens / c->page + 2 * (int64_t)b->batch > INT32_MAX / c->heads) return MX_ERR_SHAPE;
  return MX_OK;
}
mx_status_t check_cache_pointers(const mx_kv_cache_t *c, const mx_kv_batch_t *b) {
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !b->table || !b->cu ||
      !b->lengths)
    return MX_ERR_NULL;
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes)) return MX_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(b->table) | reinterpret_cast<uintptr_t>(b->cu) |
       reinterpret_cast<uintptr_t>(b->lengths)) & 3u)
    return MX_ERR_ALIGN;
  return MX_OK;
}

}  // namespace

extern "C" {

mx_status_t mx_quantize_mxfp8_blocks(const void *x, mx_dtype_t x_dtype, int64_t rows, int64_t k,
                                     int block, uint8_t *codes, uint8_t *scales, uint8_t *codes_t,
                                     uint8_t *scales_t, void *stream) {
  if (!dtype_ok(x_dtype)) return MX_ERR_DTYPE;
  if (!block_ok(block)) return MX_ERR_SHAPE;
  if (mx_status_t s = check_rows(rows, k, kMaxColumns)) return s;
  if (rows == 0) return MX_OK;
  if (!x || (!codes && !codes_t) || !codes != !scales || !codes_t != !scales_t) return MX_ERR_NULL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned16(codes_t) ||
      !aligned16(scales_t))
    return MX_ERR_ALIGN;
  const int64_t padded = (rows + 31) & ~(int64_t)31;
  const Range out[] = {{codes, rows * k},
                       {scales, rows * blocks(k, block)},
                       {codes_t, padded * k},
                       {scales_t, k * blocks(rows, block)}};
  const Range in[] = {{x, rows * k * elem_bytes(x_dtype)}};
  if (clash(out, in)) return MX_ERR_ALIAS;
  return finish(mxi_launch_quantize8_blocks(x, x_dtype == MX_BF16, rows, k, block, codes, scales,
                                            codes_t, scales_t, stream_of(stream)));
}

mx_status_t mx_rmsnorm_mxfp8(const void *x, const void *residual, const void *weight,
                             mx_dtype_t dtype, int64_t rows, int64_t k, float eps, int block,
                             uint8_t *codes, uint8_t *scales, void *h_out, void *stream) {
  if (!dtype_ok(dtype)) return MX_ERR_DTYPE;
  if (!block_ok(block) || !(eps >= 0.0f)) return MX_ERR_SHAPE;
  if (mx_status_t s = check_rows(rows, k, kNormMaxK)) return s;
  if (rows == 0) return MX_OK;
  if (!x || !weight || !codes || !scales || (h_out && !residual)) return MX_ERR_NULL;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(codes) ||
      !aligned16(scales) || !aligned16(h_out))
    return MX_ERR_ALIGN;
  const int64_t n = rows * k * elem_bytes(dtype);
  const Range w = {weight, k * elem_bytes(dtype)}, xr = {x, n}, rr = {residual, n}, hr = {h_out, n};
  const Range out[] = {{codes, rows * k}, {scales, rows * blocks(k, block)}};
  const Range in[] = {xr, rr, w, hr};
  if (clash(out, in)) return MX_ERR_ALIAS;
  if (overlap(hr, w) || (h_out != x && overlap(hr, xr)) || (h_out != residual && overlap(hr, rr)))
    return MX_ERR_ALIAS;
  return finish(mxi_launch_rmsnorm(x, residual, weight, dtype == MX_BF16, rows, k, eps, block,
                                   codes, scales, h_out, stream_of(stream)));
}

size_t mx_rmsnorm_backward_workspace_size(int64_t rows, int64_t k) {
  if (check_rows(rows, k, kNormMaxK) != MX_OK) return 0;
  return (size_t)mxi_rmsnorm_partials(rows, k) * k * sizeof(float);
}

mx_status_t mx_rmsnorm_backward(const void *dy, const void *h, const void *weight,
                                const void *through, mx_dtype_t dtype, int64_t rows, int64_t k,
                                float eps, void *dx, float *dweight, void *workspace,
                                size_t workspace_bytes, void *stream) {
  if (!dtype_ok(dtype)) return MX_ERR_DTYPE;
  if (!(eps >= 0.0f)) return MX_ERR_SHAPE;
  if (mx_status_t s = check_rows(rows, k, kNormMaxK)) return s;
  if (!dweight) return MX_ERR_NULL;
  if (!aligned16(dweight)) return MX_ERR_ALIGN;
  if (rows > 0) {
    if (!dy || !h || !weight || !dx) return MX_ERR_NULL;
    if (!aligned16(dy) || !aligned16(h) || !aligned16(weight) || !aligned16(through) ||
        !aligned16(dx))
      return MX_ERR_ALIGN;
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < mx_rmsnorm_backward_workspace_size(rows, k))
      return MX_ERR_WORKSPACE;
    const int64_t n = rows * k * elem_bytes(dtype);
    const Range in[] = {{dy, n}, {h, n}, {through, n}, {weight, k * elem_bytes(dtype)}};
    const Range out[] = {{dweight, 4 * k}, {workspace, (int64_t)workspace_bytes}};
    const Range xr = {dx, n};
    if (clash(out, in)) return MX_ERR_ALIAS;
    for (const Range &r : in)
      if (r.p != dx && overlap(xr, r)) return MX_ERR_ALIAS;
    if (weight == dx || overlap(xr, out[0]) || overlap(xr, out[1])) return MX_ERR_ALIAS;
  }
  return finish(mxi_launch_rmsnorm_backward(dy, h, weight, through, dtype == MX_BF16, rows, k, eps,
                                            dx, dweight, static_cast<float *>(workspace),
                                            stream_of(stream)));
}

static mx_status_t check_product(int64_t m, int64_t n, int64_t k, int block, int c_dtype) {
  if (!dtype_ok(c_dtype)) return MX_ERR_DTYPE;
  if (!block_ok(block)) return MX_ERR_SHAPE;
  if (m < 0 || m > INT32_MAX || n < 0 || n > INT32_MAX || k <= 0 || k % 32 != 0 ||
      k > kMaxProductK)
    return MX_ERR_SHAPE;
  // the output's elements, and one launch's tiles of 128 x 128, 256 threads
  // each, whose threads (and those of tiles of 256 x 256) are fewer than 2^32
  if (m > 0 && n > 0 &&
      (n > INT64_MAX / 8 / m || ((m + 127) / 128) * ((n + 127) / 128) > (1 << 24) - 2))
    return MX_ERR_SHAPE;
  return MX_OK;
}

size_t mx_matmul_mxfp8_workspace_size(int64_t m, int64_t n, int64_t k, int block,
                                      mx_dtype_t c_dtype) {
  if (check_product(m, n, k, block, c_dtype) != MX_OK || m == 0 || n == 0) return 0;
  return mxi_matmul8_workspace(m, n, k, block, c_dtype == MX_BF16);
}

mx_status_t mx_matmul_mxfp8(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b,
                            const uint8_t *b_scales, int64_t m, int64_t n, int64_t k, int block,
                            mx_dtype_t c_dtype, void *c, void *workspace, size_t workspace_bytes,
                            void *stream) {
  if (mx_status_t s = check_product(m, n, k, block, c_dtype)) return s;
  if (m == 0 || n == 0) return MX_OK;
  if (!a || !a_scales || !b || !b_scales || !c) return MX_ERR_NULL;
  if (!aligned16(a) || !aligned16(a_scales) || !aligned16(b) || !aligned16(b_scales) ||
      !aligned16(c))
    return MX_ERR_ALIGN;
  const size_t need = mxi_matmul8_workspace(m, n, k, block, c_dtype == MX_BF16);
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return MX_ERR_WORKSPACE;
  const Range in[] = {{a, m * k}, {a_scales, m * blocks(k, block)}, {b, n * k},
                      {b_scales, n * blocks(k, block)}};
  const Range out[] = {{c, m * n * elem_bytes(c_dtype)}, {workspace, (int64_t)need}};
  if (clash(out, in)) return MX_ERR_ALIAS;
  return finish(mxi_launch_matmul8(a, a_scales, b, b_scales, m, n, k, block, c_dtype == MX_BF16, c,
                                   workspace, stream_of(stream)));
}

mx_status_t mx_kv_append(const void *k, const void *v, mx_dtype_t dtype, int64_t k_stride,
                         int64_t v_stride, const mx_kv_cache_t *cache, const mx_kv_batch_t *batch,
                         void *stream) {
  if (!dtype_ok(dtype)) return MX_ERR_DTYPE;
  if (mx_status_t s = check_cache(cache, batch)) return s;
  if (batch->tokens == 0) return MX_OK;
  const int64_t row = (int64_t)cache->heads * cache->dim, e = elem_bytes(dtype);
  if (k_stride < row || v_stride < row || k_stride > INT32_MAX || v_stride > INT32_MAX)
    return MX_ERR_SHAPE;
  if (!k || !v) return MX_ERR_NULL;
  if (mx_status_t s = check_cache_pointers(cache, batch)) return s;
  if (!aligned16(k) || !aligned16(v) || (k_stride * e) % 16 || (v_stride * e) % 16)
    return MX_ERR_ALIGN;
  const int64_t codes = cache->pages * row * cache->page, scales = cache->pages * cache->heads;
  const Range out[] = {{cache->k_codes, codes}, {cache->k_scales, scales},
                       {cache->v_codes, codes}, {cache->v_scales, scales}};
  const Range in[] = {{k, ((batch->tokens - 1) * k_stride + row) * e},
                      {v, ((batch->tokens - 1) * v_stride + row) * e},
                      {batch->table, 4 * (int64_t)batch->batch * batch->width},
                      {batch->cu, 4 * ((int64_t)batch->batch + 1)},
                      {batch->lengths, 4 * (int64_t)batch->batch}};
  if (clash(out, in)) return MX_ERR_ALIAS;
  return finish(mxi_launch_kv_append(k, v, dtype == MX_BF16, k_stride, v_stride, *cache, *batch,
                                     stream_of(stream)));
}

static mx_status_t check_attention(int64_t tokens, int batch, int q_heads, int heads, int dim,
                                   int64_t max_length) {
  if (tokens < 0 || tokens > INT32_MAX / 2 || batch < 0 || batch > (1 << 24)) return MX_ERR_SHAPE;
  if (heads < 1 || heads > 65535 || q_heads < heads || q_heads % heads || q_heads / heads > 128)
    return MX_ERR_SHAPE;
  if ((dim != 64 && dim != 128) || max_length < 0 || max_length > INT32_MAX) return MX_ERR_SHAPE;
  // workgroups of one launch: a row of heads per token, and per sequence
  if (tokens > 0 && (batch < 1 || (tokens + batch) > INT32_MAX / q_heads)) return MX_ERR_SHAPE;
  return MX_OK;
}

size_t mx_kv_attention_workspace_size(int64_t tokens, int batch, int q_heads, int heads, int dim,
                                      int64_t max_length) {
  if (check_attention(tokens, batch, q_heads, heads, dim, max_length) != MX_OK || tokens == 0)
    return 0;
  // the call plans for the table's room where that is less: the size grows with the length
  return mxi_kv_attention_workspace(tokens, batch, q_heads, heads, dim,
                                    max_length == 0 ? INT32_MAX : max_length);
}

mx_status_t mx_kv_attention(const void *q, int64_t q_stride, int q_heads,
                            const mx_kv_cache_t *cache, const mx_kv_batch_t *batch,
                            int64_t max_length, float scale, void *out, void *workspace,
                            size_t workspace_bytes, void *stream) {
  if (mx_status_t s = check_cache(cache, batch)) return s;
  if (mx_status_t s = check_attention(batch->tokens, batch->batch, q_heads, cache->heads,
                                      cache->dim, max_length))
    return s;
  if (!(scale > 0.0f) || isinf(scale)) return MX_ERR_SHAPE;
  if (batch->tokens == 0) return MX_OK;
  const int64_t row = (int64_t)q_heads * cache->dim;
  if (q_stride < row || q_stride > INT32_MAX) return MX_ERR_SHAPE;
  if (!q || !out) return MX_ERR_NULL;
  if (mx_status_t s = check_cache_pointers(cache, batch)) return s;
  if (!aligned16(q) || !aligned16(out) || q_stride % 8) return MX_ERR_ALIGN;
  if (max_length == 0 || max_length > (int64_t)batch->width * cache->page)
    max_length = (int64_t)batch->width * cache->page;
  const size_t need = mxi_kv_attention_workspace(batch->tokens, batch->batch, q_heads,
                                                 cache->heads, cache->dim, max_length);
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return MX_ERR_WORKSPACE;
  const int64_t codes = cache->pages * (int64_t)cache->heads * cache->dim * cache->page;
  const int64_t scales = cache->pages * cache->heads;
  const Range in[] = {{q, ((batch->tokens - 1) * q_stride + row) * 2},
                      {cache->k_codes, codes},
                      {cache->k_scales, scales},
                      {cache->v_codes, codes},
                      {cache->v_scales, scales},
                      {batch->table, 4 * (int64_t)batch->batch * batch->width},
                      {batch->cu, 4 * ((int64_t)batch->batch + 1)},
                      {batch->lengths, 4 * (int64_t)batch->batch}};
  const Range outs[] = {{out, batch->tokens * row * 2}, {workspace, (int64_t)need}};
  if (clash(outs, in)) return MX_ERR_ALIAS;
  return finish(mxi_launch_kv_attention(q, q_stride, q_heads, *cache, *batch, max_length, scale,
                                        out, workspace, stream_of(stream)));
}

}  // extern "C"
