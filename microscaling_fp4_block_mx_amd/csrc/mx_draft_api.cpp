// mx_draft_api.cpp - C ABI of positions and drafted tokens: synchronous
// host-side argument validation, then asynchronous launches on the caller's
// stream. Every check runs before any HIP call.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "mx_internal.h"
#include "mx_layer.h"
#include "mx_layer_checks.h"

using namespace mxc;

namespace {

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Rows of `width` bytes, `stride` bytes apart.
struct Rows {
  const void *p;
  int64_t width, stride, rows;
  int64_t bytes() const { return rows > 0 ? (rows - 1) * stride + width : 0; }
};
// Whether two sets of rows share bytes. Parts of the same rows (one stride) lie
// between each other without sharing any.
bool share(const Rows &a, const Rows &b) {
  if (!overlap(Range{a.p, a.bytes()}, Range{b.p, b.bytes()})) return false;
  if (a.stride != b.stride) return true;
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  const int64_t at = ((d % a.stride) + a.stride) % a.stride;  // of b's row inside a's
  return at < a.width || at + b.width > a.stride;
}
bool share(const Rows &a, const void *p, int64_t bytes) {
  return share(a, Rows{p, bytes, bytes, bytes > 0 && p ? 1 : 0});
}

mx_status_t check_rotary(const mx_rotary_t *r, int dim) {
  if (!r || r->rot == 0) return MX_OK;
  if (r->rot < 0 || r->rot % 16 || r->rot > dim || r->length < 1 ||
      r->length > INT64_MAX / 4 / r->rot)
    return MX_ERR_SHAPE;
  return MX_OK;
}
mx_status_t check_rotary_pointers(const mx_rotary_t *r, bool positions) {
  if (!r || r->rot == 0) return MX_OK;
  if (!r->table || (positions && !r->positions)) return MX_ERR_NULL;
  if (!aligned16(r->table) || !aligned4(r->positions)) return MX_ERR_ALIGN;
  return MX_OK;
}
bool shares_rotary(const Rows &out, const mx_rotary_t *r, int64_t tokens) {
  if (!r || r->rot == 0) return false;
  return share(out, r->table, r->length * r->rot * 4) || share(out, r->positions, tokens * 4);
}

// Norm and rotation: what q's and k's shapes have to be.
mx_status_t check_norm_rotate(int q_heads, int k_heads, int dtype, int64_t tokens, int dim, float eps,
                              const mx_rotary_t *rotary) {
  if (!dtype_ok(dtype)) return MX_ERR_DTYPE;
  if (!(eps >= 0.0f) || isinf(eps)) return MX_ERR_SHAPE;
  if (dim != 64 && dim != 128 && dim != 256) return MX_ERR_SHAPE;
  if (tokens < 0 || tokens > INT32_MAX) return MX_ERR_SHAPE;
  if (q_heads < 1 || q_heads > 65535 || k_heads < 0 || k_heads > 65535) return MX_ERR_SHAPE;
  return check_rotary(rotary, dim);
}
mx_status_t check_stride(int64_t stride, int heads, int dim, int64_t tokens) {
  if (stride < (int64_t)heads * dim || stride > INT32_MAX) return MX_ERR_SHAPE;
  return tokens > 0 && stride > INT64_MAX / 8 / tokens ? MX_ERR_SHAPE : MX_OK;
}
bool stride_aligned(int64_t stride, int dtype) { return stride * elem_bytes(dtype) % 16 == 0; }

const mx_rotary_t kNoRotation = {};

}  // namespace

extern "C" {

mx_status_t mx_norm_rotate(const mx_heads_t *q, const mx_heads_t *k, mx_dtype_t dtype,
                           int64_t tokens, int dim, float eps, const mx_rotary_t *rotary,
                           void *stream) {
  if (!q) return MX_ERR_NULL;
  if (k && k->heads < 1) return MX_ERR_SHAPE;
  if (mx_status_t s = check_norm_rotate(q->heads, k ? k->heads : 0, dtype, tokens, dim, eps, rotary))
    return s;
  const mx_heads_t *both[] = {q, k};
  for (const mx_heads_t *h : both) {
    if (!h) continue;
    if (mx_status_t s = check_stride(h->x_stride, h->heads, dim, tokens)) return s;
    if (mx_status_t s = check_stride(h->y_stride, h->heads, dim, tokens)) return s;
  }
  if (tokens == 0) return MX_OK;
  const int64_t e = elem_bytes(dtype);
  for (const mx_heads_t *h : both) {
    if (!h) continue;
    if (!h->x || !h->y) return MX_ERR_NULL;
    if (!aligned16(h->x) || !aligned16(h->y) || !aligned16(h->weight) ||
        !stride_aligned(h->x_stride, dtype) || !stride_aligned(h->y_stride, dtype))
      return MX_ERR_ALIGN;
  }
  if (mx_status_t s = check_rotary_pointers(rotary, true)) return s;
  for (const mx_heads_t *h : both) {
    if (!h) continue;
    const Rows y = {h->y, h->heads * dim * e, h->y_stride * e, tokens};
    for (const mx_heads_t *o : both) {
      if (!o) continue;
      const Rows x = {o->x, o->heads * dim * e, o->x_stride * e, tokens};
      const bool in_place = o == h && h->x == h->y && h->x_stride == h->y_stride;
      if (!in_place && share(y, x)) return MX_ERR_ALIAS;
      if (o->weight && share(y, o->weight, dim * e)) return MX_ERR_ALIAS;
      if (o != h && share(y, Rows{o->y, o->heads * dim * e, o->y_stride * e, tokens}))
        return MX_ERR_ALIAS;
    }
    if (shares_rotary(y, rotary, tokens)) return MX_ERR_ALIAS;
  }
  return finish(mxi_launch_norm_rotate(*q, k, dtype == MX_BF16, tokens, dim, eps,
                                       rotary && rotary->rot ? *rotary : kNoRotation, stream_of(stream)));
}

size_t mx_norm_rotate_backward_workspace_size(int64_t tokens, int dim) {
  if (check_norm_rotate(1, 0, MX_BF16, tokens, dim, 0.0f, nullptr) != MX_OK) return 0;
  return (size_t)mxi_norm_rotate_partials(tokens) * dim * sizeof(float);
}

mx_status_t mx_norm_rotate_backward(const mx_heads_grad_t *q, const mx_heads_grad_t *k,
                                    mx_dtype_t dtype, int64_t tokens, int dim, float eps,
                                    const mx_rotary_t *rotary, void *workspace,
                                    size_t workspace_bytes, void *stream) {
  if (!q) return MX_ERR_NULL;
  if (k && k->heads < 1) return MX_ERR_SHAPE;
  if (mx_status_t s = check_norm_rotate(q->heads, k ? k->heads : 0, dtype, tokens, dim, eps, rotary))
    return s;
  const mx_heads_grad_t *both[] = {q, k};
  bool sums = false;
  for (const mx_heads_grad_t *h : both) {
    if (!h) continue;
    if (mx_status_t s = check_stride(h->dy_stride, h->heads, dim, tokens)) return s;
    if (mx_status_t s = check_stride(h->dx_stride, h->heads, dim, tokens)) return s;
    if (!h->weight) continue;
    sums = true;
    if (mx_status_t s = check_stride(h->x_stride, h->heads, dim, tokens)) return s;
    if (!h->dweight) return MX_ERR_NULL;
    if (!aligned16(h->dweight)) return MX_ERR_ALIGN;
  }
  if (q->weight && k && k->weight &&
      overlap(Range{q->dweight, 4 * (int64_t)dim}, Range{k->dweight, 4 * (int64_t)dim}))
    return MX_ERR_ALIAS;
  if (tokens > 0) {
    const int64_t e = elem_bytes(dtype);
    for (const mx_heads_grad_t *h : both) {
      if (!h) continue;
      if (!h->dy || !h->dx || (h->weight && !h->x)) return MX_ERR_NULL;
      if (!aligned16(h->dy) || !aligned16(h->dx) || !stride_aligned(h->dy_stride, dtype) ||
          !stride_aligned(h->dx_stride, dtype))
        return MX_ERR_ALIGN;
      if (h->weight &&
          (!aligned16(h->x) || !aligned16(h->weight) || !stride_aligned(h->x_stride, dtype)))
        return MX_ERR_ALIGN;
    }
    if (mx_status_t s = check_rotary_pointers(rotary, true)) return s;
    const int64_t need = sums ? (int64_t)mx_norm_rotate_backward_workspace_size(tokens, dim) : 0;
    if (need && (!workspace || !aligned16(workspace) || workspace_bytes < (size_t)need))
      return MX_ERR_WORKSPACE;
    const Rows ws = {workspace, need, need, need ? 1 : 0};
    for (const mx_heads_grad_t *h : both) {
      if (!h) continue;
      const int64_t width = h->heads * dim * e;
      const Rows dx = {h->dx, width, h->dx_stride * e, tokens};
      const Rows dw = {h->dweight, 4 * (int64_t)dim, 4 * (int64_t)dim, h->weight ? 1 : 0};
      for (const mx_heads_grad_t *o : both) {
        if (!o) continue;
        const int64_t ow = o->heads * dim * e;
        const Rows dy = {o->dy, ow, o->dy_stride * e, tokens};
        const Rows x = {o->x, ow, o->x_stride * e, o->weight ? tokens : 0};
        const Rows w = {o->weight, dim * e, dim * e, o->weight ? 1 : 0};
        const bool at_dy = o == h && h->dx == h->dy && h->dx_stride == h->dy_stride;
        const bool at_x = o == h && h->dx == h->x && h->dx_stride == h->x_stride;
        if ((!at_dy && share(dx, dy)) || (!at_x && share(dx, x)) || share(dx, w)) return MX_ERR_ALIAS;
        if (share(dw, dy) || share(dw, x) || share(dw, w)) return MX_ERR_ALIAS;
        if (share(ws, dy) || share(ws, x) || share(ws, w)) return MX_ERR_ALIAS;
        if (o != h && share(dx, Rows{o->dx, ow, o->dx_stride * e, tokens})) return MX_ERR_ALIAS;
        if (share(dx, o->dweight, o->weight ? 4 * (int64_t)dim : 0)) return MX_ERR_ALIAS;
      }
      if (share(ws, dx) || share(ws, dw) || shares_rotary(dx, rotary, tokens) ||
          shares_rotary(dw, rotary, tokens) || shares_rotary(ws, rotary, tokens))
        return MX_ERR_ALIAS;
    }
  }
  return finish(mxi_launch_norm_rotate_backward(*q, k, dtype == MX_BF16, tokens, dim, eps,
                                                rotary && rotary->rot ? *rotary : kNoRotation,
                                                static_cast<float *>(workspace), stream_of(stream)));
}

mx_status_t mx_kv_append_rotary(const void *k, const void *v, mx_dtype_t dtype, int64_t k_stride,
                                int64_t v_stride, const void *k_weight, float eps,
                                const mx_rotary_t *rotary, const mx_kv_cache_t *cache,
                                const mx_kv_batch_t *batch, void *stream) {
  if (!dtype_ok(dtype)) return MX_ERR_DTYPE;
  if (mx_status_t s = check_cache(cache, batch)) return s;
  if (!(eps >= 0.0f) || isinf(eps)) return MX_ERR_SHAPE;
  if (mx_status_t s = check_rotary(rotary, cache->dim)) return s;
  if (batch->tokens == 0) return MX_OK;
  const int64_t tokens = batch->tokens, e = elem_bytes(dtype);
  if (mx_status_t s = check_stride(k_stride, cache->heads, cache->dim, tokens)) return s;
  if (mx_status_t s = check_stride(v_stride, cache->heads, cache->dim, tokens)) return s;
  if (!k || !v) return MX_ERR_NULL;
  if (mx_status_t s = check_cache_pointers(cache, batch)) return s;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_weight) || !stride_aligned(k_stride, dtype) ||
      !stride_aligned(v_stride, dtype))
    return MX_ERR_ALIGN;
  if (mx_status_t s = check_rotary_pointers(rotary, false)) return s;
  const int64_t row = (int64_t)cache->heads * cache->dim;
  const int64_t codes = cache->pages * row * cache->page, scales = cache->pages * cache->heads;
  const bool turns = rotary && rotary->rot;
  const Range out[] = {{cache->k_codes, codes}, {cache->k_scales, scales},
                       {cache->v_codes, codes}, {cache->v_scales, scales}};
  const Range in[] = {{k, ((tokens - 1) * k_stride + row) * e},
                      {v, ((tokens - 1) * v_stride + row) * e},
                      {k_weight, cache->dim * e},
                      {turns ? rotary->table : nullptr, turns ? rotary->length * rotary->rot * 4 : 0},
                      {turns ? rotary->positions : nullptr, tokens * 4},
                      {batch->table, 4 * (int64_t)batch->batch * batch->width},
                      {batch->cu, 4 * ((int64_t)batch->batch + 1)},
                      {batch->lengths, 4 * (int64_t)batch->batch}};
  if (clash(out, in)) return MX_ERR_ALIAS;
  return finish(mxi_launch_kv_append_rotary(k, v, dtype == MX_BF16, k_stride, v_stride, k_weight,
                                            eps, turns ? *rotary : kNoRotation, *cache, *batch,
                                            stream_of(stream)));
}

size_t mx_kv_attention_tree_workspace_size(int64_t tokens, int batch, int q_heads, int heads,
                                           int dim, int64_t max_length) {
  if (check_attention(tokens, batch, q_heads, heads, dim, max_length) != MX_OK || tokens == 0)
    return 0;
  return mxi_kv_attention_tree_workspace(tokens, batch, q_heads, heads, dim,
                                         max_length == 0 ? INT32_MAX : max_length);
}

mx_status_t mx_kv_attention_tree(const void *q, int64_t q_stride, int q_heads,
                                 const mx_kv_cache_t *cache, const mx_kv_batch_t *batch,
                                 const uint32_t *mask, int words, int64_t max_length, float scale,
                                 void *out, void *workspace, size_t workspace_bytes, void *stream) {
  if (mx_status_t s = check_cache(cache, batch)) return s;
  if (mx_status_t s = check_attention(batch->tokens, batch->batch, q_heads, cache->heads,
                                      cache->dim, max_length))
    return s;
  if (words < 1 || words > 65535) return MX_ERR_SHAPE;
  if (!(scale > 0.0f) || isinf(scale)) return MX_ERR_SHAPE;
  if (batch->tokens == 0) return MX_OK;
  const int64_t row = (int64_t)q_heads * cache->dim;
  if (q_stride < row || q_stride > INT32_MAX) return MX_ERR_SHAPE;
  if (!q || !out || !mask) return MX_ERR_NULL;
  if (mx_status_t s = check_cache_pointers(cache, batch)) return s;
  if (!aligned16(q) || !aligned16(out) || q_stride % 8 || !aligned4(mask)) return MX_ERR_ALIGN;
  if (max_length == 0 || max_length > (int64_t)batch->width * cache->page)
    max_length = (int64_t)batch->width * cache->page;
  const size_t need = mxi_kv_attention_tree_workspace(batch->tokens, batch->batch, q_heads,
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
                      {mask, 4 * batch->tokens * words},
                      {batch->table, 4 * (int64_t)batch->batch * batch->width},
                      {batch->cu, 4 * ((int64_t)batch->batch + 1)},
                      {batch->lengths, 4 * (int64_t)batch->batch}};
  const Range outs[] = {{out, batch->tokens * row * 2}, {workspace, (int64_t)need}};
  if (clash(outs, in)) return MX_ERR_ALIAS;
  return finish(mxi_launch_kv_attention_tree(q, q_stride, q_heads, *cache, *batch, mask, words,
                                             max_length, scale, out, workspace, stream_of(stream)));
}

static mx_status_t check_verify(int64_t tokens, int batch, int64_t vocab) {
  if (tokens < 0 || tokens > INT32_MAX || batch < 0 || batch > 65535) return MX_ERR_SHAPE;
  if (vocab < 1 || vocab > INT32_MAX || (tokens > 0 && batch < 1)) return MX_ERR_SHAPE;
  // the rows' bytes, and workgroups of 8,192 elements of a row
  if (tokens > 0 && vocab > INT64_MAX / 8 / tokens) return MX_ERR_SHAPE;
  if ((vocab / 8192 + 2) * (int64_t)batch > INT32_MAX) return MX_ERR_SHAPE;
  return MX_OK;
}

size_t mx_verify_drafts_workspace_size(int64_t tokens, int batch, int64_t vocab) {
  if (check_verify(tokens, batch, vocab) != MX_OK || tokens == 0) return 0;
  return mxi_verify_workspace(tokens, batch, vocab);
}

mx_status_t mx_verify_drafts(const void *target, const void *draft, mx_dtype_t dtype,
                             const int32_t *ids, const int32_t *parents, const int32_t *cu,
                             const float *numbers, int64_t tokens, int batch, int64_t vocab,
                             int width, int32_t *path, int32_t *count, int32_t *token,
                             void *workspace, size_t workspace_bytes, void *stream) {
  if (!dtype_ok(dtype)) return MX_ERR_DTYPE;
  if (mx_status_t s = check_verify(tokens, batch, vocab)) return s;
  if (width < 1 || width > 1024) return MX_ERR_SHAPE;
  if (batch == 0) return MX_OK;
  if (!cu || !path || !count || !token) return MX_ERR_NULL;
  if (!aligned4(cu) || !aligned4(path) || !aligned4(count) || !aligned4(token)) return MX_ERR_ALIGN;
  const size_t need = mx_verify_drafts_workspace_size(tokens, batch, vocab);
  if (tokens > 0) {
    if (!target || !ids || !parents || !numbers) return MX_ERR_NULL;
    if (!aligned16(target) || !aligned16(draft) || !aligned4(ids) || !aligned4(parents) ||
        !aligned4(numbers))
      return MX_ERR_ALIGN;
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return MX_ERR_WORKSPACE;
  }
  const int64_t rows = tokens * vocab * elem_bytes(dtype), b = 4 * (int64_t)batch;
  const Range out[] = {{path, b * width}, {count, b}, {token, b}, {workspace, (int64_t)need}};
  const Range in[] = {{target, rows}, {draft, rows}, {ids, 4 * tokens}, {parents, 4 * tokens},
                      {cu, b + 4}, {numbers, 8 * tokens}};
  if (clash(out, in)) return MX_ERR_ALIAS;
  return finish(mxi_launch_verify(target, draft, dtype == MX_BF16, ids, parents, cu, numbers, tokens,
                                  batch, vocab, width, path, count, token, workspace,
                                  stream_of(stream)));
}

mx_status_t mx_kv_keep(const mx_kv_cache_t *cache, const mx_kv_batch_t *batch, const int32_t *path,
                       int path_width, const int32_t *count, void *stream) {
  if (!cache || !batch) return MX_ERR_NULL;
  mx_kv_batch_t of = *batch;  // its cu and tokens do not count
  of.cu = of.lengths;
  of.tokens = 0;
  if (mx_status_t s = check_cache(cache, &of)) return s;
  if (path_width < 1 || (int64_t)path_width > kMaxLength) return MX_ERR_SHAPE;
  if (of.batch == 0) return MX_OK;
  if (of.width < 1 || cache->pages < 1) return MX_ERR_SHAPE;
  if (mx_status_t s = check_cache_pointers(cache, &of)) return s;
  if (!path || !count) return MX_ERR_NULL;
  if (!aligned4(path) || !aligned4(count)) return MX_ERR_ALIGN;
  const int64_t codes = cache->pages * (int64_t)cache->heads * cache->dim * cache->page;
  const int64_t scales = cache->pages * cache->heads, b = 4 * (int64_t)of.batch;
  const Range out[] = {{cache->k_codes, codes}, {cache->k_scales, scales},
                       {cache->v_codes, codes}, {cache->v_scales, scales}};
  const Range in[] = {{of.table, b * of.width}, {of.lengths, b}, {path, b * path_width}, {count, b}};
  if (clash(out, in)) return MX_ERR_ALIAS;
  return finish(mxi_launch_kv_keep(*cache, of, path, path_width, count, stream_of(stream)));
}

}  // extern "C"
