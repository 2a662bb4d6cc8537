// mx_layer_checks.h - argument checks that the C ABI's files of the
// transformer-layer operators share. Nothing here makes a HIP call.
#ifndef MX_LAYER_CHECKS_H
#define MX_LAYER_CHECKS_H
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "mx_internal.h"
#include "mx_layer.h"

namespace mxc {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool dtype_ok(int d) { return d == MX_F32 || d == MX_BF16; }
inline int64_t elem_bytes(int d) { return d == MX_F32 ? 4 : 2; }
inline bool block_ok(int b) { return b == 32 || b == 128; }
inline int64_t blocks(int64_t k, int block) { return (k + block - 1) / block; }

// rows (< 2^31) x k (a positive multiple of 32) elements.
inline mx_status_t check_rows(int64_t rows, int64_t k, int64_t most_k) {
  if (rows < 0 || rows > INT32_MAX || k <= 0 || k % 32 != 0 || k > most_k) return MX_ERR_SHAPE;
  return MX_OK;
}

struct Range {
  const void *p;
  int64_t n;
};
inline bool overlap(const Range &a, const Range &b) {
  if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  return pa < pb + (uintptr_t)b.n && pb < pa + (uintptr_t)a.n;
}
// Any output against any input or a later output.
template <int O, int I>
inline bool clash(const Range (&out)[O], const Range (&in)[I]) {
  for (int i = 0; i < O; i++) {
    for (int j = 0; j < I; j++)
      if (overlap(out[i], in[j])) return true;
    for (int j = i + 1; j < O; j++)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

inline mx_status_t finish(hipError_t e) { return e == hipSuccess ? MX_OK : mxi_record_hip_error(e); }

inline hipStream_t stream_of(void *s) { return static_cast<hipStream_t>(s); }

constexpr int64_t kMaxColumns = 65535LL * 128;  // tiles of 128 in one grid dimension
constexpr int64_t kMaxProductK = 1 << 20;       // 32-bit offsets inside a tile of rows
constexpr int64_t kMaxLength = INT32_MAX - 2047;

inline mx_status_t check_cache(const mx_kv_cache_t *c, const mx_kv_batch_t *b) {
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
inline mx_status_t check_cache_pointers(const mx_kv_cache_t *c, const mx_kv_batch_t *b) {
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !b->table || !b->cu ||
      !b->lengths)
    return MX_ERR_NULL;
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes)) return MX_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(b->table) | reinterpret_cast<uintptr_t>(b->cu) |
       reinterpret_cast<uintptr_t>(b->lengths)) & 3u)
    return MX_ERR_ALIGN;
  return MX_OK;
}

inline mx_status_t check_attention(int64_t tokens, int batch, int q_heads, int heads, int dim,
                                   int64_t max_length) {
  if (tokens < 0 || tokens > INT32_MAX / 2 || batch < 0 || batch > (1 << 24)) return MX_ERR_SHAPE;
  if (heads < 1 || heads > 65535 || q_heads < heads || q_heads % heads || q_heads / heads > 128)
    return MX_ERR_SHAPE;
  if ((dim != 64 && dim != 128) || max_length < 0 || max_length > INT32_MAX) return MX_ERR_SHAPE;
  // workgroups of one launch: a row of heads per token, and per sequence
  if (tokens > 0 && (batch < 1 || (tokens + batch) > INT32_MAX / q_heads)) return MX_ERR_SHAPE;
  return MX_OK;
}

}  // namespace mxc
#endif  // MX_LAYER_CHECKS_H
