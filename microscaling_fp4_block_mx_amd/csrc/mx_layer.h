// mx_layer.h - launchers of the transformer-layer operators (RMS norm, MXFP8
// products, 8-bit KV cache and attention) shared by the C ABI
// (mx_layer_api.cpp) and the kernels. Arguments have been validated.
#ifndef MX_LAYER_H
#define MX_LAYER_H
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx.h"

// Longest row of the norm (and its gradient): 1024 threads hold it in
// registers, 64 elements each.
constexpr int64_t kNormMaxK = 65536;

hipError_t mxi_launch_rmsnorm(const void *x, const void *residual, const void *weight, int bf16,
                              int64_t rows, int64_t k, float eps, int block, uint8_t *codes,
                              uint8_t *scales, void *h, hipStream_t st);
// Workgroups (= rows of partial weight gradients, k floats each) of the
// gradient's launch.
int64_t mxi_rmsnorm_partials(int64_t rows, int64_t k);
hipError_t mxi_launch_rmsnorm_backward(const void *dy, const void *h, const void *weight,
                                       const void *through, int bf16, int64_t rows, int64_t k,
                                       float eps, void *dx, float *dweight, float *partial,
                                       hipStream_t st);
hipError_t mxi_launch_quantize8_blocks(const void *x, int bf16, int64_t rows, int64_t k, int block,
                                       uint8_t *codes, uint8_t *scales, uint8_t *codes_t,
                                       uint8_t *scales_t, hipStream_t st);

// Split of the product's launch: workspace bytes it needs (0 where one
// workgroup adds a whole row of K).
size_t mxi_matmul8_workspace(int64_t m, int64_t n, int64_t k, int block, int out_bf16);
hipError_t mxi_launch_matmul8(const uint8_t *a, const uint8_t *a_scales, const uint8_t *b,
                              const uint8_t *b_scales, int64_t m, int64_t n, int64_t k, int block,
                              int out_bf16, void *c, void *workspace, hipStream_t st);

hipError_t mxi_launch_kv_append(const void *k, const void *v, int bf16, int64_t k_stride,
                                int64_t v_stride, const mx_kv_cache_t &cache,
                                const mx_kv_batch_t &batch, hipStream_t st);
// Enough for a launch with this max_length or any smaller one.
size_t mxi_kv_attention_workspace(int64_t tokens, int batch, int q_heads, int heads, int dim,
                                  int64_t max_length);
hipError_t mxi_launch_kv_attention(const void *q, int64_t q_stride, int q_heads,
                                   const mx_kv_cache_t &cache, const mx_kv_batch_t &batch,
                                   int64_t max_length, float scale, void *out, void *workspace,
                                   hipStream_t st);

hipError_t mxi_launch_kv_append_rotary(const void *k, const void *v, int bf16, int64_t k_stride,
                                       int64_t v_stride, const void *weight, float eps,
                                       const mx_rotary_t &rotary, const mx_kv_cache_t &cache,
                                       const mx_kv_batch_t &batch, hipStream_t st);
size_t mxi_kv_attention_tree_workspace(int64_t tokens, int batch, int q_heads, int heads, int dim,
                                       int64_t max_length);
hipError_t mxi_launch_kv_attention_tree(const void *q, int64_t q_stride, int q_heads,
                                        const mx_kv_cache_t &cache, const mx_kv_batch_t &batch,
                                        const uint32_t *mask, int words, int64_t max_length,
                                        float scale, void *out, void *workspace, hipStream_t st);

// Heads' norms and rotation; `k` may be NULL, `rotary` with rot = 0 turns nothing.
hipError_t mxi_launch_norm_rotate(const mx_heads_t &q, const mx_heads_t *k, int bf16,
                                  int64_t tokens, int dim, float eps, const mx_rotary_t &rotary,
                                  hipStream_t st);
// Rows of partial weight gradients (dim floats each) of the gradient's launch.
int64_t mxi_norm_rotate_partials(int64_t tokens);
hipError_t mxi_launch_norm_rotate_backward(const mx_heads_grad_t &q, const mx_heads_grad_t *k,
                                           int bf16, int64_t tokens, int dim, float eps,
                                           const mx_rotary_t &rotary, float *partial,
                                           hipStream_t st);

// Drafted tokens: scratch of a verification, the verification (`draft` may be
// NULL), and the accepted tokens' move.
size_t mxi_verify_workspace(int64_t tokens, int batch, int64_t vocab);
hipError_t mxi_launch_verify(const void *target, const void *draft, int bf16, const int32_t *ids,
                             const int32_t *parents, const int32_t *cu, const float *numbers,
                             int64_t tokens, int batch, int64_t vocab, int width, int32_t *path,
                             int32_t *count, int32_t *token, void *workspace, hipStream_t st);
hipError_t mxi_launch_kv_keep(const mx_kv_cache_t &cache, const mx_kv_batch_t &batch,
                              const int32_t *path, int path_width, const int32_t *count,
                              hipStream_t st);
#endif  // MX_LAYER_H
