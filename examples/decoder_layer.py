"""A decoder layer whose products, key/value cache and attention are MXFP8.

    python -m examples.decoder_layer

Serving: prompts of different lengths enter the cache in one call, then every
sequence takes one token at a time. Training: a norm and a linear layer, both
gradients from 8-bit products. Weights are quantized once; activations where
they are made. Position encodings are left out (a rotation of q and k between
the first product and the cache).
"""
from __future__ import annotations

import torch
import torch.nn.functional as F

import microscaling_fp4_block_mx_amd as mx

EPS = 1e-6


class DecoderLayer:
    """Pre-norm attention and gated feed-forward on the residual stream."""

    def __init__(self, hidden=1024, heads=16, kv_heads=4, dim=64, ffn=2048, block=128, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def linear(n, k):
            w = torch.randn(n, k, generator=g, device=device) / k ** 0.5
            return mx.quantize_mxfp8_rows(w.to(torch.bfloat16), block)

        self.heads, self.kv_heads, self.dim, self.block = heads, kv_heads, dim, block
        self.norm1 = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.norm2 = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.qkv = linear((heads + 2 * kv_heads) * dim, hidden)
        self.o = linear(hidden, heads * dim)
        self.gate_up = linear(2 * ffn, hidden)
        self.down = linear(hidden, ffn)

    def product(self, a, a_scales, weight):
        return mx.matmul_mxfp8(a, a_scales, *weight, block=self.block)

    def __call__(self, h, update, cache, table, cu, held, lengths, max_length=0):
        """h: the residual stream [tokens, hidden]; update: what the layer before
        adds to it (None for the first). Returns both for the next layer, whose
        first norm does the addition."""
        if update is None:
            x, scales, _ = mx.rmsnorm_mxfp8(h, self.norm1, EPS, block=self.block)
        else:
            x, scales, h = mx.rmsnorm_mxfp8(update, self.norm1, EPS, residual=h, block=self.block)
        tokens = h.shape[0]
        qkv = self.product(x, scales, self.qkv).view(tokens, -1, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)  # views: strides are fine
        mx.kv_append(cache, k, v, table, cu, held)
        o = mx.kv_attention(q, cache, table, cu, lengths, max_length=max_length)
        y = self.product(*mx.quantize_mxfp8_rows(o.view(tokens, -1), self.block), self.o)
        x, scales, h = mx.rmsnorm_mxfp8(y, self.norm2, EPS, residual=h, block=self.block)
        gate, up = self.product(x, scales, self.gate_up).chunk(2, -1)
        x, scales = mx.quantize_mxfp8_rows(F.silu(gate) * up, self.block)
        return h, self.product(x, scales, self.down)


class Pages:
    """Page tables for a batch whose sequences grow: sequence i owns pages
    i width .. (i + 1) width - 1."""

    def __init__(self, batch, longest, page, device="cuda"):
        self.width = -(-longest // page)
        self.table = torch.arange(batch * self.width, dtype=torch.int32, device=device)
        self.table = self.table.view(batch, self.width)
        self.held = torch.zeros(batch, dtype=torch.int32, device=device)

    def step(self, new):
        """cu, held and lengths for `new` tokens of each sequence (a CPU list)."""
        new = torch.tensor(new, dtype=torch.int32)
        cu = F.pad(new.cumsum(0, dtype=torch.int32), (1, 0)).to(self.held.device)
        held, self.held = self.held, self.held + new.to(self.held.device)
        return cu, held, self.held


def serve(layer, prompts, steps, page=64, seed=1):
    """Prefill, then `steps` single tokens; yields each call's (h, update)."""
    longest = max(prompts) + steps
    pages = Pages(len(prompts), longest, page)
    cache = mx.kv_cache(len(prompts) * pages.width, layer.kv_heads, layer.dim, page)
    g = torch.Generator(device="cuda").manual_seed(seed)
    hidden = layer.norm1.numel()
    for new in [list(prompts)] + [[1] * len(prompts)] * steps:
        h = torch.randn(sum(new), hidden, generator=g, device="cuda").to(torch.bfloat16)
        cu, held, lengths = pages.step(new)
        yield h, layer(h, None, cache, pages.table, cu, held, lengths, max_length=longest)


def train_step(x, gain, weight, target, block=32):
    """y = norm(x) weight^T against `target` -> (loss, gradients of x, gain and
    weight), the loss being the mean square. The three products run on 8-bit
    operands: y sums over features, dx over outputs, dweight over tokens."""
    n, n_scales, _ = mx.rmsnorm_mxfp8(x, gain, EPS, block=block)
    w, w_scales, w_t, w_t_scales = mx.quantize_mxfp8_both(weight, block)
    y = mx.matmul_mxfp8(n, n_scales, w, w_scales, block=block).float()
    loss = F.mse_loss(y, target)
    dy = ((y - target) * (2 / y.numel())).to(torch.bfloat16)
    d, d_scales, d_t, d_t_scales = mx.quantize_mxfp8_both(dy, block)
    # the norm's output as the product saw it, by columns (its 8-bit values are exact in bfloat16)
    n_t, n_t_scales = mx.quantize_mxfp8_columns(mx.dequantize_mxfp8(n, n_scales), block)
    dn = mx.matmul_mxfp8(d, d_scales, w_t, w_t_scales, block=block)
    dweight = mx.matmul_mxfp8(d_t, d_t_scales, n_t, n_t_scales, torch.float32, block=block)
    dx, dgain = mx.rmsnorm_backward(dn, x, gain, EPS)
    return loss, dx, dgain, dweight


def main():
    layer = DecoderLayer()
    for i, (h, (stream, update)) in enumerate(serve(layer, [300, 7, 120, 1], 8)):
        if i in (0, 8):
            print(f"call {i}: {h.shape[0]} tokens, |update| / |h| = "
                  f"{(update.float().norm() / stream.float().norm()).item():.3f}")
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(2000, 512, generator=g, device="cuda").to(torch.bfloat16)
    weight = torch.randn(768, 512, generator=g, device="cuda") * 0.02
    gain = torch.ones(512, device="cuda")
    target = torch.randn(2000, 768, generator=g, device="cuda") * 0.5
    for step in range(5):
        loss, _, dgain, dweight = train_step(x, gain.to(x.dtype), weight.to(x.dtype), target)
        weight -= 200.0 * dweight
        gain -= 20.0 * dgain
        print(f"step {step}: loss {loss.item():.5f}")


if __name__ == "__main__":
    main()
