"""Serving with drafted tokens: positions, per-head norms, a tree of drafts a step.

    python -m examples.drafted_tokens

A small language model (embedding, decoder layers as in examples.decoder_layer with
norms of q and k and the position rotation, head) takes prompts, then, each step, a
tree of tokens that a table of token pairs proposes: every node is read in one call,
the target's probabilities decide how far down the tree the text goes, and the cache
keeps the accepted tokens alone. What comes out is distributed as the model's own
samples. Weights are random: how many drafts are taken says nothing here.
"""
from __future__ import annotations

import torch
import torch.nn.functional as F

import microscaling_fp4_block_mx_amd as mx

from .decoder_layer import EPS, DecoderLayer, Pages

TREE = [-1, 0, 0, 1, 1, 2, 3]  # each node's parent: two tokens behind the last one, two behind the first of them, ..


class PositionedLayer(DecoderLayer):
    """The decoder layer with norms of q and k per head and their rotation."""

    def __init__(self, table, **sizes):
        super().__init__(**sizes)
        self.table = table
        self.q_norm = torch.ones(self.dim, dtype=torch.bfloat16, device=table.device)
        self.k_norm = torch.ones(self.dim, dtype=torch.bfloat16, device=table.device)

    def __call__(self, h, update, cache, pages, cu, held, lengths, positions, mask=None, max_length=0):
        """As DecoderLayer's; `positions` of the new tokens, and `mask` where they are a tree's."""
        if update is None:
            x, scales, _ = mx.rmsnorm_mxfp8(h, self.norm1, EPS, block=self.block)
        else:
            x, scales, h = mx.rmsnorm_mxfp8(update, self.norm1, EPS, residual=h, block=self.block)
        tokens = h.shape[0]
        qkv = self.product(x, scales, self.qkv).view(tokens, -1, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        rotary = mx.Rotary(self.table, positions)
        q, _ = mx.norm_rotate(q, None, self.q_norm, None, rotary, EPS)
        mx.kv_append_rotary(cache, k, v, pages, cu, held, rotary, self.k_norm, EPS)
        if mask is None:
            o = mx.kv_attention(q, cache, pages, cu, lengths, max_length=max_length)
        else:
            o = mx.kv_attention_tree(q, cache, pages, cu, lengths, mask, max_length=max_length)
        y = self.product(*mx.quantize_mxfp8_rows(o.view(tokens, -1), self.block), self.o)
        x, scales, h = mx.rmsnorm_mxfp8(y, self.norm2, EPS, residual=h, block=self.block)
        gate, up = self.product(x, scales, self.gate_up).chunk(2, -1)
        x, scales = mx.quantize_mxfp8_rows(F.silu(gate) * up, self.block)
        return h, self.product(x, scales, self.down)


class Model:
    """Embedding, layers, head; probabilities of the next token behind every token given."""

    def __init__(self, vocab=1000, hidden=512, layers=2, longest=256, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        table = mx.rotary_table(longest, 64, device=device)
        self.embedding = torch.randn(vocab, hidden, generator=g, device=device).to(torch.bfloat16)
        self.layers = [PositionedLayer(table, hidden=hidden, heads=8, kv_heads=2, dim=64, ffn=2 * hidden, seed=i,
                                       device=device) for i in range(layers)]
        self.norm = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.head = mx.quantize_mxfp8_rows((torch.randn(vocab, hidden, generator=g, device=device)
                                            / hidden ** 0.5).to(torch.bfloat16))

    def caches(self, batch, longest, page=64):
        """(caches, pages) for sequences of up to `longest` tokens."""
        pages = Pages(batch, longest, page)
        return [mx.kv_cache(batch * pages.width, layer.kv_heads, layer.dim, page) for layer in self.layers], pages

    def __call__(self, ids, caches, pages, cu, held, lengths, positions, mask=None, max_length=0, temperature=1.0):
        h, update = self.embedding[ids.long()], None
        for layer, cache in zip(self.layers, caches):
            h, update = layer(h, update, cache, pages, cu, held, lengths, positions, mask, max_length)
        x, scales, _ = mx.rmsnorm_mxfp8(update, self.norm, EPS, residual=h)
        logits = mx.matmul_mxfp8(x, scales, *self.head, torch.float32)
        return torch.softmax(logits / temperature, 1)


def serve(model, prompts, steps, pairs, tree=TREE, temperature=0.7, seed=1):
    """prompts: lists of token ids; pairs [vocab, vocab]: the draft's probabilities of
    what follows a token. Yields, for the prompts and each step, (path, count, token):
    which drafts were taken, and the token behind them."""
    device, batch, nodes = pairs.device, len(prompts), len(tree)
    longest = max(len(p) for p in prompts) + (steps + 1) * nodes
    caches, pages = model.caches(batch, longest)
    g = torch.Generator(device=device).manual_seed(seed)

    def numbers(rows):
        return torch.rand(rows, 2, generator=g, device=device)

    # prompts: every prompt is a chain that has been taken but for its next token
    new = [len(p) for p in prompts]
    cu, held, lengths = pages.step(new)
    ids = torch.tensor(sum(prompts, []), dtype=torch.int32, device=device)
    positions = torch.cat([torch.arange(n, dtype=torch.int32, device=device) for n in new])
    p = model(ids, caches, pages.table, cu, held, lengths, positions, max_length=longest, temperature=temperature)
    last = (cu[1:] - 1).long()
    one = torch.arange(batch + 1, dtype=torch.int32, device=device)
    path, count, token = mx.verify_drafts(p[last].contiguous(), ids[last], torch.full_like(ids[:batch], -1), one,
                                          numbers(batch), 1)
    yield path, count, token
    # the tree's shape is the same each step: its masks and depths are formed once
    mask, depth = mx.tree_mask([tree] * batch, device=device)
    parents = torch.tensor(tree * batch, dtype=torch.int32, device=device)
    rank = torch.tensor([sum(q == up for q in tree[:j]) for j, up in enumerate(tree)], device=device)
    cu = torch.arange(batch + 1, dtype=torch.int32, device=device) * nodes
    width = int(depth.max()) + 1
    held = lengths
    for _ in range(steps):
        ids = torch.empty(batch, nodes, dtype=torch.int64, device=device)
        ids[:, 0] = token
        for j in range(1, nodes):  # children are draws from what follows their parent, one behind the other
            draws = torch.multinomial(pairs[ids[:, tree[j]]], int(rank[j]) + 1, generator=g)
            ids[:, j] = draws[:, -1]
        flat = ids.view(-1).int()
        positions = depth + held.repeat_interleave(nodes)
        p = model(flat, caches, pages.table, cu, held, held + nodes, positions, mask, longest, temperature)
        path, count, token = mx.verify_drafts(p, flat, parents, cu, numbers(batch * nodes), width,
                                              draft=pairs[flat.long()].contiguous())
        for cache in caches:
            mx.kv_keep(cache, pages.table, held, path, count)
        held = held + count
        yield path, count, token


def main():
    model = Model()
    g = torch.Generator(device="cuda").manual_seed(3)
    pairs = torch.softmax(torch.randn(1000, 1000, generator=g, device="cuda") * 2, 1)
    prompts = [[5, 17, 300], [42], list(range(100, 120))]
    total = 0
    for i, (path, count, token) in enumerate(serve(model, prompts, 6, pairs)):
        total += int(count.sum())
        print(f"step {i}: taken {count.tolist()}, next {token.tolist()}")
    print(f"{total} tokens for {len(prompts)} sequences")


if __name__ == "__main__":
    main()
