"""Scratch of the split attention: what the size query gives for a bound on the
lengths is enough for every call that may be made with that bound, whatever
room the page table has (the call plans for the shorter of the two)."""
import ctypes
import math

import pytest
import torch

import microscaling_fp4_block_mx_amd as mx

SHAPES = [(16, 16, 32, 8, 128), (1, 1, 8, 8, 64), (4, 4, 32, 8, 128), (300, 1, 8, 2, 64),
          (520, 1, 32, 8, 128), (64, 64, 64, 8, 128), (7, 3, 12, 1, 64)]


@pytest.mark.parametrize("tokens,batch,q_heads,heads,dim", SHAPES)
def test_size_covers_every_shorter_length(tokens, batch, q_heads, heads, dim):
    def size(length):
        return mx.mx_kv_attention_workspace_size(tokens, batch, q_heads, heads, dim, length)

    lengths = sorted({1 + i * 128 for i in range(1200)} | {1 << i for i in range(31)} | {2 ** 31 - 1})
    most = 0
    for length in lengths:
        now = size(length)
        assert now >= most, length
        most = now
    assert size(0) >= most  # no bound: whatever the table has room for


@pytest.mark.gpu
@pytest.mark.parametrize("bound", [0, 16384, 16640, 1 << 20])
def test_c_call_with_the_size_it_was_told(bound):
    """The C entry points with the structures of include/mx.h, a bound of 0
    and bounds past the table's room (16,384 tokens)."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    batch, heads, q_heads, dim, page, width = 16, 8, 32, 128, 64, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = mx.kv_cache(width, heads, dim, page)
    order = torch.randperm(width, generator=g, device="cuda").to(torch.int32)
    cu = torch.tensor([0, width * page], dtype=torch.int32, device="cuda")
    held = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(width * page, heads, dim, generator=g, device="cuda").bfloat16() for _ in "kv")
    mx.kv_append(cache, k, v, order.view(1, -1), cu, held)
    table = order.repeat(batch, 1)  # every sequence reads the same pages
    cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([1 + i * 1092 for i in range(batch - 1)] + [width * page],
                           dtype=torch.int32, device="cuda")
    q = torch.randn(batch, q_heads, dim, generator=g, device="cuda").bfloat16()
    want = mx.kv_attention(q, cache, table, cu, lengths)

    c = mx.MxKVCache(*(t.data_ptr() for t in cache), width, heads, dim, page)
    b = mx.MxKVBatch(table.data_ptr(), cu.data_ptr(), lengths.data_ptr(), batch, batch, width)
    size = mx.mx_kv_attention_workspace_size(batch, batch, q_heads, heads, dim, bound)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    status = mx.mx_kv_attention(q.data_ptr(), q_heads * dim, q_heads, ctypes.byref(c), ctypes.byref(b),
                                bound, 1.0 / math.sqrt(dim), out.data_ptr(),
                                ws.data_ptr() if size else None, size,
                                torch.cuda.current_stream().cuda_stream)
    assert status == mx.MX_OK
    torch.cuda.synchronize()
    assert torch.equal(out, want)
