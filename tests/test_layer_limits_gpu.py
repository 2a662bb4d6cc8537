"""Launches whose workgroups, times their threads, are more than one dimension
of a grid counts (2^32)."""
import pytest
import torch

import microscaling_fp4_block_mx_amd as mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_product_of_a_row_and_very_many():
    """2^28 + 33 columns (8.6 GB of codes): bit for bit what calls with few of them give."""
    n, k = (1 << 28) + 33, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randint(0, 0x7E, (2, k), generator=g, device="cuda", dtype=torch.uint8)
    sa = torch.randint(120, 124, (2, 1), generator=g, device="cuda", dtype=torch.uint8)
    b = torch.empty((n, k), dtype=torch.uint8, device="cuda")
    for at in range(0, n, 1 << 26):
        b[at:at + (1 << 26)].random_(0, 0x7E, generator=g)
    sb = torch.randint(120, 124, (n, 1), generator=g, device="cuda", dtype=torch.uint8)
    c = mx.matmul_mxfp8(a, sa, b, sb, block=32)
    for at in (0, (1 << 27) - 8, (1 << 28) - 8, n - 24):
        part = slice(at, at + 24)
        assert torch.equal(c[:, part], mx.matmul_mxfp8(a, sa, b[part].clone(), sb[part].clone(), block=32)), at
    # every column has been written: sums of products of positive numbers, hardly any of them 0
    assert float((c[:, ::509] > 0).float().mean()) > 0.99


def test_tiles_past_the_limit_are_refused():
    """Fails before any HIP call: the addresses are not used."""
    A, B, C, D, E = (i << 44 for i in range(1, 6))
    for m, n in ((17, 2 ** 31 - 1), (2 ** 31 - 1, 65), (1 << 20, 1 << 20)):
        assert mx.mx_matmul_mxfp8(A, B, C, D, m, n, 32, 32, mx.MX_BF16, E, None, 0, None) == mx.MX_ERR_SHAPE
    # the checks behind the shape's: two rows are fine, operands that overlap are not
    assert mx.mx_matmul_mxfp8(A, B, C, D, 2, 2 ** 31 - 256, 32, 32, mx.MX_BF16, A, None, 0,
                              None) == mx.MX_ERR_ALIAS


def test_append_to_three_of_very_many_sequences():
    """2^24 sequences, all but three of them idle."""
    batch, heads, dim, page = 1 << 24, 8, 64, 32
    at = [5, batch // 2, batch - 1]
    cache, few = mx.kv_cache(4, heads, dim, page), mx.kv_cache(4, heads, dim, page)
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(3, heads, dim, generator=g, device="cuda").bfloat16() for _ in "kv")
    new = torch.zeros(batch, dtype=torch.int32, device="cuda")
    new[at] = 1
    cu = torch.nn.functional.pad(new.cumsum(0, dtype=torch.int32), (1, 0))
    table = torch.full((batch, 1), 3, dtype=torch.int32, device="cuda")
    table[at] = torch.tensor([[2], [0], [1]], dtype=torch.int32, device="cuda")
    held = torch.zeros(batch, dtype=torch.int32, device="cuda")
    mx.kv_append(cache, k, v, table, cu, held)
    mx.kv_append(few, k, v, table[at], torch.arange(4, dtype=torch.int32, device="cuda"), held[:3])
    for a, b in zip(cache, few):
        assert torch.equal(a, b)


@pytest.mark.parametrize("heads,group", [(1, 1), (16, 33)])
def test_attention_over_very_many_sequences(heads, group):
    """2^24 sequences of one token that share two pages (the few-rows kernel),
    and 2^20 with 16 kv heads, all but four of them idle, whose queries are
    more than that kernel takes to a kv head: what a call of four gives."""
    batch, dim, page, kinds = (1 << 24) // heads, 64, 32, 4
    cache = mx.kv_cache(2, heads, dim, page)
    g = torch.Generator(device="cuda").manual_seed(5)
    i32 = dict(dtype=torch.int32, device="cuda")
    k, v = (torch.randn(64, heads, dim, generator=g, device="cuda").bfloat16() for _ in "kv")
    mx.kv_append(cache, k, v, torch.tensor([[1, 0]], **i32), torch.tensor([0, 64], **i32),
                 torch.zeros(1, **i32))
    q = torch.randn(kinds, heads * group, dim, generator=g, device="cuda").bfloat16()
    lengths = torch.tensor([64, 1, 33, 50], **i32)
    table = torch.tensor([[1, 0]], **i32).repeat(kinds, 1)
    cu = torch.arange(kinds + 1, **i32)
    want = mx.kv_attention(q, cache, table, cu, lengths)
    assert bool(torch.isfinite(want).all())
    times = batch // kinds
    if group == 1:
        got = mx.kv_attention(q.repeat(times, 1, 1), cache, table.repeat(times, 1),
                              torch.arange(batch + 1, **i32), lengths.repeat(times))
        assert bool((got.view(times, *want.shape) == want).all())
    else:
        many = torch.full((batch + 1,), kinds, **i32)
        many[:kinds + 1] = cu
        got = mx.kv_attention(q, cache, table.repeat(times, 1), many, lengths.repeat(times))
        assert torch.equal(got, want)
