"""Rows and elements past what 32 bits count: the norm with more rows than one
dimension of a grid holds, and a product whose output has more than 2^31
elements, on rows from the start, the end and between, bit for bit against
calls of few rows (which other tests hold against 64 bits)."""
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


def test_norm_of_many_rows():
    rows, k, eps = (1 << 26) + 4097, 32, 1e-6
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(rows, k, generator=g, device="cuda", dtype=torch.bfloat16)
    w = (torch.randn(k, generator=g, device="cuda") * 0.1 + 1).to(torch.bfloat16)
    codes, scales, h = mx.rmsnorm_mxfp8(x, w, eps, block=32)
    assert h is None
    for at in (0, (1 << 21) - 8, 1 << 21, 1 << 26, rows - 16):
        part = slice(at, at + 16)
        c, s, _ = mx.rmsnorm_mxfp8(x[part].contiguous(), w, eps, block=32)  # the same kernel, few rows
        assert torch.equal(codes[part], c) and torch.equal(scales[part], s), at
    # and every row has been written: no block of normal numbers has a byte of 0
    assert int(scales.min()) > 0


def test_product_with_a_large_output():
    m, n, k = 46400, 46336, 32
    assert m * n > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(7)
    a = torch.randint(0, 0x7E, (m, k), generator=g, device="cuda", dtype=torch.uint8)
    b = torch.randint(0, 0x7E, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    sa = torch.randint(120, 124, (m, 1), generator=g, device="cuda", dtype=torch.uint8)
    sb = torch.randint(120, 124, (n, 1), generator=g, device="cuda", dtype=torch.uint8)
    c = mx.matmul_mxfp8(a, sa, b, sb, block=32)
    # with k = 32 every kernel takes one matrix instruction per output: the same bits
    for at in (0, 23000, m - 8):
        few = mx.matmul_mxfp8(a[at:at + 8].clone(), sa[at:at + 8].clone(), b, sb, block=32)
        assert torch.equal(c[at:at + 8], few), at
    # and every output has been written: a sum of products of positive numbers, few of them 0
    assert float((c[::997] > 0).float().mean()) > 0.99
