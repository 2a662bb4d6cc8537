"""Rows and elements past what 32 bits count: the norm with more rows than one
dimension of a grid holds, and a product whose output has more than 2^31
elements, on rows from the start, the end and between: the norm bit for bit
against calls of few rows, the product against 64 bits."""
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
    x = torch.randn(rows, k, device="cuda", dtype=torch.bfloat16)
    w = (torch.randn(k, device="cuda") * 0.1 + 1).to(torch.bfloat16)
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
    a = torch.randint(0, 0x7E, (m, k), device="cuda", dtype=torch.uint8)
    b = torch.randint(0, 0x7E, (n, k), device="cuda", dtype=torch.uint8)
    sa = torch.randint(120, 124, (m, 1), device="cuda", dtype=torch.uint8)
    sb = torch.randint(120, 124, (n, 1), device="cuda", dtype=torch.uint8)
    c = mx.matmul_mxfp8(a, sa, b, sb, block=32)

    def value(codes, scales):
        return codes.cpu().view(torch.float8_e4m3fn).double() * torch.exp2(scales.cpu().double() - 127)

    bv = value(b, sb)
    for at in (0, 23000, m - 8):
        want = value(a[at:at + 8], sa[at:at + 8]) @ bv.t()
        # all terms are positive: bf16's rounding, 2^-8, and what the matrix core drops, 2^-13
        assert bool(((c[at:at + 8].cpu().double() - want).abs() <= (2.0 ** -8 + 2.0 ** -12) * want).all())
