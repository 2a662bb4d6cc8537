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
