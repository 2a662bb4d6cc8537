"""fp32 products at both ends of the scale bytes that their widening to
bfloat16 is exact for, 3 to 246, and past them."""
import pytest
import torch

import layer_reference as ref
import microscaling_fp4_block_mx_amd as mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("m,n,k", [(3, 40, 416), (40, 300, 416), (300, 200, 672), (1500, 1700, 160)])
@pytest.mark.parametrize("low,high", [(3, 246), (246, 3), (3, 251 - 16)])
def test_ends_of_the_range(m, n, k, block, low, high):
    """Every code, subnormal ones among them; products and sums as in the other
    fp32 tests: one rounding per addition (and 2^-149 where a result is that small)."""
    g = torch.Generator().manual_seed(m)
    nb = -(-k // block)
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    a, b = (codes[torch.randint(0, len(codes), (r, k), generator=g)] for r in (m, n))
    sa, sb = torch.full((m, nb), low, dtype=torch.uint8), torch.full((n, nb), high, dtype=torch.uint8)
    got = mx.matmul_mxfp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), torch.float32, block).cpu().double()
    av, bv = ref.dequantize(a, sa, block), ref.dequantize(b, sb, block)
    want, size = av @ bv.t(), av.abs() @ bv.abs().t()
    assert bool(((got - want).abs() <= (k + 2) * 2.0 ** -24 * size + k * 2.0 ** -149).all())


@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("m,n,k", [(3, 40, 416), (40, 300, 1440), (100, 1000, 8192 + 96), (300, 200, 672),
                                   (1500, 1700, 672)])
def test_bytes_above_246(m, n, k, block):
    """Some rows' blocks have bytes up to 254, beside others from the bottom;
    B's are small, so that every result is finite. Bounds as above."""
    g = torch.Generator().manual_seed(m + 1)
    nb = -(-k // block)
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    a, b = (codes[torch.randint(0, len(codes), (r, k), generator=g)] for r in (m, n))
    sa = torch.randint(110, 130, (m, nb), generator=g, dtype=torch.uint8)
    sa[::5] = torch.randint(240, 255, (len(sa[::5]), nb), generator=g, dtype=torch.uint8)
    sa[1::7, -1] = 254
    sa[2::9] = torch.randint(3, 20, (len(sa[2::9]), nb), generator=g, dtype=torch.uint8)
    sb = torch.randint(3, 17, (n, nb), generator=g, dtype=torch.uint8)
    sa[m // 2, nb // 2] = 255  # NaN stays in its row
    got = mx.matmul_mxfp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), torch.float32, block).cpu().double()
    turned = mx.matmul_mxfp8(b.cuda(), sb.cuda(), a.cuda(), sa.cuda(), torch.float32, block).cpu().double()
    nan = torch.zeros(m, dtype=torch.bool)
    nan[m // 2] = True
    sa[m // 2] = 127
    av, bv = ref.dequantize(a, sa, block), ref.dequantize(b, sb, block)
    want, size = av @ bv.t(), av.abs() @ bv.abs().t()
    tol = (k + 2) * 2.0 ** -24 * size + k * 2.0 ** -149
    for c in (got, turned.t()):
        assert bool(torch.isnan(c[nan]).all()) and not bool(torch.isnan(c[~nan]).any())
        assert bool(((c - want).abs() <= tol)[~nan].all())
