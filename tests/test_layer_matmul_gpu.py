"""Products of MXFP8 matrices against 64 bits: both outputs, both blocks, every
kernel the sizes choose between, odd sizes, short last blocks, NaN."""
import math

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


def operand(rows, k, block, g):
    nb = -(-k // block)
    x = (torch.randn(rows, k, generator=g) * 100).clamp(-448, 448)
    return (x.to(ref.F8).view(torch.uint8),
            torch.randint(118, 124, (rows, nb), generator=g, dtype=torch.uint8))


def bound(want, size, k, dtype):
    """bf16: half a step, and per group of eight products at most seven that
    lose less than 2^-13 of the largest. f32: one rounding per addition."""
    if dtype == torch.bfloat16:
        return 2.0 ** -8 * want.abs() + 2.0 ** -10 * size
    return (k + 2) * 2.0 ** -24 * size


def check(m, n, k, block, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + m * 31 + n * 7 + k)
    (a, sa), (b, sb) = operand(m, k, block, g), operand(n, k, block, g)
    print(m, n, k, block, dtype, flush=True)
    got = mx.matmul_mxfp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), dtype, block).cpu()
    av, bv = ref.dequantize(a, sa, block), ref.dequantize(b, sb, block)
    want, size = av @ bv.t(), av.abs() @ bv.abs().t()
    assert got.dtype == dtype and tuple(got.shape) == (m, n)
    off = (got.double() - want).abs()
    assert bool((off <= bound(want, size, k, dtype)).all()), float((off / size).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 32), (1, 17, 96), (1, 64, 4096), (3, 100, 160), (16, 33, 1568), (17, 64, 1024),
    (32, 15, 544), (33, 48, 512), (64, 129, 2080), (65, 64, 128), (100, 200, 32), (130, 70, 672),
    (257, 129, 1024), (333, 515, 1568), (80, 96, 8192 + 32), (1024, 300, 416)])
def test_product(m, n, k, block, dtype):
    check(m, n, k, block, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("m,n,k", [(2000, 2050, 160), (2049, 1800, 672), (4100, 4000, 96),
                                   (3585, 4097, 544)])
def test_product_large_tiles(m, n, k, block, dtype):
    check(m, n, k, block, dtype)


@pytest.mark.parametrize("m", [2, 40, 200, 4000])
@pytest.mark.parametrize("block", [32, 128])
def test_nan_stays_in_its_row_and_column(m, block):
    n, k = 300, 416
    g = torch.Generator().manual_seed(m)
    (a, sa), (b, sb) = operand(m, k, block, g), operand(n, k, block, g)
    sa[1, -1] = 255          # the short last block of a row of A
    b[7, 11] = 0x7F          # a NaN code in B
    for dtype in (torch.bfloat16, torch.float32):
        got = mx.matmul_mxfp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), dtype, block).cpu()
        nan = torch.isnan(got)
        want = torch.zeros_like(nan)
        want[1] = True
        want[:, 7] = True
        assert torch.equal(nan, want)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_extreme_scales_and_zeros(m):
    """Rows of zeros, scale bytes at both ends of the range that cancel."""
    n, k = 130, 256
    g = torch.Generator().manual_seed(5)
    (a, sa), (b, sb) = operand(m, k, 128, g), operand(n, k, 128, g)
    sa[:, 0], sb[:, 0] = 20, 230
    sa[:, 1], sb[:, 1] = 230, 20
    a[0] = 0
    for dtype in (torch.bfloat16, torch.float32):
        got = mx.matmul_mxfp8(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), dtype, 128).cpu()
        av, bv = ref.dequantize(a, sa, 128), ref.dequantize(b, sb, 128)
        want, size = av @ bv.t(), av.abs() @ bv.abs().t()
        assert bool((got[0] == 0).all())
        assert bool(((got.double() - want).abs() <= bound(want, size, k, dtype)).all())


def test_same_bits_every_time_and_out():
    g = torch.Generator().manual_seed(1)
    (a, sa), (b, sb) = operand(100, 8192, 128, g), operand(200, 8192, 128, g)
    a, sa, b, sb = a.cuda(), sa.cuda(), b.cuda(), sb.cuda()
    assert mx.mx_matmul_mxfp8_workspace_size(100, 200, 8192, 128, mx.MX_BF16) > 0
    first = mx.matmul_mxfp8(a, sa, b, sb)
    out = torch.empty_like(first)
    for _ in range(3):
        assert mx.matmul_mxfp8(a, sa, b, sb, out=out) is out
        assert torch.equal(out, first)
    lead = mx.matmul_mxfp8(a.view(4, 25, 8192), sa.view(4, 25, 64), b, sb)
    assert tuple(lead.shape) == (4, 25, 200) and torch.equal(lead.view(100, 200), first)


def test_empty():
    u8 = dict(dtype=torch.uint8, device="cuda")
    a, sa = torch.empty(0, 64, **u8), torch.empty(0, 1, **u8)
    b, sb = torch.zeros(5, 64, **u8), torch.zeros(5, 1, **u8)
    assert tuple(mx.matmul_mxfp8(a, sa, b, sb).shape) == (0, 5)
    assert tuple(mx.matmul_mxfp8(b, sb, a, sa).shape) == (5, 0)


@pytest.mark.parametrize("m,n,k,block", [(50, 96, 160, 32), (300, 256, 416, 128), (33, 64, 96, 128)])
def test_linear_step_gradients(m, n, k, block):
    """y = Q(x) Q(w)^T, dx = Q(dy) Q(w^T)^T, dw = Q(dy^T) Q(x^T)^T, each equal
    to the product of what the quantizer's codes stand for; and dx, dw against
    differences of sum(dy y) in the unquantized matrices, within the
    quantizer's own error."""
    g = torch.Generator().manual_seed(m)
    x, w = torch.randn(m, k, generator=g).bfloat16(), (torch.randn(n, k, generator=g) * 0.1).bfloat16()
    dy = torch.randn(m, n, generator=g).bfloat16()
    qx, qw, qd = (mx.quantize_mxfp8_both(t.cuda(), block) for t in (x, w, dy))
    y = mx.matmul_mxfp8(qx[0], qx[1], qw[0], qw[1], torch.float32, block)
    dx = mx.matmul_mxfp8(qd[0], qd[1], qw[2], qw[3], torch.float32, block)
    dw = mx.matmul_mxfp8(qd[2], qd[3], qx[2], qx[3], torch.float32, block)

    def held(t):
        return ref.dequantize(*ref.quantize(t, block), block)

    xd, wd, dd = x.double(), w.double(), dy.double()
    for got, p, q, depth in ((y, held(xd), held(wd), k),
                             (dx, held(dd), held(wd.t().contiguous()), n),
                             (dw, held(dd.t().contiguous()), held(xd.t().contiguous()), m)):
        size = p.abs() @ q.abs().t()
        off = (got.cpu().double() - p @ q.t()).abs()
        assert bool((off <= (depth + 34) * 2.0 ** -24 * size).all())
    # sum(dy (x w^T)) is linear in x and in w: its differences are dy w and
    # dy^T x; an E4M3 operand is off by at most 2^-4 of itself (plus what falls
    # below the subnormal step, 2^-10 2^-8 of the block's largest)
    tiny = 2.0 ** -17
    for got, p, q in ((dx, dd, wd.t()), (dw, dd.t(), xd.t())):
        pe = 2.0 ** -4 * p.abs() + tiny * p.abs().max()
        qe = 2.0 ** -4 * q.abs() + tiny * q.abs().max()
        tol = pe @ q.abs().t() + p.abs() @ qe.t() + pe @ qe.t()
        assert bool(((got.cpu().double() - p @ q.t()).abs() <= tol).all())
