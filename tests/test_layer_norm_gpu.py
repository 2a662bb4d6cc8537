"""RMS norm with MXFP8 output, its gradient, and the quantizer with blocks of
32 or 128 along rows and columns, against 64-bit forms."""
import math

import pytest
import torch

import layer_reference as ref
import microscaling_fp4_block_mx_amd as mx

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
# fp32 sum of squares: chains of at most 64 positive terms and a tree, below
# 2^-17 relative; its root halves that, and the products add a few 2^-24
Y_ERR = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check_codes(codes, scales, y, block, label):
    """codes x scales are y (float64) rounded once, up to y's own fp32 error:
    off by at most half a step and Y_ERR; the byte follows the largest |y|
    except within Y_ERR of a power of two."""
    rows, k = y.shape
    nb = -(-k // block)
    assert tuple(scales.shape) == (rows, nb), label
    yp = torch.nn.functional.pad(y, (0, nb * block - k)).view(rows, nb, block)
    amax = yp.abs().amax(2)
    lo, hi = ref.scale_byte(amax * (1 - Y_ERR)), ref.scale_byte(amax * (1 + Y_ERR))
    got = scales.double()
    assert bool(((got >= lo) & (got <= hi)).all()), label
    u = y / ref.pow2(ref.spread(got, block, k))
    _, e = torch.frexp(u.abs() * (1 + Y_ERR))
    step = torch.ldexp(torch.ones_like(u), (e - 1).clamp(min=-6) - 3)
    got_u = codes.view(ref.F8).double()
    target = u.clamp(-448, 448)
    off = (got_u - target).abs()
    assert bool((off <= step / 2 + 2 * Y_ERR * u.abs()).all()), (label, float((off / step).max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 32), (1, 96), (3, 160), (5, 512), (2, 1568), (7, 4096),
                                    (513, 992), (600, 4128), (3, 16384 + 32), (2, 65536)])
@pytest.mark.parametrize("block", [32, 128])
def test_norm(rows, k, block, dtype):
    g = gen(rows * 7 + k)
    x = torch.randn(rows, k, generator=g).to(DT[dtype])
    r = (torch.randn(rows, k, generator=g) * 3).to(DT[dtype])
    w = (torch.randn(k, generator=g) * 0.3 + 1).to(DT[dtype])
    for res in (None, r):
        print(rows, k, block, dtype, res is not None, flush=True)
        c, s, h = mx.rmsnorm_mxfp8(x.cuda(), w.cuda(), EPS, None if res is None else res.cuda(), block)
        wh, wy = ref.norm(x, w, EPS, res)
        check_codes(c.cpu(), s.cpu(), wy, block, (rows, k, block, dtype))
        if res is None:
            assert h is None
        else:
            assert torch.equal(h.cpu(), (x.float() + res.float()).to(DT[dtype]))


def test_norm_in_place_and_leading_dimensions():
    g = gen(1)
    x = torch.randn(2, 3, 256, generator=g).bfloat16().cuda()
    r = torch.randn(2, 3, 256, generator=g).bfloat16().cuda()
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    c0, s0, h0 = mx.rmsnorm_mxfp8(x, w, EPS, r)
    assert tuple(c0.shape) == (2, 3, 256) and tuple(s0.shape) == (2, 3, 2)
    for which in (0, 1):
        a, b = x.clone(), r.clone()
        out = (a, b)[which]
        c, s, h = mx.rmsnorm_mxfp8(a, w, EPS, b, out_h=out)
        assert h is out and torch.equal(out, h0) and torch.equal(c, c0) and torch.equal(s, s0)


def test_norm_special_rows():
    """Zeros, a NaN, an infinity, tiny and huge rows, each beside an ordinary one."""
    x = torch.ones(6, 128)
    x[0] = 0
    x[1, 5] = math.nan
    x[2, 7] = math.inf
    x[3] = 1e-30
    x[4] = 1e15
    w = torch.ones(128)
    c, s, _ = mx.rmsnorm_mxfp8(x.cuda(), w.cuda(), EPS, block=32)
    c, s = c.cpu(), s.cpu()
    assert bool((c[0] == 0).all() and (s[0] == 0).all())
    # NaN spreads over its whole row; next to an infinity every finite y is 0
    assert bool((s[1] == 255).all())
    assert int(s[2, 0]) == 255 and bool((s[2, 1:] == 0).all())
    _, y = ref.norm(x, w, EPS)
    check_codes(c[3:], s[3:], y[3:], 32, "special")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 160), (17, 1568), (700, 512), (2100, 4096),
                                    (5, 16384 + 64), (3, 65536)])
def test_norm_backward(rows, k, dtype):
    g = gen(rows + k)
    h = (torch.randn(rows, k, generator=g) * 2).to(DT[dtype])
    dy = torch.randn(rows, k, generator=g).to(DT[dtype])
    t = torch.randn(rows, k, generator=g).to(DT[dtype])
    w = (torch.randn(k, generator=g) * 0.3 + 1).to(DT[dtype])
    for through in (None, t):
        dx, dw = mx.rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), EPS,
                                     None if through is None else through.cuda())
        wx, ww = ref.norm_backward(dy, h, w, EPS, through)
        s = 1.0 / torch.sqrt(h.double().square().mean(1, keepdim=True) + EPS)
        gw = (w.double() * dy.double()).abs()
        # fp32: each term to 2^-16 of the magnitudes summed; bf16 output: half a step
        size = s * (gw + h.double().abs() * s * s * (gw * h.double().abs()).mean(1, keepdim=True))
        if through is not None:
            size = size + through.double().abs()
        tol = Y_ERR * size + (2.0 ** -8 * wx.abs() if dtype == "bf16" else 0.0)
        assert bool(((dx.cpu().double() - wx).abs() <= tol).all())
        sw = (dy.double() * h.double() * s).abs().sum(0)
        assert bool(((dw.cpu().double() - ww).abs() <= Y_ERR * sw).all())


def test_norm_backward_against_differences():
    """Central differences of sum(dy y) + sum(through h) in 64 bits."""
    g = gen(9)
    h = torch.randn(3, 64, generator=g)
    dy = torch.randn(3, 64, generator=g)
    t = torch.randn(3, 64, generator=g)
    w = torch.randn(64, generator=g) + 1
    dx, dw = mx.rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), EPS, t.cuda())

    def loss(hh, ww):
        _, y = ref.norm(hh, ww, EPS)
        return float((y * dy.double()).sum() + (hh.double() * t.double()).sum())

    e = 1e-5
    for i, j in ((0, 0), (0, 63), (1, 17), (2, 40)):
        a, b = h.double().clone(), h.double().clone()
        a[i, j] += e
        b[i, j] -= e
        want = (loss(a, w) - loss(b, w)) / (2 * e)
        assert abs(float(dx[i, j]) - want) <= 2e-4 * max(1.0, abs(want))
    for j in (0, 31, 63):
        a, b = w.double().clone(), w.double().clone()
        a[j] += e
        b[j] -= e
        want = (loss(h, a) - loss(h, b)) / (2 * e)
        assert abs(float(dw[j]) - want) <= 2e-4 * max(1.0, abs(want))


def test_norm_backward_in_place_and_empty():
    g = gen(3)
    h, dy, t = (torch.randn(50, 256, generator=g).bfloat16().cuda() for _ in range(3))
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    dx, dw = mx.rmsnorm_backward(dy, h, w, EPS, t)
    lib, n = mx.load_library(), mx.mx_rmsnorm_backward_workspace_size(50, 256)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    for which in range(3):
        bufs = [dy.clone(), h.clone(), t.clone()]
        out = torch.empty(256, device="cuda")
        assert lib.mx_rmsnorm_backward(bufs[0].data_ptr(), bufs[1].data_ptr(), w.data_ptr(),
                                       bufs[2].data_ptr(), mx.MX_BF16, 50, 256, EPS,
                                       bufs[which].data_ptr(), out.data_ptr(), ws.data_ptr(), n,
                                       st) == mx.MX_OK
        assert torch.equal(bufs[which], dx) and torch.equal(out, dw)
    dx0, dw0 = mx.rmsnorm_backward(dy[:0], h[:0], w, EPS)
    assert dx0.numel() == 0 and bool((dw0 == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 32), (31, 64), (33, 160), (128, 128), (129, 384),
                                    (300, 1568), (5, 4096)])
@pytest.mark.parametrize("block", [32, 128])
def test_quantize_both(rows, k, block, dtype):
    g = gen(rows * k)
    x = (torch.randn(rows, k, generator=g) * torch.exp(torch.randn(rows, k, generator=g) * 3))
    x[0, :3] = torch.tensor([0.0, -0.0, 448.0])
    x = x.to(DT[dtype])
    c, s, ct, st = (t.cpu() for t in mx.quantize_mxfp8_both(x.cuda(), block))
    wc, ws = ref.quantize(x.double(), block)
    assert torch.equal(s, ws) and torch.equal(c, wc)
    padded = -(-rows // 32) * 32
    xt = torch.nn.functional.pad(x.double().t(), (0, padded - rows))
    wc, ws = ref.quantize(xt, block)
    assert tuple(ct.shape) == (k, padded) and tuple(st.shape) == (k, -(-rows // block))
    assert torch.equal(st, ws) and torch.equal(ct, wc)
    c1, s1 = mx.quantize_mxfp8_rows(x.cuda(), block)
    c2, s2 = mx.quantize_mxfp8_columns(x.cuda(), block)
    assert torch.equal(c1.cpu(), c) and torch.equal(s1.cpu(), s)
    assert torch.equal(c2.cpu(), ct) and torch.equal(s2.cpu(), st)
    if block == 32:
        c3, s3 = mx.quantize_mxfp8(x.cuda())
        assert torch.equal(c3.cpu(), c) and torch.equal(s3.cpu(), s)


def test_quantize_nonfinite_blocks():
    x = torch.randn(256, 256, generator=gen(4))
    x[3, 130] = math.nan
    x[200, 5] = -math.inf
    for block in (32, 128):
        c, s, ct, st = (t.cpu() for t in mx.quantize_mxfp8_both(x.cuda(), block))
        wc, ws = ref.quantize(x.double(), block)
        assert torch.equal(s, ws) and torch.equal(c, wc)
        wc, ws = ref.quantize(x.double().t().contiguous(), block)
        assert torch.equal(st, ws) and torch.equal(ct, wc)
