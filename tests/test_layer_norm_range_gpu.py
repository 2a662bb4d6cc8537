"""The norm and its gradient on rows whose squares leave the range of 32 bits:
large ones, and with eps = 0 small ones."""
import math

import pytest
import torch

import layer_reference as ref
import microscaling_fp4_block_mx_amd as mx
from test_layer_norm_gpu import DT, Y_ERR, check_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


SIZES = [1e18, 3e19, 1e25, 1e37]
SMALL = [1e-18, 1e-20, 1e-25, 1e-36]


def rows_of(k, sizes, seed):
    """Normal rows of these sizes, an ordinary one between any two."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2 * len(sizes), k, generator=g)
    for i, s in enumerate(sizes):
        x[2 * i] *= s
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [32, 160, 4096, 16384 + 32])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_norm_of_large_and_small_rows(k, eps, dtype):
    x = rows_of(k, SIZES + (SMALL if eps == 0.0 else []), k).to(DT[dtype])
    w = (torch.randn(k, generator=torch.Generator().manual_seed(1)) * 0.3 + 1).to(DT[dtype])
    r = (x * 0.25).contiguous()
    for res in (None, r):
        for reps in (1, 200):  # one item a thread, and four
            a = x.repeat(reps, 1).cuda()
            b = None if res is None else res.repeat(reps, 1).cuda()
            c, s, _ = mx.rmsnorm_mxfp8(a, w.cuda(), eps, b, 32)
            n = x.shape[0]
            for at in (0, n * (reps - 1)):
                _, y = ref.norm(x, w, eps, res)
                check_codes(c[at:at + n].cpu(), s[at:at + n].cpu(), y, 32, (k, eps, dtype))


def test_non_finite_rows_stay_as_they_were():
    x = torch.ones(5, 64)
    x[0, 3], x[1, 3], x[2], x[3, 5] = math.inf, math.nan, 3e38, 3e38
    c, s, _ = mx.rmsnorm_mxfp8(x.cuda(), torch.ones(64, device="cuda"), 1e-6, block=32)
    s = s.cpu().tolist()
    assert s[0] == [255, 0] and s[1] == [255, 255] and 255 not in s[2] + s[3] + s[4]
    # a row of zeros without eps: 0 / 0
    c, s, _ = mx.rmsnorm_mxfp8(torch.zeros(1, 64, device="cuda"), torch.ones(64, device="cuda"), 0.0, block=32)
    assert s.cpu().tolist() == [[255, 255]]
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [32, 160, 4096, 16384 + 32])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_gradient_of_large_and_small_rows(k, eps, dtype):
    h = rows_of(k, SIZES[:3] + (SMALL if eps == 0.0 else []), k).to(DT[dtype])
    g = torch.Generator().manual_seed(2)
    # gradients as large as the row, so that dx is of ordinary size (and its
    # products are not): a gradient that meets a norm's large input is scaled back
    size = h.float().abs().amax(1, keepdim=True)
    dy = (torch.randn(h.shape, generator=g) * size.clamp(max=1e15)).to(DT[dtype])
    t = torch.randn(h.shape, generator=g).to(DT[dtype])
    w = (torch.randn(k, generator=g) * 0.3 + 1).to(DT[dtype])
    for through in (None, t):
        dx, dw = mx.rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), eps,
                                     None if through is None else through.cuda())
        wx, ww = ref.norm_backward(dy, h, w, eps, through)
        s = 1.0 / torch.sqrt(h.double().square().mean(1, keepdim=True) + eps)
        gw = (w.double() * dy.double()).abs()
        mag = s * (gw + h.double().abs() * s * s * (gw * h.double().abs()).mean(1, keepdim=True))
        if through is not None:
            mag = mag + through.double().abs()
        tol = Y_ERR * mag + (2.0 ** -8 * wx.abs() if dtype == "bf16" else 0.0) + 2.0 ** -126
        assert bool(((dx.cpu().double() - wx).abs() <= tol).all())
        sw = (dy.double() * h.double() * s).abs().sum(0)
        assert bool(((dw.cpu().double() - ww).abs() <= Y_ERR * sw + 2.0 ** -126).all())


