"""The helpers look at shapes, not at element counts alone."""
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


def test_transposed_operands_are_refused():
    u8 = dict(dtype=torch.uint8, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    a, sa = torch.zeros(6, 512, **u8), torch.zeros(6, 4, **u8)
    b, sb = torch.zeros(10, 512, **u8), torch.zeros(10, 4, **u8)
    x, w = torch.zeros(6, 512, **bf), torch.ones(512, **bf)
    t = torch.zeros(512, 6, **bf)
    cache = mx.kv_cache(4, 2, 64, 32)
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4, 64, **bf)
    bad = [
        lambda: mx.matmul_mxfp8(a, sa.view(4, 6), b, sb),              # [blocks, rows]
        lambda: mx.matmul_mxfp8(a, sa, b, sb.view(4, 10)),
        lambda: mx.matmul_mxfp8(a, sa, b, sb, out=torch.empty(10, 6, **bf)),
        lambda: mx.rmsnorm_mxfp8(x, w, residual=t),
        lambda: mx.rmsnorm_mxfp8(x, w, residual=x, out_h=torch.empty_like(t)),
        lambda: mx.rmsnorm_mxfp8(x, w.view(8, 64)),
        lambda: mx.rmsnorm_backward(t, x, w),
        lambda: mx.rmsnorm_backward(x, x, w, through=t),
        lambda: mx.kv_attention(q, cache._replace(k_scales=torch.zeros(2, 4, **u8)), table, i, i[:1]),
        lambda: mx.kv_attention(q, cache, table, i, i[:1], out=torch.empty(64, 4, 1, **bf)),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    torch.cuda.synchronize()


def test_other_leading_dimensions_are_fine():
    """The last dimension decides; a flat tensor of the right length is taken as its rows."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 3, 512, generator=g, device="cuda").bfloat16()
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    c, s, h = mx.rmsnorm_mxfp8(x, w, residual=x)
    c2, s2, h2 = mx.rmsnorm_mxfp8(x, w, residual=x.view(6, 512), out_h=torch.empty(6, 512, dtype=x.dtype, device="cuda"))
    assert torch.equal(c, c2) and torch.equal(s, s2) and torch.equal(h.view(6, 512), h2)
    y = mx.matmul_mxfp8(c, s, c.view(6, 512), s.view(6, 4))
    for scales in (s, s.view(6, 4), s.view(-1)):
        assert torch.equal(mx.matmul_mxfp8(c.view(6, 512), scales, c.view(6, 512), s.view(6, 4)).view(2, 3, 6), y)
    out = torch.empty(6, 6, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(mx.matmul_mxfp8(c, s, c.view(6, 512), s.view(6, 4), out=out).view(2, 3, 6), y)
