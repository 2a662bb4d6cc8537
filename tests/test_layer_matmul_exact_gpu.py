"""Products whose result is known to the last bit: codes of few significant
bits and scales close together, so that no product loses a bit beside another
of its group and every sum is a whole number below 2^24 of a common unit. The
fp32 result is that sum, the bf16 result its rounding. Long rows, so that the
tiled kernels run many slabs of K (and their scale bytes' buffers many turns)."""
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
    """0, +-1, +-1.5, +-2, +-3 times 1 or 2: whole multiples of 1/2, at most 6."""
    x = torch.tensor([0.0, 1.0, 1.5, 2.0, 3.0, -1.0, -1.5, -2.0, -3.0], device="cuda")
    x = x[torch.randint(0, 9, (rows, k), generator=g, device="cuda")]
    s = torch.randint(127, 129, (rows, -(-k // block)), generator=g, device="cuda", dtype=torch.uint8)
    value = x * torch.exp2(s.float() - 127).repeat_interleave(block, 1)[:, :k]
    return x.to(ref.F8).view(torch.uint8), s, value


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("m,n,k", [
    (1, 300, 8192), (16, 8200, 4128), (50, 500, 4096),      # few rows, one and two column tiles
    (100, 1000, 8192 + 96), (333, 4099, 1568),              # tiles of 64, K split and not
    (1024, 2300, 4096 + 32), (1500, 3000, 4096),            # tiles of 128, four and two buffers
    (4096, 4096, 4096), (4099, 4096, 1568), (3900, 4000, 8192 + 224)])  # tiles of 256, last rows apart
def test_exact_products(m, n, k, block, dtype):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    a, sa, av = operand(m, k, block, g)
    b, sb, bv = operand(n, k, block, g)
    assert 4 * 36 * k < 1 << 24  # in units of 1/4
    # whole numbers in 64 bits: exact in any order
    want = torch.mm(av.double(), bv.double().t().contiguous()).to(dtype)
    got = mx.matmul_mxfp8(a, sa, b, sb, dtype, block)
    assert torch.equal(got, want), int((got != want).sum())
