"""The decoder layer of examples/ against the same layer in 64 bits: prompts and
single tokens through one cache, and a training step's gradients.

Tolerances. An 8-bit rounding moves a value by at most 2^-4 of itself (its
relative step), so a vector by at most 2^-4 of its norm. On the way from h to
the layer's update there are six in a row (norm, cache, attention's output,
norm, gate, and the values' or keys' share of attention, counted as one more
than the cache's): 6 / 16 of the norm, the largest. A wrong head, page or
order gives about 1.4. In the training step each gradient's product has two
rounded operands: 2 / 16, and dx passes the norm's gradient, which is linear in
it; the loss's own dy differs by y's error, which is 2 / 16 of y's norm."""
import pytest
import torch
import torch.nn.functional as F

import microscaling_fp4_block_mx_amd as mx
from examples import decoder_layer as ex

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


def value(codes, scales, block):
    s = torch.exp2(scales.cpu().double() - 127).repeat_interleave(block, 1)[:, :codes.shape[1]]
    return codes.cpu().view(torch.float8_e4m3fn).double() * s


def norm(x, w):
    return w * x / torch.sqrt(x.square().mean(-1, keepdim=True) + ex.EPS)


class Plain:
    """The layer in 64 bits with the quantized weights' values, one sequence at a time."""

    def __init__(self, layer, batch):
        self.l = layer
        self.w = {n: value(*getattr(layer, n), layer.block) for n in ("qkv", "o", "gate_up", "down")}
        self.seen = [None] * batch

    def __call__(self, h, new):
        out, at = [], 0
        for i, n in enumerate(new):
            out.append(self.sequence(h[at:at + n].cpu().double(), i))
            at += n
        return torch.cat(out)

    def sequence(self, h, i):
        l = self.l
        qkv = (norm(h, 1.0) @ self.w["qkv"].t()).view(h.shape[0], -1, l.dim)
        q, k, v = qkv.split([l.heads, l.kv_heads, l.kv_heads], 1)
        if self.seen[i] is not None:
            k, v = torch.cat([self.seen[i][0], k]), torch.cat([self.seen[i][1], v])
        self.seen[i] = k, v
        group = l.heads // l.kv_heads
        kk, vv = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        z = torch.einsum("qhd,khd->hqk", q, kk) / l.dim ** 0.5
        past = k.shape[0] - q.shape[0]
        hide = torch.ones(q.shape[0], k.shape[0], dtype=torch.bool).triu(past + 1)
        o = torch.einsum("hqk,khd->qhd", z.masked_fill(hide, -torch.inf).softmax(-1), vv)
        h = h + o.reshape(h.shape[0], -1) @ self.w["o"].t()
        gate, up = (norm(h, 1.0) @ self.w["gate_up"].t()).chunk(2, -1)
        return (F.silu(gate) * up) @ self.w["down"].t()


@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("page", [32, 64])
def test_serving(block, page):
    layer = ex.DecoderLayer(hidden=512, heads=8, kv_heads=2, dim=64, ffn=768, block=block, seed=3)
    prompts, steps = [131, 1, 40, 64], 4
    plain = Plain(layer, len(prompts))
    for i, (h, (stream, update)) in enumerate(ex.serve(layer, prompts, steps, page)):
        want = plain(h, prompts if i == 0 else [1] * len(prompts))
        assert update.shape == h.shape and stream.shape == h.shape
        off = (update.cpu().double() - want).norm(dim=1) / want.norm(dim=1)
        assert float(off.max()) <= 6 / 16, (i, float(off.max()))


def test_layers_in_a_row():
    """The second layer's norm adds the first one's update to the stream."""
    layer = ex.DecoderLayer(hidden=256, heads=4, kv_heads=4, dim=64, ffn=512, seed=4)
    pages = ex.Pages(1, 20, 32)
    cache = mx.kv_cache(pages.width, 4, 64, 32)
    cu, held, lengths = pages.step([20])
    g = torch.Generator(device="cuda").manual_seed(8)
    h = torch.randn(20, 256, generator=g, device="cuda").to(torch.bfloat16)
    stream, update = layer(h, None, cache, pages.table, cu, held, lengths)
    a, b = layer(stream, update, cache, pages.table, cu, held, lengths)
    one = (stream.float() + update.float()).to(torch.bfloat16)
    c, d = layer(one, None, cache, pages.table, cu, held, lengths)
    # the sum is rounded to bfloat16 in the second form before the norm, not in the first
    for got, want in ((a, c), (b, d)):
        assert float((got.float() - want.float()).norm() / want.float().norm()) <= 2 / 16


def test_training_step():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(333, 256, generator=g).to(torch.bfloat16)
    w = (torch.randn(192, 256, generator=g) * 0.05).to(torch.bfloat16)
    gain = (torch.randn(256, generator=g) * 0.1 + 1).to(torch.bfloat16)
    target = torch.randn(333, 192, generator=g)
    loss, dx, dgain, dw = ex.train_step(x.cuda(), gain.cuda(), w.cuda(), target.cuda())
    xx, gg, ww = (t.double().requires_grad_() for t in (x, gain, w))
    y = norm(xx, gg) @ ww.t()
    want = F.mse_loss(y, target.double())
    want.backward()
    assert abs(loss.item() - want.item()) <= 4 / 16 * want.item()
    # dy is off by y's error, at most 2 / 16 |y| <= 2 / 16 of |dy| here (|y| < |y - target|)
    assert float(y.detach().norm()) < float((y.detach() - target).norm())
    for got, ref in ((dx, xx.grad), (dgain, gg.grad), (dw, ww.grad)):
        assert float((got.cpu().double() - ref).norm() / ref.norm()) <= 4 / 16
    # a step against the gradient lowers the loss
    w2 = (w.cuda().float() - 20.0 * dw).to(torch.bfloat16)
    assert ex.train_step(x.cuda(), gain.cuda(), w2, target.cuda())[0].item() < loss.item()


def test_example_runs(capsys):
    ex.main()
    lines = capsys.readouterr().out.splitlines()
    losses = [float(line.split()[-1]) for line in lines if line.startswith("step")]
    assert len(losses) == 5 and losses == sorted(losses, reverse=True)
