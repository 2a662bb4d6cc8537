"""Attention's accuracy where one bound on everything would hide it: weights
many powers of two below the largest, scores too large for a weight's exponent,
small elements of q beside large ones, a channel that dominates a score."""
import math

import pytest
import torch

import layer_reference as ref
import microscaling_fp4_block_mx_amd as mx
from test_layer_kv_gpu import World, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


def world_of(k, v, page=64):
    """A cache that holds these keys and values [tokens, heads, dim] as one sequence."""
    tokens, heads, dim = k.shape
    w = World([tokens], heads, dim, page, 1)
    cu, held = i32([0, tokens]), i32([0])
    ref.append(w.cpu, k, v, w.table, cu, held)
    mx.kv_append(w.gpu, k.cuda(), v.cuda(), w.table.cuda(), cu.cuda(), held.cuda())
    w.same()
    return w


@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("below", [0, 6, 10, 13, 15, 17, 20, 22, 24, 28])
def test_a_long_flat_tail(new, dim, below):
    """One key takes (nearly) all, 999 keys share what is left evenly, each with a
    weight of 2^-below of the first one's; they alone carry dims 2 and up.
    All scores and values are exact, so a weight is off by its rounding (2^-8 of
    itself as the header states it), its sum by the same, sums of 1,000 terms in
    32 bits by 2^-14, the result by 2^-9: 2^-6 in all."""
    tokens = 1000
    k = torch.zeros(tokens, 1, dim)
    k[0, 0, 0] = 16.0
    v = torch.zeros(tokens, 1, dim)
    v[1:, 0, 2:] = 1.0
    v[0, 0, 1] = 1.0
    w = world_of(k.bfloat16(), v.bfloat16())
    q = torch.zeros(new, 2, dim, dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    scale = max(below, 1e-3) / 16 * math.log(2.0)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    out = mx.kv_attention(q.cuda(), w.gpu, w.table.cuda(), i32([0, new]).cuda(),
                          i32([tokens]).cuda(), scale).cpu().double()
    weight = math.exp(-16 * scale)
    tail = torch.arange(tokens - new, tokens).double()  # keys behind the first that a row sees
    want = (tail * weight / (1 + tail * weight))[:, None, None]
    assert bool(((out[:, :, 2:] - want).abs() <= 2.0 ** -6 * want).all()), \
        float(((out[:, :, 2:] - want).abs() / want).max())
    one = (1 / (1 + tail * weight))[:, None]
    assert bool(((out[:, :, 1] - one).abs() <= 2.0 ** -6 * one).all())


@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 12, 2.0 ** 18, 2.0 ** 24, 2.0 ** 40])
def test_scores_of_any_size(new, dim, size):
    """The first key's score is far above every other one's, so the result is its
    value, however large the scores are (up to 2^92 here): half a step of bf16.
    The other scores are negative, the first one positive and above 20 dim."""
    g = torch.Generator().manual_seed(dim)
    tokens = 300
    k = -torch.rand(tokens, 2, dim, generator=g).clamp(min=0.25)
    k[0] = 8.0
    v = torch.randn(tokens, 2, dim, generator=g)
    w = world_of((k * size).bfloat16(), v.bfloat16())
    q = (torch.rand(new, 4, dim, generator=g).clamp(min=0.3) * 8 * size).bfloat16()
    out = mx.kv_attention(q.cuda(), w.gpu, w.table.cuda(), i32([0, new]).cuda(),
                          i32([tokens]).cuda(), 1.0).cpu().double()
    page = w.table[0, 0]
    first = w.cpu[2][page, :, :, 0].view(ref.F8).double() * ref.pow2(w.cpu[3][page].double())[:, None]
    want = first.repeat_interleave(2, 0).expand_as(out)
    assert bool(((out - want).abs() <= 2.0 ** -8 * want.abs()).all())


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("below", [8, 12, 14, 17, 20])
def test_small_elements_of_q(new, dim, below):
    """q's first element is 1 and meets keys of 0; the others, about 2^-below,
    decide. q is exact down to 2^-13 of its row's largest element, below that
    off by at most 2^-21 of the largest: scores by that times sum |k|, and by
    2^-10 of sum |q k| (the product), weights by twice as much."""
    g = torch.Generator().manual_seed(below)
    tokens = 200
    k = torch.randn(tokens, 2, dim, generator=g) * 2.0 ** below
    k[:, :, 0] = 0
    v = torch.randn(tokens, 2, dim, generator=g)
    w = world_of(k.bfloat16(), v.bfloat16(), 32)
    q = torch.randn(new, 4, dim, generator=g) * 2.0 ** -below
    q[:, :, 0] = 1.0
    q = q.bfloat16()
    scale = 1 / math.sqrt(dim)
    out = mx.kv_attention(q.cuda(), w.gpu, w.table.cuda(), i32([0, new]).cuda(),
                          i32([tokens]).cuda(), scale).cpu().double()
    want, mag, reach = ref.attention(q, w.cpu, w.table, i32([0, new]), i32([tokens]), scale)
    held = w.cpu[0].view(ref.F8).double() * ref.pow2(w.cpu[1].double())[..., None, None]
    held = held[w.table[0].long()].transpose(1, 2).reshape(-1, 2, dim)[:tokens]
    off = 2.0 ** -21 * scale * float(held.abs().sum(2).max())
    eps = 2.0 ** -7 + 2 * 2.0 ** -10 * reach + 2 * off
    tol = 2.0 ** -8 * want.abs() + eps[..., None] * mag
    assert bool(((out - want).abs() <= tol).all()), float(((out - want).abs() / mag).max())


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_channel_that_dominates_its_group(new, dim):
    """One channel's product is 2^9 times the others of its group of eight: the
    matrix core drops bits more than about 2^-14 below it (2^-10 of sum |q k|
    at most). The keys share that channel's value, so it decides nothing."""
    g = torch.Generator().manual_seed(4)
    tokens = 150
    k = torch.randn(tokens, 2, dim, generator=g)
    k[:, :, 3] = 32.0
    v = torch.randn(tokens, 2, dim, generator=g)
    w = world_of(k.bfloat16(), v.bfloat16(), 32)
    q = torch.randn(new, 4, dim, generator=g)
    q[:, :, 3] = 16.0
    q = q.bfloat16()
    out = mx.kv_attention(q.cuda(), w.gpu, w.table.cuda(), i32([0, new]).cuda(),
                          i32([tokens]).cuda()).cpu().double()
    want, mag, reach = ref.attention(q, w.cpu, w.table, i32([0, new]), i32([tokens]), 1 / math.sqrt(dim))
    eps = 2.0 ** -7 + 2 * 2.0 ** -10 * reach
    tol = 2.0 ** -8 * want.abs() + eps[..., None] * mag
    assert bool(((out - want).abs() <= tol).all())
