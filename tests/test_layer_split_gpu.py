"""Attention of prompts that are too few to fill the card: their keys are split
and the parts joined, by either of the two kernels that do. Against 64 bits."""
import pytest
import torch

import microscaling_fp4_block_mx_amd as mx
from test_layer_kv_gpu import World, i32, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


def check(got, want, mag, reach):
    """Half a step of bf16; weights to 2^-8 above and below the line; scores
    off by at most 2^-10 of sum |q k|, twice."""
    nan = torch.isnan(want)
    assert torch.equal(nan, torch.isnan(got))
    eps = 2 * 2.0 ** -8 + 2 * 2.0 ** -10 * reach
    tol = 2.0 ** -8 * want.abs() + eps[..., None] * mag
    assert bool(((got.double() - want).abs() <= tol)[~nan].all())


def parts(tokens, batch, q_heads, heads, dim, max_length):
    size = mx.mx_kv_attention_workspace_size(tokens, batch, q_heads, heads, dim, max_length)
    return size // (tokens * q_heads * (dim + 4) * 4)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [32, 256])
def test_few_splits_of_many_rows(dim, page):
    new, lengths = [520], [2500]
    w = World(lengths, 2, dim, page, 41)
    assert 1 < parts(520, 1, 8, 2, dim, w.table.shape[1] * page) <= 16
    w.append(lengths, [0])
    check(*run_attention(w, new, lengths, 4))


@pytest.mark.parametrize("dim", [64, 128])
def test_many_splits_of_few_rows(dim):
    new, lengths = [40], [17413]
    w = World(lengths, 1, dim, 64, 42)
    assert parts(40, 1, 1, 1, dim, w.table.shape[1] * 64) > 16
    w.append(lengths, [0])
    check(*run_attention(w, new, lengths, 1))


@pytest.mark.parametrize("max_length", [0, 1100, 3000])
@pytest.mark.parametrize("group", [2, 3])
def test_ragged_batches(max_length, group):
    """Sequences with one part beside others with several, one without new
    tokens, one whose first rows see nothing; bounds below the true lengths."""
    new, lengths = [70, 1, 130, 0, 90], [3000, 1, 2049, 128, 30]
    w = World(lengths, 2, 128, 64, 43 + group)
    assert parts(sum(new), 5, 2 * group, 2, 128, 3008) > 1
    w.append(lengths, [0] * 5)
    check(*run_attention(w, new, lengths, group, max_length=max_length, strided=True))


def test_nan_in_one_part():
    """A NaN key page is seen by every row past it, whatever part it lies in."""
    w = World([2600], 1, 64, 64, 44)

    def edit(k, v):
        v[1500, 0, 3] = float("nan")
    w.append([2600], [0], edit=edit)
    got, want, mag, reach = run_attention(w, [600], [2600], 2)
    assert bool(torch.isnan(want).any())
    check(got, want, mag, reach)


def test_repeats_and_replays():
    w = World([3000], 2, 128, 64, 45)
    w.append([3000], [0])
    cu, lengths = i32([0, 300]).cuda(), i32([3000]).cuda()
    q = w.numbers(300, 8).cuda()
    table = w.table.cuda()
    first = mx.kv_attention(q, w.gpu, table, cu, lengths)
    out = torch.empty_like(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mx.kv_attention(q, w.gpu, table, cu, lengths, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.kv_attention(q, w.gpu, table, cu, lengths, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        assert torch.equal(mx.kv_attention(q, w.gpu, table, cu, lengths), first)
