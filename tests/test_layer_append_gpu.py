"""Append of single tokens (the kernel with one wave a page), and append where
its inputs are not of the ordinary kind, bit for bit against the reference."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page", [32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 128])
def test_few_tokens_at_a_time(dim, page, dtype):
    """One to four tokens a sequence, over page boundaries, magnitudes that
    grow and shrink, a NaN and an infinity on the way, an idle sequence."""
    starts = [page - 7, 3, 2 * page - 2, page // 2 + 1]
    steps = [[1, 0, 1, 1], [4, 0, 2, 3], [3, 1, 4, 4], [1, 1, 1, 1], [4, 4, 4, 4], [2, 3, 1, 0],
             [4, 4, 4, 4], [1, 2, 3, 4]]
    totals = [s + sum(st[i] for st in steps) for i, s in enumerate(starts)]
    w = World(totals, 2, dim, page, dim + page)
    w.append(starts, [0] * 4, dtype)
    held = list(starts)
    for t, new in enumerate(steps):
        def edit(k, v):
            if t == 4:
                k[1, 0, 5] = math.nan   # sequence 0, head 0
                v[-1, 1, dim - 1] = math.inf  # the last sequence, head 1
            if t == 2:
                v[0] = 0
        w.append(new, held, dtype, by=2.0 ** ((t * 5) % 13 - 6), edit=edit)
        held = [h + n for h, n in zip(held, new)]
        w.same()


@pytest.mark.parametrize("page", [64, 256])
@pytest.mark.parametrize("dim", [64, 128])
def test_single_tokens_fill_a_page(dim, page):
    """A token at a time through a whole page, the scale growing and the kept
    codes moving at most steps."""
    w = World([page + 3], 3, dim, page, 7)
    for t in range(page + 3):
        w.append([1], [t], by=2.0 ** (t % 9 - 4 + t // 40))
    w.same()


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 2, 1], [90, 70, 50]])
def test_pages_outside_the_cache_are_not_written(new):
    """An entry that names no page (-1, or past the last one) drops its tokens;
    every page of the cache keeps what it held."""
    page = 32
    w = World([128] * 3, 2, 64, page, 21)
    held = [60, 31, 10]
    w.append(held, [0] * 3)
    pool = w.cpu[0].shape[0]
    for bad in (-1, pool, 2 ** 31 - 1, -2 ** 31):
        table = w.table.clone()
        for i in range(3):
            table[i, held[i] // page] = bad  # where the sequence's new tokens begin
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        k, v = w.numbers(cu[-1], 2), w.numbers(cu[-1], 2)
        # the reference has one page more, which takes what names no page
        more = [torch.cat([t, torch.zeros_like(t[:1])]) for t in w.cpu]
        ref.append(more, k, v, torch.where(table == bad, pool, table), i32(cu), i32(held))
        for mine, t in zip(w.cpu, more):
            mine.copy_(t[:pool])
        mx.kv_append(w.gpu, k.cuda(), v.cuda(), table.cuda(), i32(cu).cuda(), i32(held).cuda())
        w.same()


@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("byte", [246, 247, 250, 254])
def test_kept_pages_with_the_largest_scales(byte, new):
    """New tokens enter a page whose byte is one that no quantizer here makes
    (a cache filled by other means) at that byte, like any others."""
    w = World([64], 1, 64, 32, 23)
    w.append([5], [0], torch.float32)
    for t, g in zip(w.cpu, w.gpu):
        if t.dim() == 2:
            t.fill_(byte)
            g.fill_(byte)
    w.append([new], [5], torch.float32, by=2.0 ** 124)
    w.same()
