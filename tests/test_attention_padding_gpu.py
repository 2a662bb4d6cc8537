"""Rows of no sequence (in front of cu's first and behind its last, as a padded batch
has them) in attention, causal and over trees, where sequences are split and joined:
nothing of q or of the masks there is read, and those rows of `out` stay."""
import math

import pytest
import torch

import draft_reference as ref
import microscaling_fp4_block_mx_amd as mx
from test_draft_attention_gpu import masks
from test_layer_kv_gpu import World, check_attention, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch,before,behind", [
    (3, 0, 0),       # few rows, a workgroup joins a row
    (3, 2, 3),
    (3, 0, 37),      # (over a tree tiles are shared)
    (3, 5, 20),
    (70, 0, 450),    # few rows, many of which are joined at a time
    (70, 40, 410),
    (2, 0, 140),     # tiles, a workgroup joins a row
    (2, 9, 140),
    (70, 0, 600),    # tiles, many
    (70, 30, 570),
])
def test_rows_of_no_sequence(batch, before, behind, dim, tree):
    heads, group = 2, 4
    lengths = [100 + i for i in range(batch)]
    lengths[1] = 5000
    new = [1] * batch
    new[1] = 3
    w = World(lengths, heads, dim, 64, batch + behind)
    w.append(lengths, [0] * batch)
    n = sum(new)
    q = w.numbers(n, heads * group)

    def padded(x, by):
        front, back = (torch.full((m,) + x.shape[1:], by, dtype=x.dtype) for m in (before, behind))
        return torch.cat([front, x, back]).cuda()

    cu = i32([sum(new[:i]) for i in range(batch + 1)])
    args = [padded(q, math.nan), w.gpu, w.table.cuda(), (cu + before).cuda(), i32(lengths).cuda()]
    if tree:
        sees = masks(new, "tree", 3)
        args.append(padded(torch.cat([ref.words_of(m, 1) for m in sees]), -1))
    size = (mx.mx_kv_attention_tree_workspace_size if tree else mx.mx_kv_attention_workspace_size)
    assert size(before + n + behind, batch, heads * group, heads, dim, w.table.shape[1] * 64) > 0
    out = padded(torch.full_like(q, 7.0), 7.0)
    got = (mx.kv_attention_tree if tree else mx.kv_attention)(*args, out=out).cpu()
    assert bool((got[:before] == 7.0).all()) and bool((got[before + n:] == 7.0).all())
    if not tree:
        sees = masks(new, "chain", 3)
    check_attention(got[before:before + n],
                    *ref.attention_tree(q, w.cpu, w.table, cu, i32(lengths), sees, 1 / math.sqrt(dim)))
