"""Accepted tokens moved together in the cache, bit for bit, and the whole round
of a drafted step: append, attention, verification, keeping."""
import math

import pytest
import torch

import draft_reference as ref
import microscaling_fp4_block_mx_amd as mx
from test_layer_kv_gpu import World, check_attention, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


def keep(w, held, path, count):
    ref.keep(w.cpu, w.table, held, path, count)
    mx.kv_keep(w.gpu, w.table.cuda(), i32(held).cuda(), path.cuda(), i32(count).cuda())
    w.same()


def padded(paths):
    width = max(1, max(len(p) for p in paths))
    return i32([list(p) + [-1] * (width - len(p)) for p in paths])


def filled(totals, heads, dim, page, seed, edit=None):
    """Sequences whose parts have magnitudes of their own, so that pages' bytes differ."""
    w = World(totals, heads, dim, page, seed)
    held = [0] * len(totals)
    for part in range(5):
        new = [min(17 + 9 * part, t - h) if part < 4 else t - h for t, h in zip(totals, held)]
        w.append(new, held, by=2.0 ** ((part * 5) % 7 - 3), edit=edit if part == 2 else None)
        held = [h + n for h, n in zip(held, new)]
    w.same()
    return w


@pytest.mark.parametrize("page", [32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 128])
def test_paths(dim, page):
    """Within a page, over one, two and many pages, in place, nothing at all."""
    totals = [40, 100, 130, 70, 300, 33, 64, 600, 90]
    held = [20, 28, 31, 60, 20, 32, 60, 10, 64]
    paths = [[0, 2, 5], [0, 1, 3, 4, 9, 30], [0, 40, 41, 90], [0, 1, 2, 3], [5, 100, 200, 201, 270], [0], [1, 3],
             list(range(3, 590, 2)), []]
    w = filled(totals, 2, dim, page, dim + page)
    keep(w, held, padded(paths), [len(p) for p in paths])
    # once more, shorter than the paths are
    keep(w, held, padded(paths), [max(0, len(p) - 2) for p in paths])


def test_random_paths():
    g = torch.Generator().manual_seed(3)
    for seed in range(6):
        page = (32, 64, 128)[seed % 3]
        new = [int(torch.randint(1, 70, (1,), generator=g)) for _ in range(6)]
        held = [int(torch.randint(0, 150, (1,), generator=g)) for _ in range(6)]
        w = filled([h + n for h, n in zip(held, new)], 3, (64, 128)[seed % 2], page, seed)
        paths = [[j for j in range(n) if float(torch.rand(1, generator=g)) < 0.4] for n in new]
        keep(w, held, padded(paths), [len(p) for p in paths])


def test_paths_that_end_early():
    """Nodes not in rising order, below zero, past the table; counts past the path's width, and negative."""
    totals = [128] * 6
    w = filled(totals, 2, 64, 32, 7)
    held = [30, 30, 100, 30, 30, 30]
    paths = i32([[0, 3, 2, 9], [2, 2, 5, 6], [1, 20, 28, 40], [-1, 4, 5, 6], [3, 5, -1, 9], [1, 3, 6, 2 ** 31 - 1]])
    keep(w, held, paths, [4, 4, 9, 4, 4, -3])
    keep(w, held, paths, [4, 4, 4, 4, 100, 4])


def test_nan_pages():
    """A source page that is NaN makes where its token goes NaN; signs are kept."""
    def edit(k, v):
        k[20, 0, 3] = math.nan
        v[60, 1, 5] = math.inf
    w = filled([200, 200], 2, 64, 32, 8, edit)
    assert bool((w.cpu[1] == 255).any()) and bool((w.cpu[3] == 255).any())
    keep(w, [20, 30], padded([[0, 30, 60, 90, 120, 150], [2, 40, 80, 120]]), [6, 4])


def test_pages_outside_the_cache():
    w = filled([96, 96], 2, 64, 32, 9)
    w.table[0, 1], w.table[1, 2] = -1, w.cpu[0].shape[0] + 5
    # to a page that is none: dropped; from one: zeros
    keep(w, [20, 20], padded([[0, 5, 9, 20, 21, 22, 23, 24, 25, 26, 27, 28, 29, 30], [0, 2, 50, 60]]), [14, 4])


def test_negative_lengths_and_idle():
    w = filled([64, 64, 64], 1, 64, 32, 10)
    keep(w, [-5, 10, 10], padded([[1, 2], [1, 2], [1, 2]]), [2, 0, 1])


@pytest.mark.parametrize("dim", [64, 128])
def test_a_drafted_round(dim):
    """Rotated append of a tree, attention over it, verification, keeping, and then a
    plain token whose attention sees the accepted ones alone: against the same
    sequence without any drafts."""
    heads, group, page, vocab = 2, 3, 32, 500
    g = torch.Generator().manual_seed(dim)
    held, parents = [45, 3, 120], [[-1, 0, 0, 1, 2, 2, 4, 5], [-1, 0, 1], [-1, 0, 0, 0, 3, 4, 5, 6, 7]]
    new = [len(p) for p in parents]
    totals = [h + n + 4 for h, n in zip(held, new)]
    table = mx.rotary_table(300, dim)
    weight = (torch.rand(dim, generator=g) + 0.5).bfloat16().cuda()

    def randn(n, h):
        return torch.randn(n, h, dim, generator=g).bfloat16().cuda()

    w = World(totals, heads, dim, page, dim)
    pages = w.table.cuda()
    cu0 = i32([0] + torch.tensor(held).cumsum(0).tolist()).cuda()
    k0, v0 = randn(sum(held), heads), randn(sum(held), heads)
    zero = i32([0] * 3).cuda()
    mx.kv_append_rotary(w.gpu, k0, v0, pages, cu0, zero, mx.Rotary(table), weight)
    # the drafted step
    mask, depth = mx.tree_mask(parents)
    cu = i32([0] + torch.tensor(new).cumsum(0).tolist()).cuda()
    lengths = i32(held).cuda()
    positions = torch.cat([depth[a:b] + h for a, b, h in zip(cu.tolist(), cu.tolist()[1:], held)]).int()
    q, k, v = randn(sum(new), heads * group), randn(sum(new), heads), randn(sum(new), heads)
    q, _ = mx.norm_rotate(q, None, weight, None, mx.Rotary(table, positions))
    mx.kv_append_rotary(w.gpu, k, v, pages, cu, lengths, mx.Rotary(table, positions), weight)
    longest = max(h + n for h, n in zip(held, new))
    out = mx.kv_attention_tree(q, w.gpu, pages, cu, lengths + (cu[1:] - cu[:-1]), mask, max_length=longest)
    cpu = [t.cpu() for t in w.gpu]
    sees = [ref.ancestors(p) for p in parents]
    check_attention(out.cpu(), *ref.attention_tree(q.cpu(), cpu, w.table, cu.cpu(),
                                                   i32([h + n for h, n in zip(held, new)]), sees, 1 / math.sqrt(dim)))
    # verification: greedy rows lead sequence 0 to nodes 2, 5, 7, sequence 1 nowhere, sequence 2 to 3, 4
    ids = torch.arange(sum(new), dtype=torch.int32) + 10
    target = torch.zeros(sum(new), vocab)
    for a, path, last in ((0, [0, 2, 5, 7], 400), (8, [0], 401), (11, [0, 3, 4], 402)):
        for node, then in zip(path, path[1:] + [None]):
            target[a + node, last if then is None else int(ids[a + then])] = 1.0
    up = i32([p for tree in parents for p in tree])
    numbers = torch.rand(sum(new), 2, generator=g)
    path, count, token = mx.verify_drafts(target.cuda(), ids.cuda(), up.cuda(), cu, numbers.cuda(), 8)
    assert path.tolist() == [[0, 2, 5, 7] + [-1] * 4, [0] + [-1] * 7, [0, 3, 4] + [-1] * 5]
    assert count.tolist() == [4, 1, 3] and token.tolist() == [400, 401, 402]
    mx.kv_keep(w.gpu, pages, lengths, path, count)
    after = lengths + count
    # one token more, and the same without drafts in a cache of its own
    q1, k1, v1 = randn(3, heads * group), randn(3, heads), randn(3, heads)
    one = i32([0, 1, 2, 3]).cuda()
    plain = World(totals, heads, dim, page, dim)
    mx.kv_append_rotary(plain.gpu, k0, v0, pages, cu0, zero, mx.Rotary(table), weight)
    took = torch.cat([cu[i] + path[i, :int(count[i])] for i in range(3)]).long()
    cu_took = i32([0, 4, 5, 8]).cuda()
    mx.kv_append_rotary(plain.gpu, k[took], v[took], pages, cu_took, lengths, mx.Rotary(table), weight)
    got = []
    for cache in (w.gpu, plain.gpu):
        mx.kv_append_rotary(cache, k1, v1, pages, one, after, mx.Rotary(table), weight)
        q2, _ = mx.norm_rotate(q1, None, weight, None, mx.Rotary(table, after))
        got.append(mx.kv_attention(q2, cache, pages, one, after + 1, max_length=longest + 1).cpu())
    cpu = [t.cpu() for t in w.gpu]
    import layer_reference
    check_attention(got[0], *layer_reference.attention(q2.cpu(), cpu, w.table, one.cpu(), after.cpu() + 1,
                                                       1 / math.sqrt(dim)))
    # beside the cache without drafts: a page's byte may be one of a rejected token's, so each number is
    # off by at most 2^-3 of itself from a page twice rounded (2^-4 each), keys and values alike
    assert float((got[0].float() - got[1].float()).norm() / got[1].float().norm()) <= 4 / 16


def test_streams_and_graphs():
    w = filled([100, 80], 2, 128, 32, 11)
    start = [t.clone() for t in w.gpu]
    table, held, count = w.table.cuda(), i32([30, 40]).cuda(), i32([0, 0]).cuda()
    path = torch.zeros(2, 5, dtype=torch.int32, device="cuda")

    def call():
        mx.kv_keep(w.gpu, table, held, path, count)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([[0, 3, 9, 20, 35], [1, 2, 3, -1, -1]], [[5, 6, 50, -1, -1], [0, 1, 2, 10, 11]], [[0, 1, 2, 3, 4]] * 2):
        path.copy_(i32(new))
        count.copy_((path >= 0).sum(1))
        got = []
        for f in (graph.replay, call):
            for a, b in zip(w.gpu, start):
                a.copy_(b)
            f()
            torch.cuda.synchronize()
            got.append([t.clone() for t in w.gpu])
        assert all(torch.equal(a, b) for a, b in zip(*got))


def test_refusals():
    cache = mx.kv_cache(4, 2, 64, 32)
    t, i = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.kv_keep(cache, t, i, t, i)
    none = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    mx.kv_keep(cache, none, i[:0], none, i[:0])
    bad = [
        lambda: mx.kv_keep(cache, t[0], i, t, i), lambda: mx.kv_keep(cache, t, i, t[0], i),
        lambda: mx.kv_keep(cache, t.long(), i, t, i), lambda: mx.kv_keep(cache, t, i.long(), t, i),
        lambda: mx.kv_keep(cache, t, i, t.long(), i), lambda: mx.kv_keep(cache, t, i, t, i.long()),
        lambda: mx.kv_keep(cache, t, i, t.expand(2, 2), i), lambda: mx.kv_keep(cache, t, i, t, t[0]),
        lambda: mx.kv_keep(cache, t, i, t[:, :0], i), lambda: mx.kv_keep(cache, t.cpu(), i, t, i),
        lambda: mx.kv_keep(cache._replace(v_codes=cache.k_codes), t, i, t, i),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    torch.cuda.synchronize()
