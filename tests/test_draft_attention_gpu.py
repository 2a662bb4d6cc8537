"""Attention over trees of drafted tokens against 64 bits: masks of every kind,
ragged batches, both kernels, page and tile edges, rows that see nothing.

Tolerances are those of causal attention (its scores and weights are formed the
same way): half a step of bf16, weights to 2^-9 above and below the line,
scores off by at most 2^-10 of sum |q k|, twice."""
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


def masks(new, kind, seed):
    """A bool [n, n] for each sequence."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in new:
        if kind == "tree":
            parents = [int(torch.randint(max(0, j - 3), j, (1,), generator=g)) if j else -1 for j in range(n)]
            out.append(ref.ancestors(parents))
        elif kind == "chain":
            out.append(torch.ones(n, n).tril().bool())
        elif kind == "any":  # not a tree's: later tokens, not itself, and rows without any
            m = torch.rand(n, n, generator=g) < 0.4
            if n > 2:
                m[n // 2] = False
            out.append(m)
        else:
            out.append(torch.full((n, n), kind == "all"))
    return out


def run(w, new, lengths, group, sees, words=None, scale=None, max_length=0, junk=False):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    words = words or max(1, -(-max(new) // 32))
    rows = [ref.words_of(m, words) for m in sees]
    if junk:  # bits past a sequence's new tokens do not count
        for n, r in zip(new, rows):
            for b in range(n, 32 * words):
                r[:, b // 32] |= torch.tensor((1 << (b % 32)) - (1 << 32 if b % 32 == 31 else 0), dtype=torch.int32)
    q = w.numbers(cu[-1], w.heads * group)
    cu, lengths = i32(cu), i32(lengths)
    got = mx.kv_attention_tree(q.cuda(), w.gpu, w.table.cuda(), cu.cuda(), lengths.cuda(),
                               torch.cat(rows).cuda(), scale, max_length)
    used = 1 / math.sqrt(w.dim) if scale is None else scale
    return (got.cpu(),) + ref.attention_tree(q, w.cpu, w.table, cu, lengths, sees, used)


@pytest.mark.parametrize("kind", ["tree", "any", "chain", "all", "none"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 17])
def test_masks(kind, dim, group):
    new, lengths = [1, 7, 0, 33, 20, 12], [1, 130, 64, 170, 20, 127]
    w = World(lengths, 2, dim, 64, group)
    w.append(lengths, [0] * len(lengths))
    check_attention(*run(w, new, lengths, group, masks(new, kind, 1)))


@pytest.mark.parametrize("page", [32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 128])
def test_edges_of_tiles_and_pages(page, dim):
    """New tokens that begin and end at every kind of place in a tile of 128 keys."""
    new = [2, 3, 1, 2, 5, 4, 16, 9]
    lengths = [128, 129, 256, 257, 258, 300, 130, 513]
    w = World(lengths, 1, dim, page, page)
    w.append(lengths, [0] * len(lengths))
    check_attention(*run(w, new, lengths, 2, masks(new, "tree", 2)))
    check_attention(*run(w, new, lengths, 2, masks(new, "any", 3), junk=True))


@pytest.mark.parametrize("dim", [64, 128])
def test_many_nodes(dim):
    """More rows than a block holds, masks of several words, words beyond and short of the nodes."""
    new, lengths = [150, 64, 1, 97], [400, 64, 300, 129]
    w = World(lengths, 2, dim, 64, 5)
    w.append(lengths, [0] * 4)
    sees = masks(new, "any", 4)
    check_attention(*run(w, new, lengths, 3, sees, junk=True))
    check_attention(*run(w, new, lengths, 3, sees, words=9, junk=True))
    for m in sees:
        m[:, 64:] = False
    check_attention(*run(w, new, lengths, 3, sees, words=2))


@pytest.mark.parametrize("new", [1, 12, 60])
def test_more_new_tokens_than_the_cache_holds(new):
    """The keys are the last new tokens; lengths of zero give zeros."""
    lengths = [0, 50, 0, 20, 1]
    w = World([64] * 5, 2, 64, 32, 1)
    w.append(lengths, [0] * 5)
    got, want, mag, reach = run(w, [new] * 5, lengths, 4, masks([new] * 5, "any", 6))
    check_attention(got, want, mag, reach)
    assert bool((got[:new] == 0).all())


@pytest.mark.parametrize("new", [4, 40])
def test_long_contexts_in_pieces(new):
    """Sequences split over workgroups; a bound on the lengths only steers."""
    lengths = [5000, new, 2900]
    w = World(lengths, 1, 64, 64, 8)
    w.append(lengths, [0] * 3)
    sees = masks([new] * 3, "tree", 7)
    state = w.g.get_state()
    for bound in (0, 5000, 100):
        w.g.set_state(state)
        check_attention(*run(w, [new] * 3, lengths, 4, sees, max_length=bound))


@pytest.mark.parametrize("new", [3, 70])
def test_a_causal_mask_is_causal_attention(new):
    lengths = [300, 1000, new]
    w = World(lengths, 2, 128, 64, 9)
    w.append(lengths, [0] * 3)
    q = w.numbers(3 * new, 8).cuda()
    cu = i32([0, new, 2 * new, 3 * new]).cuda()
    mask = torch.cat([ref.words_of(m, 3) for m in masks([new] * 3, "chain", 0)]).cuda()
    args = (q, w.gpu, w.table.cuda(), cu, i32(lengths).cuda())
    a, b = mx.kv_attention_tree(*args, mask).cpu().double(), mx.kv_attention(*args).cpu().double()
    if new == 3:
        assert torch.equal(a, b)  # one kernel, one split of the keys
        return
    # the keys are divided otherwise: scores are the same bits, a weight is rounded to bf16 against another
    # maximum (2^-9 of itself, in the sums above and below the line, on both sides: 4 x 2^-9 of sum p |v|), the
    # result once on each side (half a step, 2^-8 of it, each); sums in 32 bits lie below 2^-14 of sum p |v|
    _, mag, _ = ref.attention_tree(q.cpu(), w.cpu, w.table, cu.cpu(), i32(lengths),
                                   masks([new] * 3, "chain", 0), 1 / math.sqrt(128))
    assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + (2.0 ** -7 + 2.0 ** -13) * mag).all())


@pytest.mark.parametrize("new", [5, 8, 70])
def test_what_is_not_seen_does_not_reach(new):
    """A NaN key among the new tokens reaches the rows that see it, the page's
    values those that see any of its tokens; nothing else."""
    w = World([200], 1, 64, 32, 9)

    w.append([190], [0])
    w.append([10], [190], edit=lambda k, v: k.__setitem__((8, 0, 3), math.nan))
    sees = masks([new], "any", 8)
    first = 200 - new
    page = max(0, 192 - first)  # the NaN's page: positions 192 to 199
    sees[0][: new // 2, page:] = False
    got, want, mag, reach = run(w, [new], [200], 2, sees)
    # 5 new tokens begin inside that page: every one of them sees its first keys
    assert bool(torch.isnan(want).any()) and bool(torch.isnan(want[: new // 2]).any()) == (first > 192)
    check_attention(got, want, mag, reach)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch,new,group,longest", [
    (5, 7, 4, 2500),     # up to 32 rows, long contexts
    (9, 16, 4, 700),     # blocks of 64 rows, some sequences with two
    (3, 40, 8, 1100),    # several blocks of 128 rows a sequence
    (2, 3, 65, 400),     # more than 64 query heads to a kv head
    (64, 12, 4, 140),    # as many sequences as share their tiles
    (70, 11, 4, 140),    # more
    (33, 9, 128, 90),    # a token a block
])
def test_divisions_of_the_work(batch, new, group, longest, dim):
    """Ragged batches with idle slots and empty sequences, through every way of dividing rows and keys."""
    g = torch.Generator().manual_seed(batch)
    counts = [int(torch.randint(1, new + 1, (1,), generator=g)) for _ in range(batch)]
    counts[0], counts[batch // 2] = new, 0
    lengths = [n + int(torch.randint(0, longest - n, (1,), generator=g)) for n in counts]
    lengths[0] = longest
    held = list(lengths)
    lengths[-1] = 0 if batch > 2 else lengths[-1]  # rows that see nothing
    w = World(held, 1, dim, 64, batch)
    w.append(held, [0] * batch)
    check_attention(*run(w, counts, lengths, group, masks(counts, "tree", 3)))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("most", [16, 32])
def test_parts_of_blocks(most, dim):
    """Blocks of 64 and of 128 rows with every number of rows that a wave or two have none of."""
    new = [n for n in range(1, most + 1) if most == 16 or n % 4 < 2]
    lengths = [n + 130 * (i % 7) + 3 * n for i, n in enumerate(new)]
    w = World(lengths, 2, dim, 32, most)
    w.append(lengths, [0] * len(new))
    check_attention(*run(w, new, lengths, 4, masks(new, "tree", 11), max_length=2000))


@pytest.mark.parametrize("new", [[3, 2], [40, 30], [4] * 70])
def test_rows_behind_the_last_sequence(new):
    """A padded batch: rows of q and of the mask behind cu's last are not read, those of out stay."""
    n, more = sum(new), 37
    lengths = [x + 500 for x in new]
    w = World(lengths, 2, 128, 64, 9)
    w.append(lengths, [0] * len(new))
    sees = masks(new, "tree", 12)
    words = -(-max(new) // 32)
    q = w.numbers(n, 8)
    cu = i32([sum(new[:i]) for i in range(len(new) + 1)])
    out = torch.full((n + more, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    bits = torch.cat([ref.words_of(m, words) for m in sees] + [torch.full((more, words), -1, dtype=torch.int32)])
    nan = torch.full((more, 8, 128), math.nan, dtype=torch.bfloat16)
    got = mx.kv_attention_tree(torch.cat([q, nan]).cuda(), w.gpu, w.table.cuda(), cu.cuda(), i32(lengths).cuda(),
                               bits.cuda(), out=out).cpu()
    assert bool((got[n:] == 7.0).all())
    check_attention(got[:n], *ref.attention_tree(q, w.cpu, w.table, cu, i32(lengths), sees, 1 / math.sqrt(128)))


@pytest.mark.parametrize("heads", [1, 5, 16])
def test_heads(heads):
    """Workgroups by kv heads, shares of one and of many tiles."""
    lengths, new = [3000, 40, 900, 33], [20, 20, 1, 33]
    w = World(lengths, heads, 128, 32, heads)
    w.append(lengths, [0] * 4)
    check_attention(*run(w, new, lengths, 4, masks(new, "tree", 5)))


def test_tree_mask():
    parents = [[-1, 0, 0, 1, 1, 2, 5], [-1], [], [-1] + list(range(39))]
    mask, depth = mx.tree_mask(parents, device="cpu")
    assert mask.shape == (48, 2) and mask.dtype == torch.int32
    assert torch.equal(mask, torch.cat([ref.words_of(ref.ancestors(p), 2) for p in parents]))
    assert depth.tolist() == [0, 1, 1, 2, 2, 2, 3, 0] + list(range(40))
    for bad in ([[0]], [[-1, 1]], [[-1, -2]]):
        with pytest.raises(ValueError):
            mx.tree_mask(bad, device="cpu")
    assert mx.tree_mask([], device="cpu")[0].shape == (0, 1)


def test_offsets_past_32_bits():
    """Mask rows and pages far into their arrays."""
    w = World([300, 65], 2, 64, 64, 6)
    w.append([300, 65], [0, 0])
    new, words = [9, 7], 60000
    sees = masks(new, "tree", 9)
    check_attention(*run(w, new, [300, 65], 2, sees, words=words))


def test_streams_and_graphs():
    lengths, new = [900, 300], 6
    w = World(lengths, 2, 128, 64, 11)
    w.append(lengths, [0, 0])
    table, cu, at = w.table.cuda(), i32([0, new, 2 * new]).cuda(), i32(lengths).cuda()
    q = w.numbers(2 * new, 8).cuda()
    mask = torch.cat([ref.words_of(m, 1) for m in masks([new] * 2, "tree", 1)]).cuda()
    out = torch.empty_like(q)

    def call(out=None):
        return mx.kv_attention_tree(q, w.gpu, table, cu, at, mask, max_length=1000, out=out)

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for seed in range(4):
        q.copy_(w.numbers(2 * new, 8))
        mask.copy_(torch.cat([ref.words_of(m, 1) for m in masks([new] * 2, "any", seed)]))
        want = call()
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    cache = mx.kv_cache(4, 2, 64, 32)
    i, t = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    bad = [
        lambda: mx.kv_attention_tree(q, cache, t, i, i[:1], m[0]),
        lambda: mx.kv_attention_tree(q, cache, t, i, i[:1], m.long()),
        lambda: mx.kv_attention_tree(q, cache, t, i, i[:1], m[:, :0]),
        lambda: mx.kv_attention_tree(q, cache, t, i, i[:1], m.cpu()),
        lambda: mx.kv_attention_tree(q, cache, t, i, i[:1], m.expand(2, 1)),
        lambda: mx.kv_attention_tree(q, cache, t, i, i[:1], torch.zeros(1, 70000, dtype=torch.int32, device="cuda")),
        lambda: mx.kv_attention_tree(q.float(), cache, t, i, i[:1], m),
        lambda: mx.kv_attention_tree(q[:, :3], cache, t, i, i[:1], m),
        lambda: mx.kv_attention_tree(q, cache, t, i, i[:1], m, scale=0.0),
        lambda: mx.kv_attention_tree(q, cache, t[0], i, i[:1], m),
        lambda: mx.kv_attention_tree(q, cache, t, i, i[:1], m, out=q),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    torch.cuda.synchronize()
