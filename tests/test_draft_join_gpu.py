"""Attention over trees whose blocks of rows are cut between workgroups, against
64 bits: large ragged batches, and query heads that do not fill the last wave of
the join. Tolerances are those of test_draft_attention_gpu.py; `out` holds a number
that no result is near, so that a row which nothing writes shows."""
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


def batch_of(batch, group, rows, longest, seed):
    """(new tokens, lengths): ragged, one sequence idle, one `longest`, more than `rows` rows in the mean."""
    g = torch.Generator().manual_seed(seed)
    most = 2 * rows // group + 2
    new = [int(torch.randint(1, most + 1, (1,), generator=g)) for _ in range(batch)]
    new[batch // 2] = 0
    while -(-sum(new) // batch) * group <= rows:
        new[int(torch.randint(0, batch // 2, (1,), generator=g))] += 1
    lengths = [n + int(torch.randint(0, 900, (1,), generator=g)) for n in new]
    lengths[batch // 3] = longest
    return new, lengths


def check(w, new, lengths, group, seed=1):
    cu = i32([sum(new[:i]) for i in range(len(new) + 1)])
    sees = masks(new, "tree", seed)
    words = max(1, -(-max(new) // 32))
    q = w.numbers(int(cu[-1]), w.heads * group)
    mask = torch.cat([ref.words_of(m, words) for m in sees])
    out = torch.full(q.shape, 1e30, dtype=torch.bfloat16, device="cuda")
    mx.kv_attention_tree(q.cuda(), w.gpu, w.table.cuda(), cu.cuda(), i32(lengths).cuda(), mask.cuda(), out=out)
    check_attention(out.cpu(), *ref.attention_tree(q, w.cpu, w.table, cu, i32(lengths), sees, 1 / math.sqrt(w.dim)))


def shares(tokens, batch, q_heads, heads, dim, room):
    """Whether workgroups share such a call's tiles: its scratch is the causal call's where they do not."""
    args = tokens, batch, q_heads, heads, dim, room
    return mx.mx_kv_attention_tree_workspace_size(*args) != mx.mx_kv_attention_workspace_size(*args)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch", [24, 33, 40, 64])
@pytest.mark.parametrize("heads,group", [(1, 1), (1, 2), (1, 3), (1, 5), (2, 3), (1, 7), (2, 7), (1, 17)])
def test_query_heads_that_leave_part_of_a_wave(heads, group, batch, dim):
    """The last wave that joins has 4 (dims of 64) or 2 rows (of 128), some of them past the query heads."""
    new, lengths = batch_of(batch, group, 32, 2500, 100 * batch + group)
    w = World(lengths, heads, dim, 64, batch + group)
    assert shares(sum(new), batch, heads * group, heads, dim, w.table.shape[1] * 64)
    w.append(lengths, [0] * batch)
    check(w, new, lengths, group)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch,heads,group,longest", [
    (65, 1, 1, 900),     # more sequences than share, in one piece
    (65, 1, 3, 5000),    # split, a workgroup joins a row
    (70, 2, 5, 5000),    # split, rows joined together, the last ones of a workgroup past the query heads
    (2, 520, 1, 100),    # more kv heads than share
    (64, 64, 40, 300),   # more blocks of rows than share
])
def test_batches_that_do_not_share(batch, heads, group, longest, dim):
    """More than 32 rows in the mean, divided as causal attention divides prompts."""
    new, lengths = batch_of(batch, group, 32, longest, 10 * batch + group)
    if heads > 2:  # short sequences: the reference takes them a head and token at a time
        lengths = [n + x % 40 if x < longest else x for n, x in zip(new, lengths)]
    w = World(lengths, heads, dim, 64, batch + group)
    assert not shares(sum(new), batch, heads * group, heads, dim, w.table.shape[1] * 64)
    w.append(lengths, [0] * batch)
    check(w, new, lengths, group)


@pytest.mark.parametrize("new,group", [(8, 4), (3, 7)])
def test_as_many_sequences_as_share(new, group):
    """Up to 32 rows of 128 dims share in long contexts: 64 sequences do, 65 do not."""
    for batch in (64, 65):
        lengths = [new + 13 * i % 700 for i in range(batch)]
        lengths[5], lengths[63] = 2500, 1300
        w = World(lengths, 1, 128, 64, 3)
        room = w.table.shape[1] * 64
        assert shares(batch * new, batch, group, 1, 128, room) == (batch == 64)
        w.append(lengths, [0] * batch)
        check(w, [new] * batch, lengths, group)


@pytest.mark.parametrize("dim", [64, 128])
def test_cut_blocks_on_streams_and_in_graphs(dim):
    """A captured call, replayed for other inputs, and one on another stream, beside eager ones."""
    new, lengths = batch_of(40, 5, 32, 2500, dim)
    w = World(lengths, 1, dim, 64, 2)
    assert shares(sum(new), 40, 5, 1, dim, w.table.shape[1] * 64)
    w.append(lengths, [0] * 40)
    words = max(1, -(-max(new) // 32))
    table, at = w.table.cuda(), i32(lengths).cuda()
    cu = i32([sum(new[:i]) for i in range(41)]).cuda()
    q = w.numbers(sum(new), 5).cuda()
    mask = torch.cat([ref.words_of(m, words) for m in masks(new, "tree", 1)]).cuda()
    out = torch.empty_like(q)

    def call(out=None):
        return mx.kv_attention_tree(q, w.gpu, table, cu, at, mask, out=out)

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
        q.copy_(w.numbers(sum(new), 5))
        mask.copy_(torch.cat([ref.words_of(m, words) for m in masks(new, "any", seed)]))
        want = call()
        out.fill_(1e30)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
