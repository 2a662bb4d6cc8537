"""Verification of drafted tokens against a walk in 64 bits, node by node: the
same paths, counts and tokens. A border between two tokens is hit by rounding
with a chance of some 10^-13 a draw, so none of these differs by it."""
import math

import pytest
import torch

import draft_reference as ref
import microscaling_fp4_block_mx_amd as mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def world(sizes, vocab, seed, dtype=torch.float32, chain=False, peaked=4.0, near=0.5):
    """Probabilities of a target and a draft, and trees drawn from the draft's."""
    g = torch.Generator().manual_seed(seed)
    rows = sum(sizes)
    logits = torch.randn(rows, vocab, generator=g) * peaked
    target = torch.softmax(logits, 1).to(dtype)
    draft = torch.softmax(logits + near * torch.randn(rows, vocab, generator=g), 1).to(dtype)
    cu, parents, ids = [0], [], []
    for n in sizes:
        a = cu[-1]
        for j in range(n):
            up = -1 if j == 0 else j - 1 if chain else int(torch.randint(max(0, j - 4), j, (1,), generator=g))
            parents.append(up)
            ids.append(int(torch.multinomial(draft[a + max(up, 0)].float(), 1, generator=g)))
        cu.append(a + n)
    numbers = torch.rand(rows, 2, generator=g)
    return target, draft, i32(ids), i32(parents), i32(cu), numbers


def call(target, draft, ids, parents, cu, numbers, width):
    out = mx.verify_drafts(target.cuda(), ids.cuda(), parents.cuda(), cu.cuda(), numbers.cuda(), width,
                           None if draft is None else draft.cuda())
    return [t.tolist() for t in out]


def same(target, draft, ids, parents, cu, numbers, width):
    got = call(target, draft, ids, parents, cu, numbers, width)
    want = ref.verify(target, draft, ids, parents, cu, numbers, width)
    assert got[0] == want[0] and got[1] == want[1] and got[2] == want[2], (got, want)
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1, 2, 7, 63, 1000, 2047, 2048, 2049, 8191, 33003])
def test_trees_and_chains(vocab, dtype):
    sizes = [5, 1, 12, 0, 9, 30, 2]
    reached = 0
    for chain in (False, True):
        w = world(sizes, vocab, vocab + chain, dtype, chain)
        for draft in (w[1], None):
            got = same(w[0], draft, *w[2:], 31)
            reached += sum(got[1])
    assert reached > 4 * 6  # some child or other was followed


@pytest.mark.parametrize("width", [1, 2, 3, 5])
def test_width_ends_paths(width):
    w = world([20, 20, 20], 50, 3, peaked=6.0, near=0.05)
    for draft in (w[1], None):
        got = same(w[0], draft, *w[2:], width)
        assert max(got[1]) <= width
    same(w[0], w[1], *w[2:], 1024)


@pytest.mark.parametrize("sizes", [[200], [64, 65, 63], [1024], [1100, 3], [1] * 300])
def test_numbers_of_nodes(sizes):
    for chain in (False, True):
        w = world(sizes, 40, len(sizes), chain=chain, peaked=8.0, near=0.02)
        for draft in (w[1], None):
            same(w[0], draft, *w[2:], 1024)


def test_a_long_chain_is_followed_to_its_end():
    """Target and draft alike: every drafted token is taken, unless u q < p fails at equality."""
    w = list(world([70, 1024], 30, 5, chain=True))
    got = same(w[0], w[0], *w[2:], 1024)
    assert got[1] == [70, 1024]
    w[5][:, 0] = 1.0  # not below 1: never q < p, nothing is left of p - q, p itself is drawn from
    got = same(w[0], w[0], *w[2:], 1024)
    assert got[1] == [1, 1]


def test_greedy_and_empty_rows():
    """One-hot rows (temperature zero), rows of zeros, and what is no probability."""
    w = list(world([6, 6, 6, 6], 300, 6, chain=True))
    target = torch.zeros_like(w[0])
    for j in range(24):
        target[j, int(w[2][min(j + 1, 23)]) if j % 6 < 3 else 5] = 1.0
    for draft in (None, w[1]):
        got = same(target, draft, *w[2:], 6)
        assert got[1] == [4] * 4 or draft is not None
    target[6:12] = 0.0  # sequence 1: nothing to draw
    target[12, 10], target[12, 20], target[12, 30] = math.nan, -1.0, math.inf
    for draft in (None, w[1]):
        got = same(target, draft, *w[2:], 6)
        assert got[2][1] == -1 and got[1][1] == 1
    # the draft's rows hold what is no probability
    w[1][0, :100], w[1][6, :100], w[1][12] = math.nan, math.inf, -3.0
    same(w[0], w[1], *w[2:], 6)


def test_random_numbers_at_their_ends():
    w = list(world([4] * 4, 3000, 7))
    for value in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0):
        w[5][:, 1] = value
        w[5][:, 0] = min(value, 0.999)
        for draft in (None, w[1]):
            same(w[0], draft, *w[2:], 4)


def test_tokens_and_parents_out_of_range():
    """Tokens outside the vocabulary are never taken, nodes whose parents lead nowhere never reached."""
    w = list(world([12, 12], 40, 8, peaked=6.0, near=0.02))
    w[2][3], w[2][5], w[2][14] = -1, 40, 2 ** 31 - 1
    same(w[0], w[1], *w[2:], 12)
    w[3][4], w[3][7], w[3][9], w[3][13], w[3][0] = 4, 11, -7, 2 ** 31 - 1, 5
    for draft in (None, w[1]):
        got = same(w[0], draft, *w[2:], 12)
        assert not {4, 7, 9} & set(got[0][0]) and 1 not in got[0][1]


@pytest.mark.parametrize("with_draft", [False, True])
def test_rows_behind_the_last_sequence(with_draft):
    """A padded batch: the rows behind cu's last do not count."""
    w = world([5, 9, 30], 700, 22)
    cu = i32([0, 5, 14])
    draft = w[1] if with_draft else None
    want = ref.verify(w[0][:14], None if draft is None else draft[:14], w[2][:14], w[3][:14], cu, w[5][:14], 9)
    w[0][14:] = math.nan
    w[1][14:] = math.nan
    w[2][14:], w[3][14:] = -1, 1 << 30
    assert call(w[0], draft, w[2], w[3], cu, w[5], 9) == [want[0], want[1], want[2]]


@pytest.mark.parametrize("with_draft", [False, True])
def test_sequences_that_share_rows(with_draft):
    """Where cu falls, against its description, the sequences that share rows have
    any result that is one: rising nodes of theirs, a token of the vocabulary."""
    w = world([700, 24, 3], 50, 21, chain=True, near=0.01)
    cu = [0, 700, 24, 724, 3, 727]
    path, count, token = call(w[0], w[1] if with_draft else None, w[2], w[3], i32(cu), w[5], 600)
    for i, (p, c, t) in enumerate(zip(path, count, token)):
        n = max(cu[i + 1] - cu[i], 0)
        assert (c == 0 and t == -1) if n == 0 else (1 <= c <= min(n, 600) and -1 <= t < 50)
        assert p[c:] == [-1] * (600 - c) and sorted(set(p[:c])) == p[:c]
        assert n == 0 or (p[0] == 0 and p[c - 1] < n)


def test_siblings_with_one_token():
    """Of several children with the drawn token the first is followed."""
    parents, ids = i32([-1, 0, 0, 0, 2, 2]), i32([0, 7, 9, 9, 3, 3])
    target = torch.full((6, 16), 1e-9)
    target[0, 9] = target[1, 9] = target[2, 3] = target[4, 1] = 1.0
    numbers = torch.full((6, 2), 0.5)
    got = same(target, None, ids, parents, i32([0, 6]), numbers, 6)
    assert got[0][0][:3] == [0, 2, 4] and got[2] == [1]
    draft = torch.full((6, 16), 1.0 / 16)
    draft[2] = 0.0
    draft[2, 3] = 1.0
    got = same(target, draft, ids, parents, i32([0, 6]), numbers, 6)
    assert got[0][0][:3] == [0, 2, 4]


@pytest.mark.parametrize("with_draft", [False, True])
def test_tokens_are_distributed_as_the_targets(with_draft):
    """The first token behind the root, whether drafted or drawn, over 40,000 trees:
    each frequency lies within 6 standard deviations of the target's probability."""
    n, vocab = 40000, 6
    g = torch.Generator().manual_seed(9)
    p = torch.tensor([0.4, 0.25, 0.2, 0.1, 0.05, 0.0])
    q = torch.tensor([0.1, 0.3, 0.1, 0.1, 0.3, 0.1])
    parents = i32([-1, 0, 0] * n)
    ids = torch.multinomial(q.expand(n, -1), 2, replacement=True, generator=g)
    ids = torch.cat([torch.zeros(n, 1, dtype=torch.long), ids], 1).int().view(-1)
    cu = torch.arange(n + 1, dtype=torch.int32) * 3
    target, draft = p.expand(3 * n, -1).contiguous(), q.expand(3 * n, -1).contiguous()
    numbers = torch.rand(3 * n, 2, generator=g)
    path, count, token = call(target, draft if with_draft else None, ids, parents, cu, numbers, 3)
    first = [int(ids[3 * i + path[i][1]]) if count[i] > 1 else token[i] for i in range(n)]
    seen = torch.bincount(torch.tensor(first), minlength=vocab).double() / n
    bound = 6 * torch.sqrt(p.double() * (1 - p.double()) / n)
    assert bool(((seen - p.double()).abs() <= bound).all()), seen


def test_no_tokens_and_no_sequences():
    empty = torch.empty(0, 10, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    two = torch.empty(0, 2, device="cuda")
    path, count, token = mx.verify_drafts(empty, none, none, i32([0, 0, 0]).cuda(), two, 3)
    assert path.tolist() == [[-1] * 3] * 2 and count.tolist() == [0, 0] and token.tolist() == [-1, -1]
    path, count, token = mx.verify_drafts(empty, none, none, i32([0]).cuda(), two, 3)
    assert path.shape == (0, 3) and count.shape == token.shape == (0,)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_past_32_bits(dtype):
    """Rows that begin more than 2^31 elements into the array, of odd length."""
    vocab = (1 << 28) + 13
    rows = 10
    target = torch.zeros(rows, vocab, dtype=dtype, device="cuda")
    ids, parents = i32([0] + [vocab - 1] * 9), i32([-1] + list(range(9)))
    target[:9, vocab - 1] = 1.0
    target[9, 123456789] = 0.25
    target[9, vocab - 2] = 0.75
    numbers = torch.full((rows, 2), 0.3, device="cuda")
    args = (target, ids.cuda(), parents.cuda(), i32([0, 10]).cuda(), numbers, 10)
    path, count, token = mx.verify_drafts(*args)
    assert count.tolist() == [10] and token.tolist() == [vocab - 2]
    numbers[9, 1] = 0.2
    assert mx.verify_drafts(*args)[2].tolist() == [123456789]


def test_streams_and_graphs():
    w = [t.cuda() for t in world([8, 9, 0, 5], 5000, 10)]

    def step():
        return mx.verify_drafts(w[0], w[2], w[3], w[4], w[5], 9, w[1]) + mx.verify_drafts(w[0], *w[2:], 9)

    here = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(here, there))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for seed in range(5):
        w[5].copy_(torch.rand(w[5].shape, generator=torch.Generator().manual_seed(seed)))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_refusals():
    t = torch.ones(3, 10, device="cuda")
    i, cu, u = torch.zeros(3, dtype=torch.int32, device="cuda"), i32([0, 3]).cuda(), torch.zeros(3, 2, device="cuda")
    mx.verify_drafts(t, i, i, cu, u, 3, t)
    bad = [
        lambda: mx.verify_drafts(t.half(), i, i, cu, u, 3), lambda: mx.verify_drafts(t[0], i, i, cu, u, 3),
        lambda: mx.verify_drafts(t[:, ::2], i, i, cu, u, 3), lambda: mx.verify_drafts(t.cpu(), i, i, cu, u, 3),
        lambda: mx.verify_drafts(t, i, i, cu, u, 3, t.bfloat16()), lambda: mx.verify_drafts(t, i, i, cu, u, 3, t[:2]),
        lambda: mx.verify_drafts(t, i.long(), i, cu, u, 3), lambda: mx.verify_drafts(t, i[:2], i, cu, u, 3),
        lambda: mx.verify_drafts(t, i, i.long(), cu, u, 3), lambda: mx.verify_drafts(t, i, i, cu.long(), u, 3),
        lambda: mx.verify_drafts(t, i, i, cu[:0], u, 3), lambda: mx.verify_drafts(t, i, i, cu, u.double(), 3),
        lambda: mx.verify_drafts(t, i, i, cu, u[:2], 3), lambda: mx.verify_drafts(t, i, i, cu, u, 0),
        lambda: mx.verify_drafts(t, i, i, cu, u, 1025), lambda: mx.verify_drafts(t[:, :0], i, i, cu, u, 3),
        lambda: mx.verify_drafts(t, i, i, cu, u.view(2, 3), 3),
        lambda: mx.verify_drafts(t, i, i, torch.zeros(70000, dtype=torch.int32, device="cuda"), u, 3),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    torch.cuda.synchronize()
