"""The paged 8-bit key/value cache and its attention against 64 bits: ragged
batches, page and tile edges, growing scales, what old memory holds, NaN,
rows that see nothing, strides, streams and graphs."""
import math

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


class World:
    """A CPU cache, its GPU twin, and page tables for sequences of these final lengths."""

    def __init__(self, totals, heads, dim, page, seed, junk=True):
        self.g = torch.Generator().manual_seed(seed)
        need = [-(-t // page) for t in totals]
        pool = sum(need) + 2
        self.heads, self.dim, self.page = heads, dim, page
        shape = [(pool, heads, page, dim), (pool, heads), (pool, heads, dim, page), (pool, heads)]
        # what the memory held before: any bytes, NaN codes and scales among them
        self.cpu = [torch.randint(0, 256, s, generator=self.g, dtype=torch.uint8) if junk
                    else torch.zeros(s, dtype=torch.uint8) for s in shape]
        order = torch.randperm(pool, generator=self.g)
        self.table = torch.zeros((len(totals), max(1, max(need))), dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n].int()
            at += n
        self.gpu = mx.KVCache(*(t.cuda() for t in self.cpu))

    def numbers(self, tokens, heads, dtype=torch.bfloat16, by=1.0):
        return (torch.randn(tokens, heads, self.dim, generator=self.g) * by).to(dtype)

    def append(self, new, held, dtype=torch.bfloat16, by=1.0, edit=None):
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        k, v = self.numbers(cu[-1], self.heads, dtype, by), self.numbers(cu[-1], self.heads, dtype, by)
        if edit:
            edit(k, v)
        cu, held = i32(cu), i32(held)
        ref.append(self.cpu, k, v, self.table, cu, held)
        mx.kv_append(self.gpu, k.cuda(), v.cuda(), self.table.cuda(), cu.cuda(), held.cuda())

    def same(self):
        for a, b, name in zip(self.cpu, self.gpu, mx.KVCache._fields):
            assert torch.equal(a, b.cpu()), name


@pytest.mark.parametrize("page", [32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_append(page, dim, dtype):
    totals = [0, 1, 31, 32, 33, 64, 129, 300, 513]
    w = World(totals, 2, dim, page, page + dim)
    first = [t // 3 for t in totals]
    w.append(first, [0] * len(totals), dtype)
    w.same()
    # the rest in two steps, larger and then smaller values
    second = [(t - f) // 2 for t, f in zip(totals, first)]
    w.append(second, first, dtype, by=50.0)
    w.same()
    held = [f + s for f, s in zip(first, second)]
    w.append([t - h for t, h in zip(totals, held)], held, dtype, by=0.01)
    w.same()


@pytest.mark.parametrize("heads", [1, 3, 8])
def test_append_token_by_token(heads):
    """Single tokens whose magnitude grows and shrinks, so that a page's scale
    moves many times; an idle sequence between."""
    w = World([70, 40, 70], heads, 64, 32, heads)
    for t in range(70):
        w.append([1, 0, 1], [t, 40, t], by=2.0 ** ((t * 7) % 23 - 11))
    w.same()


def test_append_nonfinite_and_zeros():
    w = World([40, 40, 40], 2, 128, 32, 3)
    w.append([20, 20, 20], [0, 0, 0])

    def edit(k, v):
        k[0, 0, 5] = math.nan          # its page's keys, head 0
        v[5, 1, 7] = -math.inf         # sequence 1's first page, head 1
        k[10:15] = 0
    w.append([5, 5, 5], [20, 20, 20], edit=edit)
    w.same()
    w.append([15, 15, 15], [25, 25, 25])   # NaN stays in the page; the next one starts anew
    w.same()

    z = World([64], 2, 64, 64, 4)
    z.append([10], [0], edit=lambda k, v: (k.zero_(), v.zero_()))
    z.append([10], [10])
    z.same()


def test_append_drops_what_the_table_has_no_room_for():
    w = World([64], 1, 64, 32, 5)
    w.append([100], [20])
    w.same()


def split(total, parts):
    return [total * (i + 1) // parts - total * i // parts for i in range(parts)]


def run_attention(w, new, lengths, group, scale=None, strided=False, max_length=0, big=1.0):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = w.numbers(cu[-1], w.heads * group, by=big)
    cu, lengths = i32(cu), i32(lengths)
    qg = q.cuda()
    if strided:
        wide = torch.full((cu[-1], w.heads * (group + 2), w.dim), math.nan, dtype=torch.bfloat16,
                          device="cuda")
        wide[:, :w.heads * group] = qg
        qg = wide[:, :w.heads * group]
    got = mx.kv_attention(qg, w.gpu, w.table.cuda(), cu.cuda(), lengths.cuda(), scale, max_length)
    used = 1 / math.sqrt(w.dim) if scale is None else scale
    want, mag, reach = ref.attention(q, w.cpu, w.table, cu, lengths, used)
    return got.cpu(), want, mag, reach


def check_attention(got, want, mag, reach):
    """Half a step of bf16; weights to 2^-9 above and below the line; scores
    off by at most 2^-10 of sum |q k| (see the product's bound), twice."""
    nan = torch.isnan(want)
    assert torch.equal(nan, torch.isnan(got))
    eps = 2.0 ** -8 + 2 * 2.0 ** -10 * reach
    tol = 2.0 ** -8 * want.abs() + eps[..., None] * mag
    off = (got.double() - want).abs()
    assert bool((off <= tol)[~nan].all()), float((off / (mag + 1e-30))[~nan].max())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [32, 64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 4, 8])
def test_attention_single_tokens(dim, page, group):
    lengths = [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 257, 700]
    w = World(lengths, 2, dim, page, dim + page + group)
    w.append(lengths, [0] * len(lengths))
    check_attention(*run_attention(w, [1] * len(lengths), lengths, group))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 5, 16, 17, 40])
def test_attention_several_tokens(dim, group):
    """Few new tokens and prompts in one batch; blocks of rows that end inside a token group."""
    new, lengths = [1, 5, 0, 40, 130], [130, 5, 64, 170, 131]
    w = World(lengths, 2, dim, 64, group)
    w.append(lengths, [0] * len(lengths))
    check_attention(*run_attention(w, new, lengths, group))
    check_attention(*run_attention(w, [2, 1, 1, 3, 1], lengths, group))


@pytest.mark.parametrize("page", [32, 64, 256])
def test_attention_prompts(page):
    new, lengths = [300, 1, 129, 128, 127], [300, 700, 200, 128, 128]
    w = World(lengths, 1, 128, page, page)
    w.append(lengths, [0] * len(lengths))
    check_attention(*run_attention(w, new, lengths, 2, strided=True))


@pytest.mark.parametrize("new", [1, 60])
def test_attention_rows_that_see_nothing(new):
    """Empty sequences, and more new tokens than the sequence holds."""
    lengths = [0, 50, 0, 20]
    w = World([64] * 4, 2, 64, 32, 1)
    w.append(lengths, [0] * 4)
    got, want, mag, reach = run_attention(w, [new] * 4, lengths, 4)
    check_attention(got, want, mag, reach)
    assert bool((got[:new] == 0).all())


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_nan_reaches_only_rows_that_see_it(new, dim):
    """A NaN value or key late in the sequence: earlier rows stay finite."""
    w = World([200, 200, 200], 1, dim, 32, 9)
    for which in (0, 1):
        def edit(k, v):
            (k, v)[which][190, 0, 3] = math.nan      # sequence 0, position 190
        w.append([200] * 3, [0] * 3, edit=edit)
        got, want, mag, reach = run_attention(w, [new] * 3, [200] * 3, 2)
        if which == 1:
            # the page's values are all NaN to rows that see any of its tokens
            assert bool(torch.isnan(want[new - 1]).all())
        check_attention(got, want, mag, reach)


@pytest.mark.parametrize("new", [1, 100])
def test_attention_large_scores_and_scales(new):
    """Scores in the hundreds (one weight takes all), pages whose scales lie
    2^24 apart, a softmax scale of its own."""
    lengths = [257, 140]
    w = World(lengths, 2, 128, 64, 12)
    held = [0, 0]
    for part in range(4):
        step = [split(n, 4)[part] for n in lengths]
        w.append(step, held, by=2.0 ** (8 * part - 16))
        held = [h + s for h, s in zip(held, step)]
    check_attention(*run_attention(w, [new] * 2, lengths, 4, scale=0.3))
    check_attention(*run_attention(w, [new] * 2, lengths, 4, big=1e-20))
    check_attention(*run_attention(w, [new] * 2, lengths, 4, scale=1e-6, big=30.0))


@pytest.mark.parametrize("new", [1, 64])
def test_attention_nonfinite_queries(new):
    w = World([100, 100], 1, 64, 32, 2)
    w.append([100, 100], [0, 0])
    q = w.numbers(2 * new, 2)
    q[0, 0, 3], q[new, 1, 5] = math.nan, math.inf
    out = mx.kv_attention(q.cuda(), w.gpu, w.table.cuda(), i32([0, new, 2 * new]).cuda(),
                          i32([100, 100]).cuda()).cpu()
    nan = torch.isnan(out).any(2)
    want = torch.zeros_like(nan)
    want[0, 0] = want[new, 1] = True
    assert torch.equal(nan, want)


def test_attention_bound_on_lengths_only_steers():
    lengths = [3000, 1, 2000]
    w = World(lengths, 1, 64, 64, 8)
    w.append(lengths, [0, 0, 0])
    state = w.g.get_state()
    outs = []
    for bound in (0, 3000, 100, 1):
        w.g.set_state(state)
        got, want, mag, reach = run_attention(w, [1, 1, 1], lengths, 4, max_length=bound)
        check_attention(got, want, mag, reach)
        outs.append(got)


def test_attention_past_32_bit_offsets():
    """Pages whose codes lie more than 2^32 bytes into the cache."""
    pages, heads, dim, page = 70000, 8, 128, 64
    cache = mx.kv_cache(pages, heads, dim, page)
    assert cache.k_codes.numel() > 1 << 32
    w = World([300, 65], heads, dim, page, 6)
    w.append([300, 65], [0, 0])
    far = w.table + (pages - 20)
    g = torch.Generator().manual_seed(6)
    cu, held = i32([0, 300, 365]), i32([0, 0])
    w2 = World([300, 65], heads, dim, page, 6)
    k, v = w2.numbers(365, heads), w2.numbers(365, heads)
    mx.kv_append(cache, k.cuda(), v.cuda(), far.cuda(), cu.cuda(), held.cuda())
    assert torch.equal(cache.k_scales[-20:][w.table[0].long().cuda()],
                       w.gpu.k_scales[w.table[0].long().cuda()])
    for new in ([1, 1], [200, 60]):
        n = sum(new)
        q = torch.randn(n, heads * 2, dim, generator=g).bfloat16().cuda()
        c = i32([0, new[0], n]).cuda()
        lengths = i32([300, 65]).cuda()
        a = mx.kv_attention(q, cache, far.cuda(), c, lengths)
        b = mx.kv_attention(q, w.gpu, w.table.cuda(), c, lengths)
        assert torch.equal(a, b)


def test_stream_and_graph():
    """On a stream of its own, and in a graph that is replayed between eager work."""
    lengths = [1300, 200]
    w = World([l + 8 for l in lengths], 2, 128, 64, 11)
    w.append(lengths, [0, 0])
    q, k, v = w.numbers(2, 8).cuda(), w.numbers(2, 2).cuda(), w.numbers(2, 2).cuda()
    table, cu = w.table.cuda(), i32([0, 1, 2]).cuda()
    held, after = i32(lengths).cuda(), i32([l + 1 for l in lengths]).cuda()

    def step(out):
        mx.kv_append(w.gpu, k, v, table, cu, held)
        return mx.kv_attention(q, w.gpu, table, cu, after, max_length=1400, out=out)

    want = step(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    with torch.cuda.stream(side):
        step(out)
        side.synchronize()
        assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(out)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        q.copy_(w.numbers(2, 8))
        eager = step(None)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
