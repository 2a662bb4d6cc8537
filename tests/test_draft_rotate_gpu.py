"""Norms per head with the rotation, and their gradients, against 64 bits.

Tolerances. The kernels form the norm and the rotation in 64 bits and round to
32, then (bfloat16) to 16: a result is off by half a step of each, relative
2^-24 and 2^-8, by the table's entries not at all (both sides read the same
ones), and by 64-bit roundings of the pair's members, below 2^-48 of their
size. A gradient's elements are the same: its cancelling sums are in 64 bits.
Below 2^-126 steps do not shrink with the number any more: bfloat16's are 2^-133
there (7 bits behind the point of 2^-126), fp32's 2^-149, half of which is off
by more than 2^-8 (2^-24) of a small result.
dweight adds fp32 terms: each is rounded once, and passes at most as many
additions as its thread makes in a row plus 40 for the trees behind them."""
import pytest
import torch

import draft_reference as ref
import microscaling_fp4_block_mx_amd as mx

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


def inputs(tokens, q_heads, k_heads, dim, dtype, seed=0, norm=True):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(tokens, q_heads + 2 * k_heads, dim, generator=g).to(dtype)
    w = [(torch.randn(dim, generator=g) * 0.3 + 1).to(dtype) if norm else None for _ in range(2)]
    pos = torch.randint(0, 50, (tokens,), generator=g, dtype=torch.int32)
    return qkv, w, pos


def on_gpu(t):
    return None if t is None else t.cuda()


def near(got, want, dtype, reach=None):
    """|got - want| within the roundings; `reach`: the size of what went into a result."""
    got, want = got.cpu().double(), want.double()
    half = 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    tiny = 2.0 ** -126 if reach is None else 2.0 ** -48 * reach + 2.0 ** -134 + 2.0 ** -150
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    off = (got - want).abs() - half * want.abs() - tiny
    assert float(torch.nan_to_num(off, -1.0).max()) <= 0.0, float(torch.nan_to_num(off, -1.0).max())


CASES = [  # tokens, q heads, k heads, dim, rot, paired, norm
    (1, 1, 1, 64, 64, False, True), (5, 32, 8, 128, 128, False, True), (3, 2, 1, 256, 256, False, True),
    (7, 5, 3, 64, 32, True, True), (33, 3, 2, 128, 32, False, True), (2, 40, 8, 128, 64, True, False),
    (129, 4, 4, 256, 64, False, False), (65, 17, 1, 64, 16, False, True), (4, 33, 11, 128, 128, True, True),
    (300, 9, 3, 256, 240, True, True), (10, 1, 7, 128, 112, False, True), (6, 3, 3, 64, 48, False, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,q_heads,k_heads,dim,rot,paired,norm", CASES)
def test_forward(tokens, q_heads, k_heads, dim, rot, paired, norm, dtype):
    qkv, w, pos = inputs(tokens, q_heads, k_heads, dim, dtype, 1, norm)
    table = ref.table_of(50, rot)
    rows = qkv.cuda()
    before = rows.clone()
    rotary = mx.Rotary(table.cuda(), pos.cuda(), paired)
    q, k = mx.norm_rotate(rows[:, :q_heads], rows[:, q_heads:q_heads + k_heads], on_gpu(w[0]),
                          on_gpu(w[1]), rotary, EPS)
    assert q.is_contiguous() and k.is_contiguous() and q.dtype == dtype and torch.equal(rows, before)
    for got, x, weight in ((q, qkv[:, :q_heads], w[0]), (k, qkv[:, q_heads:q_heads + k_heads], w[1])):
        near(got, ref.heads(x, weight, EPS, (table, pos, paired)), dtype,
             ref.heads(x, weight, EPS, None).abs().amax())
    # in place, and q alone, are the same bits
    q2, k2 = mx.norm_rotate(rows[:, :q_heads], rows[:, q_heads:q_heads + k_heads], on_gpu(w[0]),
                            on_gpu(w[1]), rotary, EPS, out_q=rows[:, :q_heads],
                            out_k=rows[:, q_heads:q_heads + k_heads])
    assert q2.data_ptr() == rows.data_ptr()
    assert torch.equal(q2, q) and torch.equal(k2, k)
    assert torch.equal(rows[:, q_heads + k_heads:], before[:, q_heads + k_heads:])
    alone, none = mx.norm_rotate(before[:, :q_heads], None, on_gpu(w[0]), None, rotary, EPS)
    assert none is None and torch.equal(alone, q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,q_heads,k_heads,dim,rot,paired,norm", CASES)
def test_backward(tokens, q_heads, k_heads, dim, rot, paired, norm, dtype):
    qkv, w, pos = inputs(tokens, q_heads, k_heads, dim, dtype, 2, norm)
    table = ref.table_of(50, rot)
    g = torch.Generator().manual_seed(3)
    dy = torch.randn(tokens, q_heads + k_heads, dim, generator=g).to(dtype)
    rows, grads = qkv.cuda(), dy.cuda()
    rotary = mx.Rotary(table.cuda(), pos.cuda(), paired)
    x = [qkv[:, :q_heads], qkv[:, q_heads:q_heads + k_heads]]
    d = [dy[:, :q_heads], dy[:, q_heads:]]
    args = (grads[:, :q_heads], rows[:, :q_heads], grads[:, q_heads:], rows[:, q_heads:q_heads + k_heads],
            on_gpu(w[0]), on_gpu(w[1]), rotary, EPS)
    dq, dk, dwq, dwk = mx.norm_rotate_backward(*args)
    for got, dweight, i in ((dq, dwq, 0), (dk, dwk, 1)):
        want, dw, mag = ref.heads_backward(d[i], x[i], w[i], EPS, (table, pos, paired))
        near(got, want, dtype, want.abs().amax())
        assert (dweight is None) == (w[i] is None)
        if dweight is not None:
            in_a_row = tokens * (q_heads + k_heads)
            bound = (in_a_row + 40) * 2.0 ** -24 * mag
            assert bool(((dweight.cpu().double() - dw).abs() <= bound).all())
    again = mx.norm_rotate_backward(*args)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip((dq, dk, dwq, dwk), again))


def test_backward_against_differences():
    """The gradient of a weighted sum of outputs, by central differences in 64 bits."""
    tokens, heads, dim, rot = 2, 2, 64, 32
    qkv, w, pos = inputs(tokens, heads, heads, dim, torch.float32, 4)
    table, c = ref.table_of(50, rot), torch.randn(tokens, heads, dim, generator=torch.Generator().manual_seed(5))
    dq, _, dw, _ = mx.norm_rotate_backward(c.cuda(), qkv[:, :heads].contiguous().cuda(), None, None, w[0].cuda(),
                                           None, mx.Rotary(table.cuda(), pos.cuda()), EPS)

    def loss(x, weight):
        return float((ref.heads(x, weight, EPS, (table, pos, False)) * c.double()).sum())

    x0, w0, h = qkv[:, :heads].double(), w[0].double(), 1e-5
    for i in (0, 13, 31, 32, 63):
        for t in range(tokens):
            up, down = x0.clone(), x0.clone()
            up[t, 1, i] += h
            down[t, 1, i] -= h
            # the difference's own error: h^2 times a third derivative of about 1, and 2^-52 / h
            assert abs((loss(up, w0) - loss(down, w0)) / (2 * h) - float(dq[t, 1, i])) <= 1e-6
        up, down = w0.clone(), w0.clone()
        up[i] += h
        down[i] -= h
        assert abs((loss(x0, up) - loss(x0, down)) / (2 * h) - float(dw[i])) <= 2e-6


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("paired", [False, True])
def test_sizes_of_numbers(dtype, paired):
    """Heads whose squares leave 32 bits, zeros, and what is not a number."""
    g = torch.Generator().manual_seed(6)
    tokens, dim = 9, 128
    x = torch.randn(tokens, 1, dim, generator=g)
    scale = torch.tensor([1e30, 1e-30, 3e38 / 6, 1e-37, 0.0, 1.0, 1.0, 1.0, 1.0])
    x = (x * scale[:, None, None]).to(dtype)
    x[6, 0, 3], x[7, 0, 70] = torch.inf, torch.nan
    w = torch.ones(dim).to(dtype)
    pos = torch.arange(tokens, dtype=torch.int32)
    pos[8] = 50
    table = ref.table_of(50, 64)
    for eps in (0.0, EPS):
        y, _ = mx.norm_rotate(x.cuda(), None, w.cuda(), None, mx.Rotary(table.cuda(), pos.cuda(), paired), eps)
        want = ref.heads(x, w, eps, (table, pos, paired))
        near(y, want, dtype)
        dy = torch.randn(tokens, 1, dim, generator=g).to(dtype)
        dx, _, _, _ = mx.norm_rotate_backward(dy.cuda(), x.cuda(), None, None, w.cuda(), None,
                                              mx.Rotary(table.cuda(), pos.cuda(), paired), eps)
        want = ref.heads_backward(dy, x, w, eps, (table, pos, paired))[0]
        fine = want.abs() < 3.3e38  # past it the result may round to infinity
        near(torch.where(fine, dx.cpu().double(), 0), torch.where(fine, want, 0), dtype,
             torch.where(fine, want, 0).abs().amax((1, 2), keepdim=True))


def test_positions_outside_the_table():
    x = torch.randn(4, 2, 64, generator=torch.Generator().manual_seed(7))
    pos = torch.tensor([-1, 0, 9, 10], dtype=torch.int32)
    table = ref.table_of(10, 32)
    y, _ = mx.norm_rotate(x.cuda(), rotary=mx.Rotary(table.cuda(), pos.cuda()))
    y = y.cpu()
    assert bool(y[0, :, :32].isnan().all()) and bool(y[3, :, :32].isnan().all())
    assert torch.equal(y[:, :, 32:], x[:, :, 32:]) and not bool(y[1:3].isnan().any())


def test_norm_alone_and_nothing():
    x = torch.randn(6, 3, 64, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    w = torch.rand(64, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    y, _ = mx.norm_rotate(x.cuda(), None, w.cuda())
    near(y, ref.heads(x, w, 1e-6, None), torch.bfloat16)
    y, _ = mx.norm_rotate(x.cuda())
    assert torch.equal(y.cpu(), x)
    # one of the two with a weight
    q, k = mx.norm_rotate(x.cuda(), x.cuda(), None, w.cuda())
    assert torch.equal(q.cpu(), x)
    near(k, ref.heads(x, w, 1e-6, None), torch.bfloat16)
    dq, dk, dwq, dwk = mx.norm_rotate_backward(x.cuda(), x.cuda(), x.cuda(), x.cuda(), None, w.cuda())
    assert torch.equal(dq.cpu(), x) and dwq is None
    want, dw, mag = ref.heads_backward(x, x, w, 1e-6, None)
    near(dk, want, torch.bfloat16, want.abs().amax())
    assert bool(((dwk.cpu().double() - dw).abs() <= 80 * 2.0 ** -24 * mag).all())


def test_no_tokens():
    x = torch.empty(0, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, k = mx.norm_rotate(x, x, w, w)
    assert y.shape == k.shape == (0, 2, 64)
    dq, dk, dwq, dwk = mx.norm_rotate_backward(x, x, x, x, w, w)
    assert dq.shape == (0, 2, 64) and not bool(dwq.any()) and not bool(dwk.any())
    assert dwq.shape == dwk.shape == (64,)


def test_many_tokens():
    """More rows of partial sums than a thread adds at once, and every workgroup with several tokens."""
    tokens = 9000
    qkv, w, pos = inputs(tokens, 2, 1, 64, torch.float32, 10)
    table = ref.table_of(50, 64)
    dy = torch.randn(tokens, 3, 64, generator=torch.Generator().manual_seed(11))
    rotary = mx.Rotary(table.cuda(), pos.cuda())
    _, _, dwq, dwk = mx.norm_rotate_backward(dy[:, :2].cuda(), qkv[:, :2].cuda(), dy[:, 2:].cuda(), qkv[:, 2:3].cuda(),
                                             w[0].cuda(), w[1].cuda(), rotary, EPS)
    for got, i, at in ((dwq, 0, slice(0, 2)), (dwk, 1, slice(2, 3))):
        _, dw, mag = ref.heads_backward(dy[:, at], qkv[:, at], w[i], EPS, (table, pos, False))
        assert bool(((got.cpu().double() - dw).abs() <= 200 * 2.0 ** -24 * mag).all())
    y, k = mx.norm_rotate(qkv[:, :2].cuda(), qkv[:, 2:3].cuda(), w[0].cuda(), w[1].cuda(), rotary, EPS)
    near(y, ref.heads(qkv[:, :2], w[0], EPS, (table, pos, False)), torch.float32, 4.0)
    near(k, ref.heads(qkv[:, 2:3], w[1], EPS, (table, pos, False)), torch.float32, 4.0)


def test_rows_past_32_bits():
    """More than 2^31 elements, forward in place and backward, the last tokens against 64 bits."""
    tokens, heads, dim = 131100, 128, 128
    assert tokens * heads * dim > 2 ** 31
    x = torch.empty(tokens, heads, dim, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for at in range(0, tokens, 8192):
        x[at:at + 8192].normal_(generator=g)
    w = (torch.rand(dim, generator=torch.Generator().manual_seed(2)) + 0.5).bfloat16()
    pos = (torch.arange(tokens, dtype=torch.int32) % 50)
    table = ref.table_of(50, 128)
    rotary = mx.Rotary(table.cuda(), pos.cuda())
    some = [0, 65535, tokens - 9, tokens - 1]
    kept = x[some].cpu()
    dx, _, dw, _ = mx.norm_rotate_backward(x, x, None, None, w.cuda(), None, rotary)
    want = ref.heads_backward(kept, kept, w, EPS, (table, pos[some], False))[0]
    near(dx[some], want, torch.bfloat16, want.abs().amax())
    assert bool(torch.isfinite(dw).all())
    del dx
    mx.norm_rotate(x, None, w.cuda(), None, rotary, EPS, out_q=x)
    near(x[some], ref.heads(kept, w, EPS, (table, pos[some], False)), torch.bfloat16, 8.0)


def test_tables_past_32_bits():
    """A table of more than 2^31 bytes, positions at its end."""
    length = (1 << 23) + 5
    table = torch.zeros(length, 128, device="cuda")
    table[:, :64] = 1.0
    last = ref.table_of(4, 128)
    table[-4:] = last.cuda()
    x = torch.randn(4, 2, 128, generator=torch.Generator().manual_seed(3))
    pos = torch.arange(length - 4, length, dtype=torch.int32)
    y, _ = mx.norm_rotate(x.cuda(), rotary=mx.Rotary(table, pos.cuda()))
    near(y, ref.heads(x, None, 0.0, (last, torch.arange(4), False)), torch.float32, 4.0)


def test_streams_and_graphs():
    """Replays of a captured pass, forward and backward, with eager work between them."""
    qkv, w, pos = inputs(70, 4, 2, 128, torch.bfloat16, 12)
    rows, table = qkv.cuda(), ref.table_of(50, 128).cuda()
    w = [t.cuda() for t in w]
    pos = pos.cuda()
    dy = torch.randn(70, 6, 128, device="cuda").to(torch.bfloat16)

    def both(x):
        rotary = mx.Rotary(table, pos)
        out = mx.norm_rotate(x[:, :4], x[:, 4:6], *w, rotary)
        return out + mx.norm_rotate_backward(dy[:, :4], x[:, :4], dy[:, 4:], x[:, 4:6], *w, rotary)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        there = both(rows)
    side.synchronize()
    here = both(rows)
    assert all(torch.equal(a, b) for a, b in zip(here, there))
    x = rows.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both(x)
    for seed in range(4):
        x.copy_(torch.randn(rows.shape, generator=torch.Generator().manual_seed(seed)).to(x.dtype))
        graph.replay()
        want = both(x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want)), seed


def test_refusals():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    t, p = torch.zeros(8, 64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    wide = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: mx.norm_rotate(x.half()),
        lambda: mx.norm_rotate(x[:, :, :32].contiguous()),              # heads of 32
        lambda: mx.norm_rotate(x[:, :, ::2]),
        lambda: mx.norm_rotate(x.transpose(0, 1)),                      # heads not adjacent
        lambda: mx.norm_rotate(x, wide),
        lambda: mx.norm_rotate(x, x.float()),
        lambda: mx.norm_rotate(x, x[:3]),
        lambda: mx.norm_rotate(x, None, w.float()),
        lambda: mx.norm_rotate(x, None, w[:32].contiguous()),
        lambda: mx.norm_rotate(x, None, None, w),                       # k's weight without k
        lambda: mx.norm_rotate(x, eps=-1.0),
        lambda: mx.norm_rotate(x, rotary=mx.Rotary(t)),                 # no positions
        lambda: mx.norm_rotate(x, rotary=mx.Rotary(t, p.long())),
        lambda: mx.norm_rotate(x, rotary=mx.Rotary(t, p[:3])),
        lambda: mx.norm_rotate(x, rotary=mx.Rotary(t.double(), p)),
        lambda: mx.norm_rotate(x, rotary=mx.Rotary(t[:, :40].contiguous(), p)),
        lambda: mx.norm_rotate(x, rotary=mx.Rotary(t[:0], p)),
        lambda: mx.norm_rotate(x, rotary=mx.Rotary(torch.zeros(8, 128, device="cuda"), p)),
        lambda: mx.norm_rotate(x, out_q=x.float()),
        lambda: mx.norm_rotate(x, out_q=x[:3]),
        lambda: mx.norm_rotate(x[:3], out_q=x[1:]),                     # shifted by a token
        lambda: mx.norm_rotate(x, out_k=x),
        lambda: mx.norm_rotate(x.cpu()),
        lambda: mx.norm_rotate(x, x, out_q=wide[:, :, :64]),
        lambda: mx.norm_rotate_backward(x, x, x),
        lambda: mx.norm_rotate_backward(x[:3], x),
        lambda: mx.norm_rotate_backward(x.float(), x),
        lambda: mx.norm_rotate_backward(x, x, None, None, None, w),
        lambda: mx.rotary_table(8, 24),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    torch.cuda.synchronize()


def test_table():
    t = mx.rotary_table(70000, 64, 500000.0).cpu()
    p = torch.arange(70000, dtype=torch.float64)[:, None]
    a = p * 500000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    assert t.shape == (70000, 64) and t.dtype == torch.float32
    assert float((t[:, :32] - a.cos()).abs().max()) <= 2.0 ** -24
    assert float((t[:, 32:] - a.sin()).abs().max()) <= 2.0 ** -24
