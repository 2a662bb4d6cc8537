"""Append with the keys' norm and rotation on the way, bit for bit.

The reference forms the keys in 64 bits, rounds them to fp32 and appends them
with the cache's own reference. The kernel's 64-bit keys differ from those by
some 2^-50 of a head's largest element, which moves an fp32 rounding in one of
2^20 elements, and only one in 2^20 of those moves a code: the bytes here (some
millions) are the same but with a chance of about 2^-18."""
import math

import pytest
import torch

import draft_reference as dref
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


class Turned(World):
    """A world whose keys are normed and rotated on their way in."""

    def turn(self, rot, paired, norm, length, dtype, eps=1e-6):
        self.eps, self.paired, self.dtype, self.length = eps, paired, dtype, length
        self.angles = dref.table_of(length, rot, rot) if rot else None
        self.weight = (torch.randn(self.dim, generator=self.g) * 0.3 + 1).to(dtype) if norm else None

    def append(self, new, held, by=1.0, positions=None, edit=None, strided=False, behind=0):
        cu, place = [0], []
        for n, h in zip(new, held):
            cu.append(cu[-1] + n)
            place += range(h, h + n)
        k, v = self.numbers(cu[-1], self.heads, self.dtype, by), self.numbers(cu[-1], self.heads, self.dtype, by)
        if edit:
            edit(k, v)
        at = i32(place if positions is None else positions)
        keys = dref.heads(k, self.weight, self.eps,
                          (self.angles, at, self.paired) if self.angles is not None else None).float()
        cu, held = i32(cu), i32(held)
        ref.append(self.cpu, keys, v, self.table, cu, held)
        rotary = None
        if self.angles is not None:
            rotary = mx.Rotary(self.angles.cuda(), None if positions is None else at.cuda(), self.paired)
        more = torch.full((behind, self.heads, self.dim), math.nan, dtype=self.dtype)  # of no sequence
        gk, gv = torch.cat([k, more]).cuda(), torch.cat([v, more]).cuda()
        if strided:  # parts of one projection's rows
            rows = torch.cat([gk, gk, gv], 1)
            gk, gv = rows[:, self.heads:2 * self.heads], rows[:, 2 * self.heads:]
        mx.kv_append_rotary(self.gpu, gk, gv, self.table.cuda(), cu.cuda(), held.cuda(), rotary,
                            None if self.weight is None else self.weight.cuda(), self.eps)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dim,page,rot,paired,norm", [
    (64, 32, 64, False, True), (64, 64, 32, True, True), (64, 128, 48, False, False), (64, 256, 16, False, True),
    (128, 32, 128, True, False), (128, 64, 128, False, True), (128, 128, 112, False, True),
    (128, 256, 64, False, False), (128, 64, 16, True, True), (128, 32, 0, False, True)])
def test_prompts(dim, page, rot, paired, norm, dtype):
    totals = [0, 1, 31, 32, 33, 64, 129, 300, 513]
    w = Turned(totals, 2, dim, page, page + dim)
    w.turn(rot, paired, norm, 513, dtype)
    first = [t // 3 for t in totals]
    w.append(first, [0] * len(totals))
    w.same()
    second = [(t - f) // 2 for t, f in zip(totals, first)]
    w.append(second, first, by=50.0, strided=True)
    w.same()
    held = [f + s for f, s in zip(first, second)]
    w.append([t - h for t, h in zip(totals, held)], held, by=0.01)
    w.same()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("paired", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_few_tokens_at_a_time(dim, paired, norm):
    page = 64
    starts = [page - 7, 3, 2 * page - 2, page // 2 + 1]
    steps = [[1, 0, 1, 1], [4, 0, 2, 3], [3, 1, 4, 4], [1, 1, 1, 1], [4, 4, 4, 4], [2, 3, 1, 0]]
    totals = [s + sum(st[i] for st in steps) for i, s in enumerate(starts)]
    w = Turned(totals, 3, dim, page, dim + page)
    w.turn(dim // 2, paired, norm, max(totals), torch.bfloat16)
    w.append(starts, [0] * 4)
    held = list(starts)
    for t, new in enumerate(steps):
        w.append(new, held, by=2.0 ** ((t * 5) % 13 - 6))
        held = [h + n for h, n in zip(held, new)]
        w.same()


def test_given_positions():
    """Drafted tokens: several at one depth; the place in the cache is another."""
    w = Turned([50, 20], 2, 128, 32, 5)
    w.turn(128, False, True, 60, torch.bfloat16)
    w.append([40, 10], [0, 0])
    w.append([7, 5], [40, 10], positions=[40, 41, 41, 42, 42, 42, 43, 10, 11, 11, 12, 59])
    w.same()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("paired", [False, True])
def test_positions_outside_the_table(paired, norm):
    """Such a token makes its page NaN for every head, and no other page."""
    w = Turned([96], 2, 64, 32, 6)
    w.turn(64, paired, norm, 70, torch.float32)
    w.append([96], [0], positions=list(range(70)) + [70] + [-1] * 2 + [0] * 23)
    got = [t.cpu() for t in w.gpu]
    pages = w.table[0].long()
    assert bool((got[1][pages[2]] == 255).all())
    # the codes of a NaN's own sign are not defined: the other pages are
    for a, b in zip(w.cpu, got):
        assert torch.equal(a[pages[:2]], b[pages[:2]])
    assert torch.equal(w.cpu[3], got[3]) and torch.equal(w.cpu[1], got[1])
    fine = [i for i in range(32) if 64 + i < 70 or 64 + i > 72]
    assert torch.equal(w.cpu[0][pages[2]][:, fine], got[0][pages[2]][:, fine])


def test_sizes_of_numbers():
    """Keys whose squares leave 32 bits, zeros, infinity and NaN."""
    w = Turned([64] * 6, 1, 128, 32, 7)
    w.turn(64, False, True, 64, torch.float32, eps=0.0)

    def edit(k, v):
        k[0:64] *= 1e30
        k[64:128] *= 1e-30
        k[128:192] *= 1e37
        k[200, 0, 3] = math.inf
        k[260, 0, 70] = math.nan
        k[330] = 0  # and eps = 0

    w.append([64] * 6, [0] * 6, edit=edit)
    for a, b, name in zip(w.cpu, w.gpu, mx.KVCache._fields):
        b = b.cpu()
        if name == "k_codes":
            # of a head with a NaN or infinity the signs alone are kept, its own NaNs' are not defined
            for i in range(6):
                for j in range(2):
                    p = int(w.table[i, j])
                    if w.cpu[1][p, 0] != 255:
                        assert torch.equal(a[p], b[p])
        else:
            assert torch.equal(a, b), name


def test_nothing_on_the_way_is_the_plain_append():
    w = Turned([77, 3], 2, 64, 32, 8)
    w.turn(0, False, False, 1, torch.bfloat16)
    w.append([77, 3], [0, 0])
    w.same()


def test_tokens_behind_the_last_sequence():
    """A padded batch: tokens behind cu's last are dropped."""
    w = Turned([200, 90], 2, 64, 32, 10)
    w.turn(64, False, True, 400, torch.bfloat16)
    w.append([150, 77], [0, 0], behind=300)
    w.append([1, 1], [150, 77], behind=1)
    w.append([1, 1], [151, 78], behind=90)
    w.same()


def test_pages_outside_the_cache_and_offsets():
    w = Turned([64, 64], 2, 64, 32, 9)
    w.turn(64, False, True, 64, torch.bfloat16)
    w.append([10, 20], [0, 0])
    k = w.numbers(30, 2)
    table = torch.tensor([[-1, 2 ** 31 - 1], [-2 ** 31, w.cpu[0].shape[0]]], dtype=torch.int32)
    before = [t.clone() for t in w.gpu]
    rotary = mx.Rotary(w.angles.cuda())
    mx.kv_append_rotary(w.gpu, k.cuda(), k.cuda(), table.cuda(), i32([0, 12, 30]).cuda(), i32([5, 31]).cuda(), rotary,
                        w.weight.cuda())
    assert all(torch.equal(a, b) for a, b in zip(before, w.gpu))


@pytest.mark.parametrize("paired", [False, True])
@pytest.mark.parametrize("dim,page", [(64, 256), (128, 128), (128, 256)])
def test_scales_that_grow(dim, page, paired):
    """Kept codes of both kinds move to new bytes, a step and many, under new tokens of every slot."""
    totals = [page + 40, 3 * page, 37]
    w = Turned(totals, 2, dim, page, page)
    w.turn(dim, paired, False, max(totals), torch.bfloat16)
    held = [0, 0, 0]
    for t, step in enumerate((3, 16, 17, 1, 40, 33)):
        new = [min(step, n - h) for n, h in zip(totals, held)]
        w.append(new, held, by=2.0 ** (3 * t))
        w.same()
        held = [h + n for h, n in zip(held, new)]


def test_streams_and_graphs():
    """A captured append, replayed for other tokens, over a cache set back in between."""
    w = Turned([40, 90], 2, 128, 32, 10)
    w.turn(128, False, True, 128, torch.bfloat16)
    w.append([30, 70], [0, 0])
    start = [t.clone() for t in w.gpu]
    k = torch.zeros(30, 2, 128, dtype=torch.bfloat16, device="cuda")
    v, cu, held = k.clone(), i32([0, 10, 30]).cuda(), i32([30, 70]).cuda()
    rotary, weight, table = mx.Rotary(w.angles.cuda()), w.weight.cuda(), w.table.cuda()

    def call():
        mx.kv_append_rotary(w.gpu, k, v, table, cu, held, rotary, weight)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(3):
        for x in (k, v):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).to(x.dtype))
        got = []
        for f in (graph.replay, call):
            for a, b in zip(w.gpu, start):
                a.copy_(b)
            f()
            torch.cuda.synchronize()
            got.append([t.clone() for t in w.gpu])
        assert all(torch.equal(a, b) for a, b in zip(*got)), seed
        assert not torch.equal(got[0][0], start[0])


def test_refusals():
    cache = mx.kv_cache(4, 2, 64, 32)
    kv = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    i, t = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    angles = torch.zeros(8, 64, device="cuda")

    def call(k=kv, v=kv, table=t, cu=i, lengths=i[:1], **more):
        mx.kv_append_rotary(cache, k, v, table, cu, lengths, **more)

    call(rotary=mx.Rotary(angles), weight=w)
    bad = [
        dict(weight=w.float()), dict(weight=w[:32].contiguous()), dict(eps=-1.0), dict(eps=math.inf),
        dict(rotary=mx.Rotary(angles.half())), dict(rotary=mx.Rotary(angles[:, :24].contiguous())),
        dict(rotary=mx.Rotary(torch.zeros(8, 128, device="cuda"))), dict(rotary=mx.Rotary(angles[:0])),
        dict(rotary=mx.Rotary(angles, i)), dict(rotary=mx.Rotary(angles, i[:1].long())),
        dict(rotary=mx.Rotary(angles[0])), dict(rotary=mx.Rotary(angles.cpu())),
        dict(k=kv[..., ::2]), dict(v=kv.float()), dict(k=kv[:, :1], v=kv[:, :1]), dict(table=t.long()),
        dict(cu=i[:1]), dict(lengths=i),
    ]
    for more in bad:
        with pytest.raises(ValueError):
            call(**more)
    torch.cuda.synchronize()
