"""Batches whose first offset is not 0: the tokens before it belong to no
sequence, so units of work before the first sequence's find none."""
import math

import pytest
import torch

import layer_reference as ref
import microscaling_fp4_block_mx_amd as mx
from test_layer_kv_gpu import World, i32
from test_layer_split_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("batch", [1, 2, 70])
@pytest.mark.parametrize("n", [1, 40])
def test_append(n, batch):
    first = 100  # more than three pages of tokens
    w = World([64] * batch, 2, 64, 32, 22)
    cu, held = i32([first + i * n for i in range(batch + 1)]), i32([0] * batch)
    k, v = w.numbers(first + batch * n, 2), w.numbers(first + batch * n, 2)
    ref.append(w.cpu, k, v, w.table, cu, held)
    print("append", n, batch, flush=True)
    mx.kv_append(w.gpu, k.cuda(), v.cuda(), w.table.cuda(), cu.cuda(), held.cuda())
    w.same()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("first,n,longest", [(20, 1, 100), (20, 1, 2500), (100, 1, 100), (100, 40, 2500)])
def test_attention(first, n, longest, dim):
    """Either kernel, split or not."""
    lengths = [longest, 64]
    w = World(lengths, 2, dim, 32, 23)
    w.append(lengths, [0, 0])
    cu = i32([first, first + n, first + 2 * n])
    q = w.numbers(first + 2 * n, 4)
    print("attention", first, n, longest, dim, flush=True)
    out = mx.kv_attention(q.cuda(), w.gpu, w.table.cuda(), cu.cuda(), i32(lengths).cuda()).cpu()
    want, mag, reach = ref.attention(q, w.cpu, w.table, cu, i32(lengths), 1 / math.sqrt(dim))
    check(out[first:], want[first:], mag[first:], reach[first:])
