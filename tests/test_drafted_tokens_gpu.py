"""The example of serving with drafted tokens runs; what its cache holds after a
drafted step is what plain steps over the taken tokens give."""
import pytest
import torch

import microscaling_fp4_block_mx_amd as mx
from examples import drafted_tokens as ex

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mx.load_library()
    yield
    torch.cuda.synchronize()


def test_example_runs(capsys):
    ex.main()
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 8 and lines[0].startswith("step 0") and lines[-1].endswith("3 sequences")


def test_paths_are_paths_of_the_tree():
    model = ex.Model(vocab=200, hidden=256, layers=1)
    g = torch.Generator(device="cuda").manual_seed(4)
    pairs = torch.softmax(torch.randn(200, 200, generator=g, device="cuda") * 3, 1)
    for i, (path, count, token) in enumerate(ex.serve(model, [[1, 2, 3], [9], [4] * 40, [7, 8]], 8, pairs, temperature=3.0)):
        assert bool(((token >= 0) & (token < 200)).all())
        for p, n in zip(path.tolist(), count.tolist()):
            taken = p[:n]
            assert taken[0] == 0 and all(x == -1 for x in p[n:])
            assert all(ex.TREE[b] == a for a, b in zip(taken, taken[1:]))
            assert i > 0 or n == 1


def test_a_tree_reads_as_its_branches_do():
    """Probabilities at a tree's nodes against those of each branch read as a chain by
    causal attention from a cache of its own. The pages' bytes are larger where
    other branches' tokens are, so each cached number is off by at most 2^-4 of
    itself on either side: as in the decoder layer's test, 6 / 16 of a vector's norm
    bounds the logits of one layer."""
    model = ex.Model(vocab=300, hidden=256, layers=1, seed=5)
    prompt = [11, 22, 33, 44, 55]
    tree, ids = ex.TREE, [7, 70, 71, 72, 73, 74, 75]

    def start():
        caches, pages = model.caches(1, 64)
        cu, held, lengths = pages.step([len(prompt)])
        model(torch.tensor(prompt, dtype=torch.int32, device="cuda"), caches, pages.table, cu, held, lengths,
              torch.arange(5, dtype=torch.int32, device="cuda"))
        return caches, pages, lengths

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    caches, pages, held = start()
    mask, depth = mx.tree_mask([tree])
    p = model(i32(ids), caches, pages.table, i32([0, 7]), held, held + 7, depth + 5, mask)
    for leaf in (4, 5, 6):
        branch = [leaf]
        while tree[branch[0]] >= 0:
            branch.insert(0, tree[branch[0]])
        caches, pages, held = start()
        n = len(branch)
        want = model(i32([ids[j] for j in branch]), caches, pages.table, i32([0, n]), held, held + n,
                     torch.arange(5, 5 + n, dtype=torch.int32, device="cuda"))
        a, b = torch.log(p[branch]), torch.log(want)
        a, b = a - a.mean(1, keepdim=True), b - b.mean(1, keepdim=True)
        assert float(((a - b).norm(dim=1) / b.norm(dim=1)).max()) <= 6 / 16
