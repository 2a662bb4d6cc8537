"""Host side of positions and drafted tokens, without a GPU: the C ABI's
argument checks under sanitizers, and the tensor helpers' refusals."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import draft_reference as ref
import microscaling_fp4_block_mx_amd as mx
from conftest import ROOT
from microscaling_fp4_block_mx_amd import draft

CSRC = os.path.join(ROOT, "microscaling_fp4_block_mx_amd", "csrc")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(mx.LIB_PATH):
        from microscaling_fp4_block_mx_amd import build
        build.build()
    return mx.load_library()


@pytest.mark.parametrize("flags", [["-fsanitize=address,undefined", "-fno-sanitize-recover=all"],
                                   ["-fsanitize=thread"]], ids=["asan-ubsan", "tsan"])
def test_argument_checks_under_sanitizers(tmp_path, flags):
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path / "draft_driver")
    cmd = (["g++", "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__"] + flags
           + ["-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
              os.path.join(CSRC, "mx_draft_api.cpp"),
              os.path.join(ROOT, "tests", "draft_sanitize", "driver.cpp"), "-o", exe, "-lpthread"])
    subprocess.run(cmd, check=True, capture_output=True, timeout=300)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, TSAN_OPTIONS="halt_on_error=1"))
    assert r.returncode == 0, r.stdout + r.stderr
    assert "draft ABI checks passed" in r.stdout


def test_the_built_library_refuses_too():
    """The same checks through the shared library (every call fails before any HIP call)."""
    assert mx.mx_norm_rotate(None, None, mx.MX_BF16, 4, 64, 1e-6, None, None) == mx.MX_ERR_NULL
    heads = mx.MxHeads(1 << 32, 64, None, 2 << 32, 64, 1)
    assert mx.mx_norm_rotate(ctypes.byref(heads), None, mx.MX_BF16, 4, 96, 1e-6, None, None) == mx.MX_ERR_SHAPE
    assert mx.mx_norm_rotate_backward(None, None, mx.MX_BF16, 4, 64, 1e-6, None, None, 0, None) == mx.MX_ERR_NULL
    assert mx.mx_kv_append_rotary(1, 2, 1, 64, 64, None, 0.0, None, None, None, None) == mx.MX_ERR_NULL
    assert mx.mx_kv_attention_tree(1, 64, 1, None, None, None, 1, 0, 1.0, 2, None, 0, None) == mx.MX_ERR_NULL
    assert mx.mx_verify_drafts(None, None, 0, None, None, None, None, 1, 1, 10, 0, None, None, None, None, 0,
                               None) == mx.MX_ERR_SHAPE
    assert mx.mx_kv_keep(None, None, None, 1, None, None) == mx.MX_ERR_NULL


def test_packed_structures_have_the_headers_sizes():
    for packer, kind, fields in ((draft._pack_rotary, mx.MxRotary, 5), (draft._pack_heads, mx.MxHeads, 6),
                                 (draft._pack_grad, mx.MxHeadsGrad, 9)):
        raw = packer(*range(1, fields + 1))
        assert len(raw) == ctypes.sizeof(kind)
        back = kind.from_buffer_copy(raw)
        assert [getattr(back, name) for name, _ in kind._fields_] == list(range(1, fields + 1))


def test_workspace_sizes():
    assert mx.mx_norm_rotate_backward_workspace_size(0, 64) == 0
    assert mx.mx_norm_rotate_backward_workspace_size(5, 100) == 0
    for tokens in (1, 5, 1000, 1 << 20):
        size = mx.mx_norm_rotate_backward_workspace_size(tokens, 128)
        assert size > 0 and size % (2 * 128 * 4) == 0 and size <= max(1, tokens) * 2 * 128 * 4
    assert mx.mx_verify_drafts_workspace_size(0, 4, 100) == 0
    assert mx.mx_verify_drafts_workspace_size(4, 0, 100) == 0
    assert mx.mx_verify_drafts_workspace_size(4, 1, 0) == 0
    assert mx.mx_verify_drafts_workspace_size(4, 1, 100) % 16 == 0
    assert mx.mx_verify_drafts_workspace_size(8, 1, 1 << 20) > mx.mx_verify_drafts_workspace_size(8, 1, 1 << 10)


def test_attention_scratch_is_bounded_and_grows_with_the_length():
    for tokens, batch, q_heads, heads, dim in (
            (1, 1, 128, 1, 64), (63, 1, 600, 600, 64), (40, 1, 2000, 2000, 128), (33, 1, 4096, 4096, 128),
            (384, 16, 32, 8, 128), (4096, 64, 64, 8, 128), (4160, 65, 64, 8, 128), (8192, 1, 64, 8, 64)):
        before = 0
        for length in (1, 100, 1024, 1025, 5000, 33000, 1 << 20, 1 << 30, 0):  # 0: any
            size = mx.mx_kv_attention_tree_workspace_size(tokens, batch, q_heads, heads, dim, length)
            assert before <= size <= 66 << 20
            before = size


def test_helpers_refuse_cpu_tensors():
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    cache = mx.kv_cache(2, 1, 64, 32, device="cpu")
    i, t = torch.zeros(2, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    p = torch.zeros(1, 8)
    for f in (lambda: mx.norm_rotate(x), lambda: mx.norm_rotate_backward(x, x),
              lambda: mx.kv_append_rotary(cache, x, x, t, i, i[:1]),
              lambda: mx.kv_attention_tree(x, cache, t, i, i[:1], t[:, :1]),
              lambda: mx.verify_drafts(p, i[:1], i[:1], i, torch.zeros(1, 2), 1),
              lambda: mx.kv_keep(cache, t, i[:1], t, i[:1])):
        with pytest.raises(ValueError):
            f()


def test_tree_masks_and_tables_on_the_cpu():
    parents = [[-1, 0, 0, 1, 1, 2, 5], [-1], [], [-1] + list(range(70))]
    mask, depth = mx.tree_mask(parents, device="cpu")
    assert mask.shape == (79, 3) and torch.equal(mask, torch.cat([ref.words_of(ref.ancestors(p), 3) for p in parents]))
    assert depth.tolist() == [0, 1, 1, 2, 2, 2, 3, 0] + list(range(71))
    for bad in ([[0]], [[-1, 1]], [[-1, -2]]):
        with pytest.raises(ValueError):
            mx.tree_mask(bad, device="cpu")
    table = mx.rotary_table(100, 32, 500.0, device="cpu")
    angles = torch.arange(100).double()[:, None] * 500.0 ** (-torch.arange(0, 32, 2).double() / 32)
    assert float((table - torch.cat([angles.cos(), angles.sin()], 1)).abs().max()) <= 2.0 ** -24
    for rot in (0, -16, 24):
        with pytest.raises(ValueError):
            mx.rotary_table(100, rot, device="cpu")


def test_the_references_agree_with_each_other():
    """The walk's tokens are the target's over many trees (by count, on the CPU)."""
    g = torch.Generator().manual_seed(1)
    p, q, n = torch.tensor([0.5, 0.3, 0.2]), torch.tensor([0.2, 0.2, 0.6]), 4000
    ids = torch.multinomial(q.expand(n, -1), 2, replacement=True, generator=g)
    ids = torch.cat([torch.zeros(n, 1, dtype=torch.long), ids], 1).view(-1)
    cu, parents = list(range(0, 3 * n + 1, 3)), [-1, 0, 0] * n
    numbers = torch.rand(3 * n, 2, generator=g)
    for draft_rows in (None, q.expand(3 * n, -1)):
        path, count, token = ref.verify(p.expand(3 * n, -1), draft_rows, ids, parents, cu, numbers, 2)
        first = [int(ids[3 * i + path[i][1]]) if count[i] > 1 else token[i] for i in range(n)]
        seen = torch.bincount(torch.tensor(first), minlength=3).double() / n
        assert bool(((seen - p).abs() <= 6 * torch.sqrt(p * (1 - p) / n)).all())
