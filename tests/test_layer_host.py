"""Host side of the transformer-layer operators, without a GPU: the C ABI's
argument checks under sanitizers, and the tensor helpers' refusals."""
import os
import shutil
import subprocess

import pytest
import torch

import microscaling_fp4_block_mx_amd as mx
from conftest import ROOT

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
    exe = str(tmp_path / "layer_driver")
    cmd = (["g++", "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__"] + flags
           + ["-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
              os.path.join(CSRC, "mx_layer_api.cpp"),
              os.path.join(ROOT, "tests", "layer_sanitize", "driver.cpp"), "-o", exe, "-lpthread"])
    subprocess.run(cmd, check=True, capture_output=True, timeout=300)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, TSAN_OPTIONS="halt_on_error=1"))
    assert r.returncode == 0, r.stdout + r.stderr
    assert "layer ABI checks passed" in r.stdout


def test_the_built_library_refuses_too():
    """The same checks through the shared library (every call fails before any HIP call)."""
    A, B, C, D = (i << 32 for i in range(1, 5))
    assert mx.mx_rmsnorm_mxfp8(A, None, B, mx.MX_BF16, 4, 48, 1e-5, 32, C, D, None,
                               None) == mx.MX_ERR_SHAPE
    assert mx.mx_matmul_mxfp8(A, B, C, D, 4, 4, 64, 32, 5, 5 << 32, None, 0, None) == mx.MX_ERR_DTYPE
    assert mx.mx_quantize_mxfp8_blocks(A, 1, 4, 64, 32, B, None, None, None, None) == mx.MX_ERR_NULL
    assert mx.mx_kv_append(A, B, 1, 64, 64, None, None, None) == mx.MX_ERR_NULL
    assert mx.mx_rmsnorm_backward(A, B, C, None, 1, 4, 64, 1e-5, D, None, None, 0,
                                  None) == mx.MX_ERR_NULL
    assert mx.mx_kv_attention(A, 64, 1, None, None, 0, 1.0, B, None, 0, None) == mx.MX_ERR_NULL


@pytest.mark.parametrize("m,n,k", [(1, 8192, 4096), (65, 64, 8192), (100, 100, 65536),
                                   (300, 300, 4096), (8192, 8192, 4096), (64, 64, 1 << 20)])
def test_workspace_sizes(m, n, k):
    """A multiple of the fp32 output, and nothing where the tiles fill the card."""
    for block in (32, 128):
        for dt in (mx.MX_BF16, mx.MX_F32):
            size = mx.mx_matmul_mxfp8_workspace_size(m, n, k, block, dt)
            assert size % (4 * m * n) == 0
            if m <= 64 or m * n >= 1 << 24:
                assert size == 0
    assert mx.mx_matmul_mxfp8_workspace_size(m, n, 40, 32, mx.MX_BF16) == 0
    assert mx.mx_matmul_mxfp8_workspace_size(0, n, k, 32, mx.MX_BF16) == 0
    assert mx.mx_rmsnorm_backward_workspace_size(0, 64) == 0
    assert mx.mx_rmsnorm_backward_workspace_size(3, 64) == 3 * 64 * 4
    assert mx.mx_kv_attention_workspace_size(8, 8, 32, 8, 96, 4096) == 0
    assert mx.mx_kv_attention_workspace_size(8, 8, 32, 8, 128, 64) == 0
    split = mx.mx_kv_attention_workspace_size(8, 8, 32, 8, 128, 65536)
    assert split > 0 and split % (8 * 32 * 132 * 4) == 0


def test_helpers_refuse_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    u8 = torch.zeros(4, 64, dtype=torch.uint8)
    s = torch.zeros(4, 1, dtype=torch.uint8)
    cache = mx.kv_cache(2, 1, 64, 32, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(1, 2, dtype=torch.int32)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for f in (lambda: mx.rmsnorm_mxfp8(x, x[0]), lambda: mx.rmsnorm_backward(x, x, x[0]),
              lambda: mx.quantize_mxfp8_both(x), lambda: mx.quantize_mxfp8_rows(x),
              lambda: mx.quantize_mxfp8_columns(x), lambda: mx.matmul_mxfp8(u8, s, u8, s),
              lambda: mx.kv_append(cache, q, q, t, i, i[:1]),
              lambda: mx.kv_attention(q, cache, t, i, i[:1])):
        with pytest.raises(ValueError):
            f()


@pytest.mark.gpu
def test_helpers_refuse_bad_tensors():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    u8 = torch.zeros(4, 64, dtype=torch.uint8, device="cuda")
    s = torch.zeros(4, 1, dtype=torch.uint8, device="cuda")
    cache = mx.kv_cache(4, 2, 64, 32)
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    t = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: mx.rmsnorm_mxfp8(x, w.float()),                        # weight's dtype
        lambda: mx.rmsnorm_mxfp8(x, w[:32].contiguous()),              # weight's length
        lambda: mx.rmsnorm_mxfp8(x.t(), w),                            # not contiguous
        lambda: mx.rmsnorm_mxfp8(x[:, :48].contiguous(), w[:48].contiguous()),
        lambda: mx.rmsnorm_mxfp8(x, w, block=64),
        lambda: mx.rmsnorm_mxfp8(x, w, eps=-1.0),
        lambda: mx.rmsnorm_mxfp8(x, w, out_h=torch.empty_like(x)),     # nothing to write there
        lambda: mx.rmsnorm_mxfp8(x, w, residual=x[:2]),
        lambda: mx.rmsnorm_mxfp8(x.half(), w.half()),
        lambda: mx.rmsnorm_backward(x.float(), x, w),
        lambda: mx.rmsnorm_backward(x, x, w, through=x[:2]),
        lambda: mx.quantize_mxfp8_both(x, block=16),
        lambda: mx.quantize_mxfp8_rows(torch.zeros(4, 40, device="cuda")),
        lambda: mx.matmul_mxfp8(u8, s, u8[:, :32].contiguous(), s),    # other k
        lambda: mx.matmul_mxfp8(u8, s, u8.view(2, 2, 64), s),
        lambda: mx.matmul_mxfp8(u8, s[:2], u8, s),
        lambda: mx.matmul_mxfp8(u8, s, u8, s, torch.float16),
        lambda: mx.matmul_mxfp8(u8, s, u8, s, block=32),               # scales of 128
        lambda: mx.matmul_mxfp8(u8, s, u8, s, out=torch.empty(4, 4, device="cuda")),
        lambda: mx.matmul_mxfp8(x, s, u8, s),
        lambda: mx.kv_append(cache, kv[..., ::2], kv, t, i, i[:1]),
        lambda: mx.kv_append(cache, kv, kv.float(), t, i, i[:1]),
        lambda: mx.kv_append(cache, q, q, t, i, i[:1]),                # other heads
        lambda: mx.kv_append(cache, kv, kv, t.long(), i, i[:1]),
        lambda: mx.kv_append(cache, kv, kv, t, i[:1], i[:1]),          # cu too short
        lambda: mx.kv_append(cache, kv.transpose(0, 1), kv.transpose(0, 1), t, i, i[:1]),
        lambda: mx.kv_attention(q.float(), cache, t, i, i[:1]),
        lambda: mx.kv_attention(q[:, :3], cache, t, i, i[:1]),         # heads not a multiple
        lambda: mx.kv_attention(q, cache, t, i, i[:1], scale=0.0),
        lambda: mx.kv_attention(q, cache._replace(v_codes=cache.k_codes), t, i, i[:1]),
        lambda: mx.kv_attention(q, cache, t[0], i, i[:1]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    torch.cuda.synchronize()
