"""MXFP8 through a transformer layer: tensor-level helpers.

The norm that hands over 8-bit rows and its gradient, the quantizer with
blocks along rows and columns, products of 8-bit matrices, the paged 8-bit
key/value cache and the attention that reads it. Every step runs in the HIP
kernels behind include/mx.h; this module allocates outputs and scratch with
torch (on the current stream) and checks what the C entry points cannot see:
devices, dtypes, shapes and contiguity. Bad arguments raise ``ValueError``,
HIP errors ``RuntimeError``.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from . import _DTYPES, _need, _raise, _stream, load_library

BLOCKS = (32, 128)


class MxKVCache(ctypes.Structure):
    """mx_kv_cache_t of include/mx.h (pointers as integers)."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("heads", ctypes.c_int), ("dim", ctypes.c_int),
                ("page", ctypes.c_int)]


class MxKVBatch(ctypes.Structure):
    """mx_kv_batch_t of include/mx.h (pointers as integers)."""
    _fields_ = [("table", ctypes.c_void_p), ("cu", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("tokens", ctypes.c_int64), ("batch", ctypes.c_int), ("width", ctypes.c_int)]


class KVCache(NamedTuple):
    """A paged cache: ``k_codes`` uint8 [pages, heads, page, dim], ``v_codes``
    uint8 [pages, heads, dim, page], scales uint8 [pages, heads]."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


def kv_cache(pages: int, heads: int, dim: int, page: int = 64, device="cuda") -> KVCache:
    """An empty cache of `pages` pages of `page` tokens (contents are zeros)."""
    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device=device)
    return KVCache(zeros(pages, heads, page, dim), zeros(pages, heads),
                   zeros(pages, heads, dim, page), zeros(pages, heads))


# ---- C entry points, same names -------------------------------------------

def mx_quantize_mxfp8_blocks(x, x_dtype, rows, k, block, codes, scales, codes_t, scales_t,
                             stream) -> int:
    return load_library().mx_quantize_mxfp8_blocks(x, x_dtype, rows, k, block, codes, scales,
                                                   codes_t, scales_t, stream)


def mx_rmsnorm_mxfp8(x, residual, weight, dtype, rows, k, eps, block, codes, scales, h_out,
                     stream) -> int:
    return load_library().mx_rmsnorm_mxfp8(x, residual, weight, dtype, rows, k, eps, block, codes,
                                           scales, h_out, stream)


def mx_rmsnorm_backward_workspace_size(rows, k) -> int:
    return load_library().mx_rmsnorm_backward_workspace_size(rows, k)


def mx_rmsnorm_backward(dy, h, weight, through, dtype, rows, k, eps, dx, dweight, workspace,
                        workspace_bytes, stream) -> int:
    return load_library().mx_rmsnorm_backward(dy, h, weight, through, dtype, rows, k, eps, dx,
                                              dweight, workspace, workspace_bytes, stream)


def mx_matmul_mxfp8_workspace_size(m, n, k, block, c_dtype) -> int:
    return load_library().mx_matmul_mxfp8_workspace_size(m, n, k, block, c_dtype)


def mx_matmul_mxfp8(a, a_scales, b, b_scales, m, n, k, block, c_dtype, c, workspace,
                    workspace_bytes, stream) -> int:
    return load_library().mx_matmul_mxfp8(a, a_scales, b, b_scales, m, n, k, block, c_dtype, c,
                                          workspace, workspace_bytes, stream)


def mx_kv_append(k, v, dtype, k_stride, v_stride, cache, batch, stream) -> int:
    return load_library().mx_kv_append(k, v, dtype, k_stride, v_stride, cache, batch, stream)


def mx_kv_attention_workspace_size(tokens, batch, q_heads, heads, dim, max_length) -> int:
    return load_library().mx_kv_attention_workspace_size(tokens, batch, q_heads, heads, dim,
                                                         max_length)


def mx_kv_attention(q, q_stride, q_heads, cache, batch, max_length, scale, out, workspace,
                    workspace_bytes, stream) -> int:
    return load_library().mx_kv_attention(q, q_stride, q_heads, cache, batch, max_length, scale,
                                          out, workspace, workspace_bytes, stream)


def declare(lib) -> None:
    """Argument and result types of the entry points."""
    p, i64, i32, f32, size = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                              ctypes.c_size_t)
    types = {
        "mx_quantize_mxfp8_blocks": [p, i32, i64, i64, i32, p, p, p, p, p],
        "mx_rmsnorm_mxfp8": [p, p, p, i32, i64, i64, f32, i32, p, p, p, p],
        "mx_rmsnorm_backward": [p, p, p, p, i32, i64, i64, f32, p, p, p, size, p],
        "mx_matmul_mxfp8": [p, p, p, p, i64, i64, i64, i32, i32, p, p, size, p],
        "mx_kv_append": [p, p, i32, i64, i64, p, p, p],
        "mx_kv_attention": [p, i64, i32, p, p, i64, f32, p, p, size, p],
        "mx_rmsnorm_backward_workspace_size": [i64, i64],
        "mx_matmul_mxfp8_workspace_size": [i64, i64, i64, i32, i32],
        "mx_kv_attention_workspace_size": [i64, i32, i32, i32, i32, i64],
    }
    for name, args in types.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = size if name.endswith("_size") else i32


# ---- tensor helpers --------------------------------------------------------
#
# They run once per layer and token, where the host's time counts: small
# allocations go by the call that is fastest here, and the two structures are
# packed as bytes.

_pack_cache = struct.Struct("@PPPPqiii4x").pack
_pack_batch = struct.Struct("@PPPqii").pack


def _bytes(like, rows: int, cols: int, two: bool):
    """uint8 [rows, cols] on like's device, or in like's leading shape."""
    if two:
        return torch.empty(rows, cols, dtype=torch.uint8, device=like.device)
    return torch.empty((*like.shape[:-1], cols), dtype=torch.uint8, device=like.device)


def _matrix(x, name: str, dtypes=_DTYPES):
    """A contiguous GPU tensor [..., k], k a multiple of 32: (rows, k)."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if x.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {list(dtypes)}, got {x.dtype}")
    shape = x.shape
    if not shape or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous, with at least one dimension")
    k = shape[-1]
    if k <= 0 or k % 32:
        raise ValueError(f"{name}'s last dimension must be a positive multiple of 32")
    return (shape[0] if len(shape) == 2 else x.numel() // k), k


def _want(t, name: str, dev, dtype, numel: int, last: int = 0):
    """_need() with its outcome found in fewer steps where all is well. `last`:
    what the last dimension must be (0: any) of more than one."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == numel
            and t.device == dev and t.is_contiguous()):
        _need(t, name, dev, dtype, numel)
    if last and t.dim() > 1 and t.size(-1) != last:
        raise ValueError(f"{name} must be [..., {last}], got {tuple(t.shape)}")


def _block(block: int) -> int:
    if block not in BLOCKS:
        raise ValueError(f"block must be one of {BLOCKS}, got {block!r}")
    return block


def _ptr(t):
    return None if t is None else t.data_ptr()


# torch's own quick ways to the current device and stream (1.4 us a call less than
# the public ones); a torch without them has the public ones
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)


def _call(device, fn, *args):
    """fn(*args, stream) on the device's current stream, raising on a bad status."""
    index = device.index
    if _device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index))
    if status:
        _raise(status)


def _scratch(size: int, device):
    return torch.empty(size, dtype=torch.uint8, device=device) if size else None


def _quantize_blocks(x, block, rows_too: bool, columns: bool):
    rows, k = _matrix(x, "x")
    nb, dev, two = -(-k // _block(block)), x.device, x.dim() == 2
    codes = scales = codes_t = scales_t = None
    if rows_too:
        codes, scales = torch.empty_like(x, dtype=torch.uint8), _bytes(x, rows, nb, two)
    if columns:
        codes_t = torch.empty(k, -(-rows // 32) * 32, dtype=torch.uint8, device=dev)
        scales_t = torch.empty(k, -(-rows // block), dtype=torch.uint8, device=dev)
    _call(dev, load_library().mx_quantize_mxfp8_blocks, x.data_ptr(), _DTYPES[x.dtype], rows, k,
          block, _ptr(codes), _ptr(scales), _ptr(codes_t), _ptr(scales_t))
    return codes, scales, codes_t, scales_t


def quantize_mxfp8_rows(x: torch.Tensor, block: int = 128):
    """x [..., k] -> (codes uint8 [..., k], scales uint8 [..., ceil(k / block)]),
    blocks of 32 or 128 along the last dimension."""
    return _quantize_blocks(x, block, True, False)[:2]


def quantize_mxfp8_columns(x: torch.Tensor, block: int = 128):
    """x [..., k] seen as [rows, k] -> its transpose quantized along the rows:
    (codes uint8 [k, R], scales uint8 [k, ceil(rows / block)]), R = rows
    rounded up to a multiple of 32 (codes past rows are 0)."""
    return _quantize_blocks(x, block, False, True)[2:]


def quantize_mxfp8_both(x: torch.Tensor, block: int = 128):
    """quantize_mxfp8_rows and quantize_mxfp8_columns from one read of x:
    (codes, scales, codes_t, scales_t)."""
    return _quantize_blocks(x, block, True, True)


def rmsnorm_mxfp8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                  residual: torch.Tensor | None = None, block: int = 128,
                  out_h: torch.Tensor | None = None):
    """h = x + residual (or x); weight * h / sqrt(mean(h^2) + eps) in MXFP8 ->
    (codes uint8 [..., k], scales uint8 [..., ceil(k / block)], h in x's dtype,
    or None without a residual). out_h may be x or residual."""
    rows, k = _matrix(x, "x")
    dev = x.device
    _want(weight, "weight", dev, x.dtype, k, k)
    nb = -(-k // _block(block))
    if residual is not None:
        _want(residual, "residual", dev, x.dtype, x.numel(), k)
        if out_h is None:
            out_h = torch.empty_like(x)
        else:
            _want(out_h, "out_h", dev, x.dtype, x.numel(), k)
    elif out_h is not None:
        raise ValueError("out_h needs a residual")
    codes, scales = torch.empty_like(x, dtype=torch.uint8), _bytes(x, rows, nb, x.dim() == 2)
    _call(dev, load_library().mx_rmsnorm_mxfp8, x.data_ptr(), _ptr(residual), weight.data_ptr(),
          _DTYPES[x.dtype], rows, k, eps, block, codes.data_ptr(), scales.data_ptr(), _ptr(out_h))
    return codes, scales, out_h


def rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                     through: torch.Tensor | None = None):
    """Gradient of rmsnorm_mxfp8 (the quantizer passing gradients through) ->
    (dx in h's dtype, dweight float32 [k]); `through` is the gradient that
    reaches h past the norm. dx is the gradient of x and of residual alike."""
    rows, k = _matrix(h, "h")
    dev = h.device
    _want(dy, "dy", dev, h.dtype, h.numel(), k)
    _want(weight, "weight", dev, h.dtype, k, k)
    if through is not None:
        _want(through, "through", dev, h.dtype, h.numel(), k)
    lib = load_library()
    dx = torch.empty_like(h)
    dweight = torch.empty(k, dtype=torch.float32, device=dev)
    size = lib.mx_rmsnorm_backward_workspace_size(rows, k)
    ws = _scratch(size, dev)
    _call(dev, lib.mx_rmsnorm_backward, dy.data_ptr(), h.data_ptr(), weight.data_ptr(),
          _ptr(through), _DTYPES[h.dtype], rows, k, eps, dx.data_ptr(), dweight.data_ptr(),
          _ptr(ws), size)
    return dx, dweight


def matmul_mxfp8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                 dtype=torch.bfloat16, block: int = 128, out: torch.Tensor | None = None):
    """a [..., k] times b [n, k] transposed, both MXFP8 codes with scales per
    `block` elements of a row -> [..., n] in dtype (float32 keeps fp32
    accuracy at half the rate)."""
    m, k = _matrix(a, "a", (torch.uint8,))
    n, kb = _matrix(b, "b", (torch.uint8,))
    dev = a.device
    if b.dim() != 2 or kb != k:
        raise ValueError(f"b must be [n, {k}], got {tuple(b.shape)}")
    if b.device != dev:
        raise ValueError(f"b is on {b.device}, expected {dev}")
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
    nb = -(-k // _block(block))
    _want(a_scales, "a_scales", dev, torch.uint8, m * nb, nb)
    _want(b_scales, "b_scales", dev, torch.uint8, n * nb, nb)
    if out is None:
        out = (torch.empty(m, n, dtype=dtype, device=dev) if a.dim() == 2
               else torch.empty(a.shape[:-1] + (n,), dtype=dtype, device=dev))
    else:
        _want(out, "out", dev, dtype, m * n, n)
    lib, cd = load_library(), _DTYPES[dtype]
    size = lib.mx_matmul_mxfp8_workspace_size(m, n, k, block, cd)
    ws = _scratch(size, dev)
    _call(dev, lib.mx_matmul_mxfp8, a.data_ptr(), a_scales.data_ptr(), b.data_ptr(),
          b_scales.data_ptr(), m, n, k, block, cd, out.data_ptr(), _ptr(ws), size)
    return out


def _heads_of(t, name: str, dev, dtypes):
    """[tokens, heads, dim] with adjacent heads; any stride between tokens."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be a tensor on {dev}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {list(dtypes)}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim]")
    tokens, heads, dim = t.shape
    step, head, one = t.stride()
    if (dim > 1 and one != 1) or (heads > 1 and head != dim):
        raise ValueError(f"{name}'s heads must lie next to each other")
    return tokens, heads, dim, step if tokens > 1 else heads * dim


def _cache_of(cache: KVCache):
    """(device, heads, dim, page, mx_kv_cache_t)"""
    k, ks, v, vs = cache
    dev = getattr(k, "device", None)
    _need(k, "k_codes", dev, torch.uint8)
    if k.dim() != 4:
        raise ValueError("k_codes must be [pages, heads, page, dim]")
    pages, heads, page, dim = k.shape
    _want(v, "v_codes", dev, torch.uint8, k.numel())
    if v.shape != (pages, heads, dim, page):
        raise ValueError(f"v_codes must be {(pages, heads, dim, page)}, got {tuple(v.shape)}")
    _want(ks, "k_scales", dev, torch.uint8, pages * heads, heads)
    _want(vs, "v_scales", dev, torch.uint8, pages * heads, heads)
    return dev, heads, dim, page, _pack_cache(k.data_ptr(), ks.data_ptr(), v.data_ptr(),
                                              vs.data_ptr(), pages, heads, dim, page)


def _batch_of(dev, table, cu, lengths, tokens):
    """(batch, width, mx_kv_batch_t)"""
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [batch, width]")
    batch, width = table.shape
    _want(table, "table", dev, torch.int32, batch * width)
    _want(cu, "cu", dev, torch.int32, batch + 1)
    _want(lengths, "lengths", dev, torch.int32, batch)
    return batch, width, _pack_batch(table.data_ptr(), cu.data_ptr(), lengths.data_ptr(), tokens,
                                     batch, width)


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor,
              cu: torch.Tensor, lengths: torch.Tensor) -> None:
    """Append new tokens' k and v [tokens, heads, dim] (slices of one
    projection's rows are fine) to the cache, in place. table int32 [batch,
    width]: each sequence's pages; cu int32 [batch + 1]: where its new tokens
    start; lengths int32 [batch]: what it held before."""
    dev, held_heads, held_dim, _, c = _cache_of(cache)
    tokens, heads, dim, stride = _heads_of(k, "k", dev, _DTYPES)
    v_tokens, v_heads, v_dim, v_stride = _heads_of(v, "v", dev, (k.dtype,))
    if v_tokens != tokens or v_heads != heads or v_dim != dim:
        raise ValueError("k and v must have one shape")
    if heads != held_heads or dim != held_dim:
        raise ValueError(f"the cache holds {held_heads} heads of {held_dim}, got {heads} of {dim}")
    b = _batch_of(dev, table, cu, lengths, tokens)[2]
    _call(dev, load_library().mx_kv_append, k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype], stride,
          v_stride, c, b)


def kv_attention(q: torch.Tensor, cache: KVCache, table: torch.Tensor, cu: torch.Tensor,
                 lengths: torch.Tensor, scale: float | None = None, max_length: int = 0,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention of q bfloat16 [tokens, q_heads, dim] over the cache ->
    [tokens, q_heads, dim]; lengths int32 [batch] count each sequence's new
    tokens too. scale defaults to 1 / sqrt(dim); max_length bounds the lengths
    (0: what the table has room for) and only steers the launch."""
    dev, heads, held_dim, page, c = _cache_of(cache)
    tokens, q_heads, dim, stride = _heads_of(q, "q", dev, (torch.bfloat16,))
    if dim != held_dim:
        raise ValueError(f"the cache holds heads of {held_dim}, got {dim}")
    if q_heads < heads or q_heads % heads:
        raise ValueError(f"q_heads must be a multiple of the cache's {heads}, got {q_heads}")
    batch, width, b = _batch_of(dev, table, cu, lengths, tokens)
    if out is None:
        out = torch.empty(tokens, q_heads, dim, dtype=torch.bfloat16, device=dev)
    else:
        _want(out, "out", dev, torch.bfloat16, tokens * q_heads * dim, dim)
    room = width * page
    max_length = room if max_length <= 0 else min(max_length, room)
    lib = load_library()
    size = lib.mx_kv_attention_workspace_size(tokens, batch, q_heads, heads, dim, max_length)
    ws = _scratch(size, dev)
    _call(dev, lib.mx_kv_attention, q.data_ptr(), stride, q_heads, c, b, max_length,
          1.0 / math.sqrt(dim) if scale is None else scale, out.data_ptr(), _ptr(ws), size)
    return out
