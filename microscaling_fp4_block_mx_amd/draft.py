"""Positions and drafted tokens beside the 8-bit cache: tensor-level helpers.

The norms of queries and keys per head with the position rotation, their
gradient, the append that has both on the way, attention over a tree of drafted
tokens, their verification, and keeping the accepted ones. Every step runs in the
HIP kernels behind include/mx.h; this module allocates outputs and scratch with
torch (on the current stream) and checks what the C entry points cannot see:
devices, dtypes, shapes and contiguity. Bad arguments raise ``ValueError``, HIP
errors ``RuntimeError``.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from . import _DTYPES, _need, load_library
from .layer import (_I32, KVCache, _batch_of, _cache_of, _call, _heads_of, _pack_batch, _ptr,
                    _scratch, _Tensor, _want)

_F32 = torch.float32


class MxRotary(ctypes.Structure):
    """mx_rotary_t of include/mx.h (pointers as integers)."""
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("length", ctypes.c_int64), ("rot", ctypes.c_int), ("paired", ctypes.c_int)]


class MxHeads(ctypes.Structure):
    """mx_heads_t of include/mx.h (pointers as integers)."""
    _fields_ = [("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64), ("heads", ctypes.c_int)]


class MxHeadsGrad(ctypes.Structure):
    """mx_heads_grad_t of include/mx.h (pointers as integers)."""
    _fields_ = [("dy", ctypes.c_void_p), ("dy_stride", ctypes.c_int64), ("x", ctypes.c_void_p),
                ("x_stride", ctypes.c_int64), ("weight", ctypes.c_void_p), ("dx", ctypes.c_void_p),
                ("dx_stride", ctypes.c_int64), ("dweight", ctypes.c_void_p),
                ("heads", ctypes.c_int)]


class Rotary(NamedTuple):
    """A rotation: ``table`` float32 [length, rot] (rotary_table), ``positions``
    int32 [tokens], ``paired``: dims (2 i, 2 i + 1) turn instead of (i, i + rot / 2)."""
    table: torch.Tensor
    positions: torch.Tensor | None = None
    paired: bool = False


def rotary_table(length: int, rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """float32 [length, rot]: row p has the cosines, then the sines, of p / base^(2 i / rot),
    i = 0 .. rot / 2 - 1 (angles in 64 bits)."""
    if rot <= 0 or rot % 16:
        raise ValueError(f"rot must be a positive multiple of 16, got {rot}")
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angles = torch.arange(length, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([angles.cos(), angles.sin()], 1).float()


def tree_mask(parents, device="cuda"):
    """(mask int32 [tokens, words], depth int32 [tokens]) of drafted tokens: `parents`
    lists, for each sequence, each node's parent (-1: none; parents come first). A
    node sees its ancestors and itself; depth counts its ancestors. Formed on the
    host, once for a tree's shape."""
    parents = [list(p) for p in parents]
    words = max(1, -(-max((len(p) for p in parents), default=0) // 32))
    rows, depth = [], []
    for tree in parents:
        bits, deep = [], []
        for j, up in enumerate(tree):
            if not -1 <= up < j:
                raise ValueError(f"node {j}'s parent must come before it, got {up}")
            bits.append(1 << j | (bits[up] if up >= 0 else 0))
            deep.append(deep[up] + 1 if up >= 0 else 0)
        for b in bits:
            for w in range(words):
                word = b >> 32 * w & 0xFFFFFFFF
                rows.append(word - (1 << 32) if word >> 31 else word)
        depth += deep
    return (torch.tensor(rows, dtype=torch.int32, device=device).view(-1, words),
            torch.tensor(depth, dtype=torch.int32, device=device))


# ---- C entry points, same names -------------------------------------------

def mx_norm_rotate(q, k, dtype, tokens, dim, eps, rotary, stream) -> int:
    return load_library().mx_norm_rotate(q, k, dtype, tokens, dim, eps, rotary, stream)


def mx_norm_rotate_backward_workspace_size(tokens, dim) -> int:
    return load_library().mx_norm_rotate_backward_workspace_size(tokens, dim)


def mx_norm_rotate_backward(q, k, dtype, tokens, dim, eps, rotary, workspace, workspace_bytes,
                            stream) -> int:
    return load_library().mx_norm_rotate_backward(q, k, dtype, tokens, dim, eps, rotary, workspace,
                                                  workspace_bytes, stream)


def mx_kv_append_rotary(k, v, dtype, k_stride, v_stride, k_weight, eps, rotary, cache, batch,
                        stream) -> int:
    return load_library().mx_kv_append_rotary(k, v, dtype, k_stride, v_stride, k_weight, eps, rotary,
                                              cache, batch, stream)


def mx_kv_attention_tree_workspace_size(tokens, batch, q_heads, heads, dim, max_length) -> int:
    return load_library().mx_kv_attention_tree_workspace_size(tokens, batch, q_heads, heads, dim,
                                                              max_length)


def mx_kv_attention_tree(q, q_stride, q_heads, cache, batch, mask, words, max_length, scale, out,
                         workspace, workspace_bytes, stream) -> int:
    return load_library().mx_kv_attention_tree(q, q_stride, q_heads, cache, batch, mask, words,
                                               max_length, scale, out, workspace, workspace_bytes,
                                               stream)


def mx_verify_drafts_workspace_size(tokens, batch, vocab) -> int:
    return load_library().mx_verify_drafts_workspace_size(tokens, batch, vocab)


def mx_verify_drafts(target, draft, dtype, ids, parents, cu, numbers, tokens, batch, vocab, width,
                     path, count, token, workspace, workspace_bytes, stream) -> int:
    return load_library().mx_verify_drafts(target, draft, dtype, ids, parents, cu, numbers, tokens,
                                           batch, vocab, width, path, count, token, workspace,
                                           workspace_bytes, stream)


def mx_kv_keep(cache, batch, path, path_width, count, stream) -> int:
    return load_library().mx_kv_keep(cache, batch, path, path_width, count, stream)


def declare(lib) -> None:
    """Argument and result types of the entry points."""
    p, i64, i32, f32, size = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                              ctypes.c_size_t)
    types = {
        "mx_norm_rotate": [p, p, i32, i64, i32, f32, p, p],
        "mx_norm_rotate_backward": [p, p, i32, i64, i32, f32, p, p, size, p],
        "mx_kv_append_rotary": [p, p, i32, i64, i64, p, f32, p, p, p, p],
        "mx_kv_attention_tree": [p, i64, i32, p, p, p, i32, i64, f32, p, p, size, p],
        "mx_verify_drafts": [p, p, i32, p, p, p, p, i64, i32, i64, i32, p, p, p, p, size, p],
        "mx_kv_keep": [p, p, p, i32, p, p],
        "mx_kv_attention_tree_workspace_size": [i64, i32, i32, i32, i32, i64],
        "mx_norm_rotate_backward_workspace_size": [i64, i32],
        "mx_verify_drafts_workspace_size": [i64, i32, i64],
    }
    for name, args in types.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = size if name.endswith("_size") else i32


# ---- tensor helpers --------------------------------------------------------

_pack_rotary = struct.Struct("@PPqii").pack
_pack_heads = struct.Struct("@PqPPqi4x").pack
_pack_grad = struct.Struct("@PqPqPPqPi4x").pack


def _rotary_of(rotary: Rotary | None, dev, dim: int, tokens: int, positions: bool):
    """mx_rotary_t, or None without a rotation. `positions`: they must be given."""
    if rotary is None:
        return None
    table, pos, paired = rotary
    if not isinstance(table, _Tensor) or len(table.shape) != 2:
        raise ValueError("the rotation's table must be [length, rot]")
    length, rot = table.shape
    if not (table.dtype is _F32 and table.device == dev and table.is_contiguous()):
        _need(table, "table", dev, _F32)
    if rot % 16 or not 0 < rot <= dim:
        raise ValueError(f"rot must be a multiple of 16 up to {dim}, got {rot}")
    if length < 1:
        raise ValueError("the rotation's table has no positions")
    if pos is not None or positions:
        _want(pos, "positions", dev, _I32, tokens)
    return _pack_rotary(table.data_ptr(), pos.data_ptr() if pos is not None else 0, length, rot,
                        bool(paired))


def _into(out, name: str, like, tokens: int, heads: int, dim: int):
    """(out, its stride): a new tensor, or the one given (any stride between tokens)."""
    if out is None:
        return torch.empty(tokens, heads, dim, dtype=like.dtype, device=like.device), heads * dim
    got = _heads_of(out, name, like.device, (like.dtype,))
    if got[:3] != (tokens, heads, dim):
        raise ValueError(f"{name} must be {(tokens, heads, dim)}, got {tuple(out.shape)}")
    return out, got[3]


def _address(t) -> int:
    return 0 if t is None else t.data_ptr()


def _on_gpu(t, name: str):
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def norm_rotate(q: torch.Tensor, k: torch.Tensor | None = None,
                q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                rotary: Rotary | None = None, eps: float = 1e-6,
                out_q: torch.Tensor | None = None, out_k: torch.Tensor | None = None):
    """Heads [tokens, heads, dim] of q (and k) through a norm over each head's
    dims (weight [dim]; None: no norm) and the position rotation (None: none) ->
    (q, k) new, contiguous, k None without one. Slices of one projection's rows
    are fine. out_q may be q and out_k may be k, in place."""
    dev = _on_gpu(q, "q")
    tokens, heads, dim, stride = _heads_of(q, "q", dev, _DTYPES)
    r = _rotary_of(rotary, dev, dim, tokens, True)

    def pack(x, name, stride, heads, weight, out):
        if weight is not None:
            _want(weight, name + "_weight", dev, x.dtype, dim)
        out, out_stride = _into(out, "out_" + name, x, tokens, heads, dim)
        return out, _pack_heads(x.data_ptr(), stride, _address(weight), out.data_ptr(), out_stride,
                                heads)

    kb = None
    if k is not None:
        k_tokens, k_heads, k_dim, k_stride = _heads_of(k, "k", dev, (q.dtype,))
        if k_tokens != tokens or k_dim != dim:
            raise ValueError(f"k must be [{tokens}, heads, {dim}], got {tuple(k.shape)}")
        out_k, kb = pack(k, "k", k_stride, k_heads, k_weight, out_k)
    elif k_weight is not None or out_k is not None:
        raise ValueError("k_weight and out_k need k")
    out_q, qb = pack(q, "q", stride, heads, q_weight, out_q)
    _call(dev, load_library().mx_norm_rotate, qb, kb, _DTYPES[q.dtype], tokens, dim, eps, r)
    return out_q, out_k


def norm_rotate_backward(dq: torch.Tensor, q: torch.Tensor, dk: torch.Tensor | None = None,
                         k: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                         k_weight: torch.Tensor | None = None, rotary: Rotary | None = None,
                         eps: float = 1e-6):
    """Gradients of norm_rotate at its inputs q and k -> (dq, dk, dq_weight,
    dk_weight); weights' in float32 [dim], None where there is no weight (or k)."""
    dev = _on_gpu(q, "q")
    tokens, heads, dim, stride = _heads_of(q, "q", dev, _DTYPES)
    r = _rotary_of(rotary, dev, dim, tokens, True)
    if (k is None) != (dk is None) or (k is None and k_weight is not None):
        raise ValueError("k, dk and k_weight go together")

    def pack(dy, x, name, stride, heads, weight):
        got = _heads_of(dy, "d" + name, dev, (x.dtype,))
        if got[:3] != (tokens, heads, dim):
            raise ValueError(f"d{name} must be {(tokens, heads, dim)}, got {tuple(dy.shape)}")
        dweight = None
        if weight is not None:
            _want(weight, name + "_weight", dev, x.dtype, dim)
            dweight = torch.empty(dim, dtype=torch.float32, device=dev)
        dx = torch.empty(tokens, heads, dim, dtype=x.dtype, device=dev)
        return dx, dweight, _pack_grad(dy.data_ptr(), got[3], x.data_ptr(), stride, _address(weight),
                                       dx.data_ptr(), heads * dim, _address(dweight), heads)

    dxk = dwk = kb = None
    if k is not None:
        k_tokens, k_heads, k_dim, k_stride = _heads_of(k, "k", dev, (q.dtype,))
        if k_tokens != tokens or k_dim != dim:
            raise ValueError(f"k must be [{tokens}, heads, {dim}], got {tuple(k.shape)}")
        dxk, dwk, kb = pack(dk, k, "k", k_stride, k_heads, k_weight)
    dxq, dwq, qb = pack(dq, q, "q", stride, heads, q_weight)
    lib = load_library()
    size = 0
    if q_weight is not None or k_weight is not None:
        size = lib.mx_norm_rotate_backward_workspace_size(tokens, dim)
    ws = _scratch(size, dev)
    _call(dev, lib.mx_norm_rotate_backward, qb, kb, _DTYPES[q.dtype], tokens, dim, eps, r, _ptr(ws),
          size)
    return dxq, dxk, dwq, dwk


def kv_append_rotary(cache: KVCache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor,
                     cu: torch.Tensor, lengths: torch.Tensor, rotary: Rotary | None = None,
                     weight: torch.Tensor | None = None, eps: float = 1e-6) -> None:
    """kv_append with the keys' norm (weight [dim]; None: no norm) and rotation
    (None: none) on the way. Without positions a token turns by its place in its
    sequence."""
    dev, held_heads, held_dim, _, c = _cache_of(cache)
    tokens, heads, dim, stride = _heads_of(k, "k", dev, _DTYPES)
    v_tokens, v_heads, v_dim, v_stride = _heads_of(v, "v", dev, (k.dtype,))
    if v_tokens != tokens or v_heads != heads or v_dim != dim:
        raise ValueError("k and v must have one shape")
    if heads != held_heads or dim != held_dim:
        raise ValueError(f"the cache holds {held_heads} heads of {held_dim}, got {heads} of {dim}")
    if weight is not None:
        _want(weight, "weight", dev, k.dtype, dim)
    r = _rotary_of(rotary, dev, dim, tokens, False)
    b = _batch_of(dev, table, cu, lengths, tokens)[2]
    _call(dev, load_library().mx_kv_append_rotary, k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype],
          stride, v_stride, _ptr(weight), eps, r, c, b)


def kv_attention_tree(q: torch.Tensor, cache: KVCache, table: torch.Tensor, cu: torch.Tensor,
                      lengths: torch.Tensor, mask: torch.Tensor, scale: float | None = None,
                      max_length: int = 0, out: torch.Tensor | None = None) -> torch.Tensor:
    """kv_attention where a sequence's new tokens see each other by `mask` int32
    [tokens, words] (tree_mask): bit b, whether a token sees new token b of its
    sequence. Every key before the new tokens is seen."""
    dev, heads, held_dim, page, c = _cache_of(cache)
    tokens, q_heads, dim, stride = _heads_of(q, "q", dev, (torch.bfloat16,))
    if dim != held_dim:
        raise ValueError(f"the cache holds heads of {held_dim}, got {dim}")
    if q_heads < heads or q_heads % heads:
        raise ValueError(f"q_heads must be a multiple of the cache's {heads}, got {q_heads}")
    if not isinstance(mask, _Tensor) or len(mask.shape) != 2 or mask.shape[1] < 1:
        raise ValueError("mask must be [tokens, words]")
    words = mask.shape[1]
    _want(mask, "mask", dev, _I32, tokens * words)
    batch, width, b = _batch_of(dev, table, cu, lengths, tokens)
    if out is None:
        out = torch.empty(tokens, q_heads, dim, dtype=torch.bfloat16, device=dev)
    else:
        _want(out, "out", dev, torch.bfloat16, tokens * q_heads * dim, dim)
    room = width * page
    max_length = room if max_length <= 0 else min(max_length, room)
    lib = load_library()
    size = lib.mx_kv_attention_tree_workspace_size(tokens, batch, q_heads, heads, dim, max_length)
    ws = _scratch(size, dev)
    _call(dev, lib.mx_kv_attention_tree, q.data_ptr(), stride, q_heads, c, b, mask.data_ptr(), words,
          max_length, 1.0 / math.sqrt(dim) if scale is None else scale, out.data_ptr(), _ptr(ws), size)
    return out


def verify_drafts(target: torch.Tensor, ids: torch.Tensor, parents: torch.Tensor,
                  cu: torch.Tensor, numbers: torch.Tensor, width: int,
                  draft: torch.Tensor | None = None):
    """Walk down each sequence's tree of drafted tokens as far as the target's
    probabilities agree -> (path int32 [batch, width]: the nodes, 0 first, then -1;
    count int32 [batch]; token int32 [batch]: the next token). target [tokens,
    vocab] (and draft, if its probabilities are known); ids, parents int32
    [tokens]; cu int32 [batch + 1]; numbers float32 [tokens, 2], uniform from 0 to
    below 1. width: the longest path, node 0 included (the tree's depth + 1)."""
    dev = _on_gpu(target, "target")
    if target.dtype not in _DTYPES or len(target.shape) != 2 or not target.is_contiguous():
        raise ValueError("target must be contiguous [tokens, vocab], float32 or bfloat16")
    tokens, vocab = target.shape
    if draft is not None:
        _want(draft, "draft", dev, target.dtype, tokens * vocab, vocab)
    _want(ids, "ids", dev, _I32, tokens)
    _want(parents, "parents", dev, _I32, tokens)
    if not isinstance(cu, _Tensor) or len(cu.shape) != 1 or not cu.shape[0]:
        raise ValueError("cu must be [batch + 1]")
    batch = cu.shape[0] - 1
    _want(cu, "cu", dev, _I32, batch + 1)
    _want(numbers, "numbers", dev, _F32, 2 * tokens, 2)
    if not 1 <= width <= 1024:
        raise ValueError(f"width must be 1 to 1024, got {width}")
    path = torch.empty(batch, width, dtype=_I32, device=dev)
    count = torch.empty(batch, dtype=_I32, device=dev)
    token = torch.empty(batch, dtype=_I32, device=dev)
    lib = load_library()
    size = lib.mx_verify_drafts_workspace_size(tokens, batch, vocab)
    ws = _scratch(size, dev)
    _call(dev, lib.mx_verify_drafts, target.data_ptr(), _ptr(draft), _DTYPES[target.dtype],
          ids.data_ptr(), parents.data_ptr(), cu.data_ptr(), numbers.data_ptr(), tokens, batch, vocab,
          width, path.data_ptr(), count.data_ptr(), token.data_ptr(), _ptr(ws), size)
    return path, count, token


def kv_keep(cache: KVCache, table: torch.Tensor, lengths: torch.Tensor, path: torch.Tensor,
            count: torch.Tensor) -> None:
    """Keep the accepted tokens in the cache, in place: behind the lengths int32
    [batch] that each sequence held, new token path[i][j] moves to place j, for j
    below count[i] (verify_drafts gives both). It then holds lengths + count."""
    dev, _, _, _, c = _cache_of(cache)
    if not isinstance(table, _Tensor) or len(table.shape) != 2:
        raise ValueError("table must be [batch, width]")
    batch, width = table.shape
    if not isinstance(path, _Tensor) or len(path.shape) != 2 or path.shape[0] != batch:
        raise ValueError(f"path must be [{batch}, width]")
    _want(table, "table", dev, _I32, batch * width)
    _want(lengths, "lengths", dev, _I32, batch)
    _want(path, "path", dev, _I32, path.numel())
    _want(count, "count", dev, _I32, batch)
    b = _pack_batch(table.data_ptr(), 0, lengths.data_ptr(), 0, batch, width)
    _call(dev, load_library().mx_kv_keep, c, b, path.data_ptr(), path.shape[1], count.data_ptr())
