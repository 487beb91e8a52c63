"""Python binding of the paged-cache operators (include/tq2_attn.h).

A cache is two tensors ``k_cache`` and ``v_cache`` of [pages, kv_heads, page,
head_dim] (any strides with contiguous components: pass ``x.transpose(1, 2)``
of a [pages, page, kv_heads, head_dim] cache), an int32 block table [batch,
columns] and the int32 lengths ``kv_len`` [batch], new tokens included.  The rows
of sequence b are ``cu_q[b]`` .. ``cu_q[b + 1]``; without ``cu_q`` each sequence
has one.  Argument marshalling only, as in ``tq2``.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from .tq2 import _check, _launch_on, lib

EXPORTED_SYMBOLS = ("tq2_kv_append", "tq2_paged_attention", "tq2_paged_attention_workspace_bytes")
HEAD_DIMS = (64, 96, 128, 192, 256)

_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.float8_e4m3fn: 3}
# tq2_paged_cache and what follows it in the two argument structs: every field is 8 bytes wide.
_CACHE = struct.Struct("=7Q17q")
_APPEND = struct.Struct("=4Q8q2Q6q2Qd")
_ATTENTION = struct.Struct("=2Q7qdQq")

lib.tq2_kv_append.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
lib.tq2_kv_append.restype = ctypes.c_int
lib.tq2_paged_attention.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
lib.tq2_paged_attention.restype = ctypes.c_int
lib.tq2_paged_attention_workspace_bytes.argtypes = [ctypes.c_char_p]
lib.tq2_paged_attention_workspace_bytes.restype = ctypes.c_size_t


def kv_append_ptr(args: bytes, stream: int = 0) -> int:
    """args: the bytes of a tq2_kv_append_args."""
    return lib.tq2_kv_append(args, stream or None)


def paged_attention_ptr(args: bytes, stream: int = 0) -> int:
    """args: the bytes of a tq2_paged_attention_args."""
    return lib.tq2_paged_attention(args, stream or None)


def paged_attention_workspace_bytes_ptr(args: bytes) -> int:
    return lib.tq2_paged_attention_workspace_bytes(args)


def _on(dev: int, t, what: str):
    if t.get_device() != dev:
        if t.get_device() < 0:
            raise ValueError("%s must be a device tensor" % what)
        raise ValueError("%s is on %s, the other tensors on cuda:%d" % (what, t.device, dev))


def _plain(dev: int, t, dtype, numel: int, what: str) -> int:
    """Address of a contiguous tensor of this type and size, or 0 for None."""
    if t is None:
        return 0
    _on(dev, t, what)
    if t.dtype is not dtype:
        raise ValueError("%s must have dtype %s, got %s" % (what, dtype, t.dtype))
    if t.numel() != numel or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %d elements" % (what, numel))
    return t.data_ptr()


def _rows(dev: int, t, dtype, shape, what: str):
    """Token and head stride of a [tokens, heads, head_dim] tensor."""
    _on(dev, t, what)
    if t.dtype is not dtype:
        raise ValueError("%s must have dtype %s, got %s" % (what, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (what, list(shape), list(t.shape)))
    st = t.stride()
    if st[2] != 1:
        raise ValueError("%s must have contiguous components" % what)
    return st[0], st[1]


def _cache(dev, act, tokens, q_heads, k_cache, v_cache, kv_len, table, cu_q, k_scale, v_scale) -> bytes:
    """The bytes of a tq2_paged_cache."""
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be [pages, kv_heads, page, head_dim]")
    pages, kv_heads, page, dim = k_cache.shape
    kind = k_cache.dtype
    if kind not in _TYPES or v_cache.dtype is not kind:
        raise ValueError("k_cache and v_cache must have one dtype of float16, bfloat16 and float8_e4m3fn")
    _on(dev, k_cache, "k_cache")
    _on(dev, v_cache, "v_cache")
    ks, vs = k_cache.stride(), v_cache.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("k_cache and v_cache must have contiguous components")
    _on(dev, table, "table")
    if table.dim() != 2 or table.dtype is not torch.int32 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be an int32 matrix with contiguous rows")
    batch, cols = table.shape
    return _CACHE.pack(
        k_cache.data_ptr(), v_cache.data_ptr(), _plain(dev, k_scale, torch.float32, kv_heads, "k_scale"),
        _plain(dev, v_scale, torch.float32, kv_heads, "v_scale"), table.data_ptr(),
        _plain(dev, kv_len, torch.int32, batch, "kv_len"), _plain(dev, cu_q, torch.int32, batch + 1, "cu_q"),
        batch, tokens, pages, page, cols, table.stride(0), kv_heads, q_heads, dim, _TYPES.get(act, -1),
        _TYPES[kind], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2])


def kv_append(k, v, k_cache, v_cache, kv_len, table, q=None, q_out=None, cu_q=None, freqs=None, positions=None,
              sections=None, interleaved=False, q_norm=None, k_norm=None, eps=1e-6, k_scale=None, v_scale=None):
    """Normalise and rotate q [tokens, q_heads, head_dim] and k [tokens, kv_heads, head_dim], store k and v in the
    cache and q in ``q_out`` (made if absent; may be q itself), which is returned.

    ``freqs`` f64 [rot / 2]: the leading ``rot`` components are rotated by position * freqs, pairs (i, i + rot / 2) or,
    ``interleaved``, (2i, 2i + 1).  The position is the place in the cache, or ``positions`` int32 [tokens] or [axes,
    tokens] with ``sections``, the number of angles that follow each axis.  ``q_norm``, ``k_norm`` f32 [head_dim]: RMS
    norms before the rotation.  ``k_scale``, ``v_scale`` f32 [kv_heads]: scales of an 8-bit cache."""
    if k.dim() != 3:
        raise ValueError("k must be [tokens, kv_heads, head_dim]")
    dev = k.get_device()
    if dev < 0:
        raise ValueError("k must be a device tensor")
    tokens, kv_heads, dim = k.shape
    act = k.dtype
    if k_cache.dim() == 4 and (k_cache.shape[1] != kv_heads or k_cache.shape[3] != dim):
        raise ValueError("k must be [tokens, %d, %d] for this cache" % (k_cache.shape[1], k_cache.shape[3]))
    k_st = _rows(dev, k, act, k.shape, "k")
    v_st = _rows(dev, v, act, k.shape, "v")
    q_heads, q_st, o_st, q_ptr, o_ptr = kv_heads, (0, 0), (0, 0), 0, 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [tokens, q_heads, head_dim]")
        q_heads = q.shape[1]
        shape = (tokens, q_heads, dim)
        q_st = _rows(dev, q, act, shape, "q")
        if q_out is None:
            q_out = torch.empty(shape, dtype=act, device=q.device)
        o_st = _rows(dev, q_out, act, shape, "q_out")
        q_ptr, o_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    half = 0 if freqs is None else freqs.numel()
    axes, cuts = 1, (half, 0, 0)
    if positions is not None:
        axes = positions.shape[0] if positions.dim() == 2 else 1
        if sections is not None:
            cuts = (tuple(sections) + (0, 0, 0))[:3]
        if axes < 1 or axes > 3 or (sections is not None and len(sections) != axes) or \
                (sections is None and axes != 1):
            raise ValueError("positions must be [tokens] or [axes, tokens], with one section for each of at most 3 axes")
    elif sections is not None and len(sections) != 1:
        raise ValueError("sections without positions")
    cache = _cache(dev, act, tokens, q_heads, k_cache, v_cache, kv_len, table, cu_q, k_scale, v_scale)
    args = cache + _APPEND.pack(
        q_ptr, k.data_ptr(), v.data_ptr(), o_ptr, *q_st, *k_st, *v_st, *o_st,
        _plain(dev, freqs, torch.float64, half, "freqs"),
        _plain(dev, positions, torch.int32, axes * tokens, "positions"), 2 * half, axes, *cuts, int(interleaved),
        _plain(dev, q_norm, torch.float32, dim, "q_norm"), _plain(dev, k_norm, torch.float32, dim, "k_norm"), eps)
    _check(_launch_on(dev, kv_append_ptr, args), "kv_append")
    return q_out


def paged_attention(q, k_cache, v_cache, kv_len, table, cu_q=None, max_q=None, max_kv=None, window=0, scale=None,
                    k_scale=None, v_scale=None, out=None):
    """softmax(scale * q K^T) V of q [tokens, q_heads, head_dim] over the cache, each token seeing its sequence up to
    itself (the last ``window`` tokens of that, if given); rows that see nothing give zeros.

    ``max_q`` and ``max_kv``, the most new tokens and the most tokens of a sequence, shape the launch (by default all
    of q and all that the table holds); larger ones are still done.  ``scale`` is 1 / sqrt(head_dim) by default.
    ``out`` may be q itself."""
    if q.dim() != 3:
        raise ValueError("q must be [tokens, q_heads, head_dim]")
    dev = q.get_device()
    if dev < 0:
        raise ValueError("q must be a device tensor")
    tokens, q_heads, dim = q.shape
    act = q.dtype
    if k_cache.dim() == 4 and k_cache.shape[3] != dim:
        raise ValueError("q must be [tokens, q_heads, %d] for this cache" % k_cache.shape[3])
    if out is None:
        out = torch.empty(q.shape, dtype=act, device=q.device)
    q_st, o_st = _rows(dev, q, act, q.shape, "q"), _rows(dev, out, act, q.shape, "out")
    cache = _cache(dev, act, tokens, q_heads, k_cache, v_cache, kv_len, table, cu_q, k_scale, v_scale)
    if max_q is None:
        max_q = 1 if cu_q is None else tokens
    if max_kv is None:
        max_kv = min(table.shape[1] * k_cache.shape[2], 2 ** 31 - 1)
    if scale is None:
        scale = dim ** -0.5
    sizes = (q.data_ptr(), out.data_ptr(), *q_st, *o_st, max_q, max_kv, window, scale)
    need = paged_attention_workspace_bytes_ptr(cache + _ATTENTION.pack(*sizes, 0, 0))
    workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    args = cache + _ATTENTION.pack(*sizes, workspace.data_ptr() if need else 0, need)
    _check(_launch_on(dev, paged_attention_ptr, args), "paged_attention")
    return out
