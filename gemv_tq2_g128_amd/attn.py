"""Python binding of the paged-cache operators (include/tq2_attn.h).

A cache is two tensors ``k_cache`` and ``v_cache`` of [pages, kv_heads, page,
head_dim] (any strides with contiguous components: pass ``x.transpose(1, 2)``
of a [pages, page, kv_heads, head_dim] cache), an int32 block table [batch,
columns] and the int32 lengths ``kv_len`` [batch], new tokens included.  The rows
of sequence b are ``cu_q[b]`` .. ``cu_q[b + 1]``; without ``cu_q`` each sequence
has one.  Argument marshalling only, as in ``tq2``: tensors go through the
compiled module ``_binding`` (csrc/tq2_binding.cpp), raw pointers through ctypes.
"""

from __future__ import annotations

import ctypes
import struct

from .tq2 import _result, lib     # first: it loads torch and libtq2, which _binding needs
from . import _binding            # isort: skip

EXPORTED_SYMBOLS = ("tq2_kv_append", "tq2_paged_attention", "tq2_paged_attention_workspace_bytes")
HEAD_DIMS = (64, 96, 128, 192, 256)

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


def kv_append(k, v, k_cache, v_cache, kv_len, table, q=None, q_out=None, cu_q=None, freqs=None, positions=None,
              sections=None, interleaved=False, q_norm=None, k_norm=None, eps=1e-6, k_scale=None, v_scale=None):
    """Normalise and rotate q [tokens, q_heads, head_dim] and k [tokens, kv_heads, head_dim], store k and v in the
    cache and q in ``q_out`` (made if absent; may be q itself), which is returned.

    ``freqs`` f64 [rot / 2]: the leading ``rot`` components are rotated by position * freqs, pairs (i, i + rot / 2) or,
    ``interleaved``, (2i, 2i + 1).  The position is the place in the cache, or ``positions`` int32 [tokens] or [axes,
    tokens] with ``sections``, the number of angles that follow each axis.  ``q_norm``, ``k_norm`` f32 [head_dim]: RMS
    norms before the rotation.  ``k_scale``, ``v_scale`` f32 [kv_heads]: scales of an 8-bit cache."""
    return _result(_binding.kv_append(k, v, k_cache, v_cache, kv_len, table, cu_q, k_scale, v_scale, q, q_out, freqs,
                                      positions, sections, interleaved, q_norm, k_norm, eps), "kv_append")


def paged_attention(q, k_cache, v_cache, kv_len, table, cu_q=None, max_q=None, max_kv=None, window=0, scale=None,
                    k_scale=None, v_scale=None, out=None):
    """softmax(scale * q K^T) V of q [tokens, q_heads, head_dim] over the cache, each token seeing its sequence up to
    itself (the last ``window`` tokens of that, if given); rows that see nothing give zeros.

    ``max_q`` and ``max_kv``, the most new tokens and the most tokens of a sequence, shape the launch; larger ones are
    still done.  By default they are all of q and all that the table holds, which is right for one sequence and slow for
    many: a decode batch given with ``cu_q`` takes the form for prompts unless ``max_q`` says 1.  ``scale`` is
    1 / sqrt(head_dim) by default.  ``out`` may be q itself."""
    return _result(_binding.paged_attention(q, k_cache, v_cache, kv_len, table, cu_q, k_scale, v_scale, max_q, max_kv,
                                            window, scale, out), "paged_attention")
