"""Python binding of the token choice (include/tq2_sample.h).

Argument marshalling only, as in ``tq2``: tensors go through the compiled module ``_decode`` (csrc/tq2_decode.cpp), raw
pointers through ctypes.
"""

from __future__ import annotations

import ctypes
import struct

from .tq2 import _result, lib     # first: it loads torch and libtq2, which _decode needs
from . import _decode             # isort: skip

EXPORTED_SYMBOLS = ("tq2_sample", "tq2_sample_workspace_bytes")
MAX_ROWS, MAX_VOCAB = 4096, 1 << 20

_ARGS = struct.Struct("=8Q5q3dQq")       # tq2_sample_args: every field is 8 bytes wide

lib.tq2_sample.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
lib.tq2_sample.restype = ctypes.c_int
lib.tq2_sample_workspace_bytes.argtypes = [ctypes.c_char_p]
lib.tq2_sample_workspace_bytes.restype = ctypes.c_size_t


def sample_ptr(args: bytes, stream: int = 0) -> int:
    """args: the bytes of a tq2_sample_args."""
    return lib.tq2_sample(args, stream or None)


def sample_workspace_bytes_ptr(args: bytes) -> int:
    return lib.tq2_sample_workspace_bytes(args)


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None, logprob=None):
    """The next token of each row of logits [rows, vocab] (float32, float16 or bfloat16; rows may be strided, expanded or overlapping), int32
    [rows], by the random numbers ``u`` f32 [rows] in [0, 1).

    In falling order of the logits (the lowest index first among equals) the first ``top_k`` tokens are kept, of these
    those with at least ``min_p`` of the largest one's probability, of these the shortest run that holds ``top_p`` of
    their probability; the token is where the running sum passes u times what is kept.  Each setting is a number or a
    device tensor of one for each row (top_k int32, the others f32); temperature 0 takes the largest logit.  ``logprob``
    f32 [rows], if given, gets the token's log probability among those kept.  A row without a logit above -infinity
    gives -1."""
    return _result(_decode.sample(logits, u, temperature, top_k, top_p, min_p, out, logprob), "sampling.sample")
