"""Python binding of the mixture-of-experts operators (include/tq2_moe.h).

``route`` chooses each token's experts, ``experts`` runs them.  The experts' weights are the framework's own formats:

* 4-bit, as in ``q4``: ``(codes, scales)`` with codes uint8 [experts, n, k / 2] and scales float16 [experts, n, k / group];
* ternary, as in ``tq2``: what ``tq2.reformat_aos_to_soa(blocks, experts * n, k)`` gives for the experts' rows one after
  another.

``gate_up`` has n = 2 * inter rows for each expert, its gate rows first, and ``down`` n = hidden.  Argument marshalling
only, as in ``tq2``: tensors go through the compiled module ``_decode`` (csrc/tq2_decode.cpp), raw pointers through ctypes.
"""

from __future__ import annotations

import ctypes
import struct

from .tq2 import _result, lib     # first: it loads torch and libtq2, which _decode needs
from . import _decode             # isort: skip

EXPORTED_SYMBOLS = ("tq2_moe_experts", "tq2_moe_experts_workspace_bytes", "tq2_moe_route",
                    "tq2_moe_route_workspace_bytes")
MAX_EXPERTS, MAX_TOP_K, MAX_TOKENS, MAX_ROUTE_TOKENS, MAX_DIM = 1024, 16, 128, 1 << 20, 16384
SCORING = ("softmax", "sigmoid")

# tq2_moe_route_args and tq2_moe_experts_args: every field is 8 bytes wide.
_ROUTE = struct.Struct("=5Q8qdQq")
_EXPERTS = struct.Struct("=9Q8qQq")

for _name in ("tq2_moe_route", "tq2_moe_experts"):
    getattr(lib, _name).argtypes = [ctypes.c_char_p, ctypes.c_void_p]
    getattr(lib, _name).restype = ctypes.c_int
    getattr(lib, _name + "_workspace_bytes").argtypes = [ctypes.c_char_p]
    getattr(lib, _name + "_workspace_bytes").restype = ctypes.c_size_t


def route_ptr(args: bytes, stream: int = 0) -> int:
    """args: the bytes of a tq2_moe_route_args."""
    return lib.tq2_moe_route(args, stream or None)


def route_workspace_bytes_ptr(args: bytes) -> int:
    return lib.tq2_moe_route_workspace_bytes(args)


def experts_ptr(args: bytes, stream: int = 0) -> int:
    """args: the bytes of a tq2_moe_experts_args."""
    return lib.tq2_moe_experts(args, stream or None)


def experts_workspace_bytes_ptr(args: bytes) -> int:
    return lib.tq2_moe_experts_workspace_bytes(args)


def route(x, weight, top_k, bias=None, scoring="softmax", renormalize=True, scale=1.0, weights=None, ids=None):
    """The ``top_k`` experts of each token of x [tokens, hidden] by the scores x weight^T, weight [experts, hidden]:
    (weights f32 [tokens, top_k], ids int32 [tokens, top_k]), largest first, the lowest index first among equals.

    The weights are the chosen experts' softmax over all experts, or sigmoid, divided by their sum (``renormalize``) and
    times ``scale``.  ``bias`` f32 [experts] is added to them for the choice alone.  x and weight may be float32, float16
    or bfloat16, each its own; ``weights`` and ``ids`` are made if absent."""
    if scoring not in SCORING:
        raise ValueError("scoring must be one of %s" % (SCORING,))
    return _result(_decode.moe_route(x, weight, top_k, bias, SCORING.index(scoring), bool(renormalize), scale, weights,
                                      ids), "moe.route")


def experts(x, gate_up, down, ids, weights, experts=None, residual=None, out=None):
    """out[t] = residual[t] + sum_j weights[t, j] * (silu(x G^T) * (x U^T)) D^T with expert ids[t, j]'s G, U and D, for
    the at most MAX_TOKENS rows of x [tokens, hidden]; more rows go in slices, a call each, which each read their
    experts' weights.

    ids int32 [tokens, top_k] and weights f32 of the same shape, as ``route`` gives them; a place whose id is no expert
    (-1, say) takes no part.  x, residual and out have one dtype of float32, float16 and bfloat16; out may be x or
    residual itself.  ``experts`` is needed for ternary weights, whose tensors do not tell how many there are."""
    g, gs = gate_up if isinstance(gate_up, (tuple, list)) else (gate_up, None)
    d, ds = down if isinstance(down, (tuple, list)) else (down, None)
    return _result(_decode.moe_experts(x, g, gs, d, ds, ids, weights, experts, residual, out), "moe.experts")
