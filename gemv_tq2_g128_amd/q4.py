"""Python binding of the 4-bit matrix-vector products (include/tq2_q4.h).

A weight of [n, k] is two plain tensors: ``codes`` uint8 [n, k / 2] (weight 2j
of a row in the low nibble of byte j) and ``scales`` float16 [n, k / group]; its
value is (code - 8) * scale.  Argument marshalling only, as in ``tq2``: tensors go
through the compiled module ``_binding`` (csrc/tq2_binding.cpp).
"""

from __future__ import annotations

import ctypes

from .tq2 import _result, lib     # first: it loads torch and libtq2, which _binding needs
from . import _binding            # isort: skip

EXPORTED_SYMBOLS = ("tq2_q4_gemv",)
MAX_M = 16                      # TQ2_Q4_MAX_M (include/tq2_q4.h)
GROUPS = (32, 64, 128)

_vp, _i64 = ctypes.c_void_p, ctypes.c_int64
lib.tq2_q4_gemv.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_int, _vp]
lib.tq2_q4_gemv.restype = ctypes.c_int


def gemv_ptr(codes_ptr: int, scales_ptr: int, x_ptr: int, residual_ptr: int, out_ptr: int, m: int,
             n: int, k: int, group: int, stream: int = 0) -> int:
    return lib.tq2_q4_gemv(codes_ptr or None, scales_ptr or None, x_ptr or None,
                           residual_ptr or None, out_ptr or None, m, n, k, group, stream or None)


def gemv(codes, scales, x, residual=None, out=None):
    """out[m, n] = residual[m, n] + sum_k x[m, k] * (code[n, k] - 8) * scale[n, k // group];
    x is f32 [m, k] (or [k], for an out of [n]) with m <= MAX_M.  The group is
    k / scales.shape[1]: 32, 64 or 128."""
    return _result(_binding.q4_gemv(codes, scales, x, residual, out), "q4_gemv")
