"""Python binding of the 4-bit matrix-vector products (include/tq2_q4.h).

A weight of [n, k] is two plain tensors: ``codes`` uint8 [n, k / 2] (weight 2j
of a row in the low nibble of byte j) and ``scales`` float16 [n, k / group]; its
value is (code - 8) * scale.  Argument marshalling only, as in ``tq2``.
"""

from __future__ import annotations

import ctypes

from .tq2 import _check, _launch, _one_device, _require, _torch, lib

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
    torch = _torch()
    if codes.dim() != 2 or scales.dim() != 2 or x.dim() not in (1, 2):
        raise ValueError("codes and scales must be matrices, x a matrix or a vector")
    n, k = codes.shape[0], 2 * codes.shape[1]
    m = x.shape[0] if x.dim() == 2 else 1
    per_row = scales.shape[1]
    if per_row == 0 or k % per_row or k // per_row not in GROUPS:
        raise ValueError("scales must be [n, k / group] with a group of 32, 64 or 128")
    _require(codes, torch.uint8, n * k // 2, "codes")
    _require(scales, torch.float16, n * per_row, "scales")
    _require(x, torch.float32, m * k, "x")
    if residual is not None:
        _require(residual, torch.float32, m * n, "residual")
    if out is None:
        out = torch.empty(x.shape[:-1] + (n,), dtype=torch.float32, device=x.device)
    _require(out, torch.float32, m * n, "out")
    dev = _one_device(("x", x), ("codes", codes), ("scales", scales), ("residual", residual),
                      ("out", out))
    _check(_launch(dev, gemv_ptr, codes.data_ptr(), scales.data_ptr(), x.data_ptr(),
                   residual.data_ptr() if residual is not None else 0, out.data_ptr(), m, n, k,
                   k // per_row), "q4_gemv")
    return out
