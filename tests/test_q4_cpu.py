"""CPU checks of tq2_q4_gemv: the header's symbols are exported and every refusal comes before any device work."""

import ctypes
import os
import re

import pytest

from gemv_tq2_g128_amd import q4, tq2

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x7F0000000000              # never dereferenced
X, S, O, R = A + (1 << 36), A + (2 << 36), A + (3 << 36), A + (4 << 36)


def call(codes=A, scales=S, x=X, residual=0, out=O, m=2, n=8, k=256, group=128):
    return q4.gemv_ptr(codes, scales, x, residual, out, m, n, k, group)


def test_header_and_binding_agree():
    with open(os.path.join(ROOT, "include", "tq2_q4.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    assert tuple(sorted(set(re.findall(r"\b(tq2_[a-z0-9_]+)\s*\(", text)))) == q4.EXPORTED_SYMBOLS
    assert int(re.search(r"#define\s+TQ2_Q4_MAX_M\s+(\d+)", text).group(1)) == q4.MAX_M
    handle = ctypes.CDLL(tq2.LIB_PATH)
    for name in q4.EXPORTED_SYMBOLS:
        assert hasattr(handle, name)


@pytest.mark.parametrize("bad", ["codes", "scales", "x", "out"])
def test_null_pointers(bad):
    assert call(**{bad: 0}) == tq2.TQ2_ERR_INVALID


@pytest.mark.parametrize("sizes", [dict(m=-1), dict(n=-1), dict(k=0), dict(k=-128), dict(m=q4.MAX_M + 1),
                                   dict(n=(1 << 30) + 1), dict(k=(1 << 21) + 128), dict(group=0), dict(group=16),
                                   dict(group=256), dict(group=-32)])
def test_sizes_out_of_range(sizes):
    assert call(**sizes) == tq2.TQ2_ERR_INVALID


@pytest.mark.parametrize("k", [1, 32, 64, 127, 129, 200])
def test_k_not_a_multiple_of_128(k):
    assert call(k=k) == tq2.TQ2_ERR_SHAPE


@pytest.mark.parametrize("name,base", [("codes", A), ("scales", S), ("x", X), ("out", O), ("residual", R)])
def test_alignment(name, base):
    for off in (1, 2, 4, 8):
        assert call(**{name: base + off}) == tq2.TQ2_ERR_ALIGN


def test_aliasing():
    assert call(out=X) == tq2.TQ2_ERR_ALIAS
    assert call(out=X + 2 * 256 * 4 - 16) == tq2.TQ2_ERR_ALIAS       # the last bytes of x
    assert call(out=A + 8 * 128 - 16) == tq2.TQ2_ERR_ALIAS           # of the codes
    assert call(out=S + 16) == tq2.TQ2_ERR_ALIAS                     # of the scales
    assert call(residual=O + 16) == tq2.TQ2_ERR_ALIAS                # part of the residual


def test_empty_problems_are_no_ops():
    assert q4.gemv_ptr(0, 0, 0, 0, 0, 0, 8, 256, 128) == tq2.TQ2_OK
    assert q4.gemv_ptr(0, 0, 0, 0, 0, 2, 0, 256, 128) == tq2.TQ2_OK
    assert q4.gemv_ptr(0, 0, 0, 0, 0, 0, 8, 200, 128) == tq2.TQ2_ERR_SHAPE


def test_valid_arguments_reach_the_device_check():
    torch = pytest.importorskip("torch")
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible; this check is for GPU-less hosts")
    assert call() == tq2.TQ2_ERR_DEVICE
    assert call(residual=O) == tq2.TQ2_ERR_DEVICE                    # in place
    assert call(residual=R, m=q4.MAX_M, group=32) == tq2.TQ2_ERR_DEVICE


def test_front_end_checks():
    torch = pytest.importorskip("torch")
    codes = torch.zeros(8, 128, dtype=torch.uint8)
    scales = torch.zeros(8, 2, dtype=torch.float16)
    x = torch.zeros(2, 256)
    with pytest.raises(ValueError, match="device tensor"):
        q4.gemv(codes, scales, x)
    with pytest.raises(ValueError, match="group of 32"):
        q4.gemv(codes, torch.zeros(8, 3, dtype=torch.float16), x)
    with pytest.raises(ValueError, match="group of 32"):
        q4.gemv(codes, torch.zeros(8, 16, dtype=torch.float16), x)
    with pytest.raises(ValueError, match="matrices"):
        q4.gemv(codes.reshape(-1), scales, x)
