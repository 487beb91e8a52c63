"""Places of new tokens for lengths and offsets that no sequence has (csrc/tq2_pages.h, compiled for the host)."""

import ctypes

import pytest

torch = pytest.importorskip("torch")
from tests.test_attn_cpu import pages_lib  # noqa: E402, F401


def test_places_do_not_wrap(pages_lib):  # noqa: F811
    """A row's place is its distance from the sequence's end, cut to 32 bits: never a place that it does not have."""
    edge = [-2 ** 31, -2 ** 31 + 1, -7, 0, 5, 1000, 2 ** 31 - 1]
    for length in edge:
        for lo in edge:
            for hi in edge:
                kv, cu = torch.tensor([length], dtype=torch.int32), torch.tensor([lo, hi], dtype=torch.int32)
                out = (ctypes.c_int32 * 4)()
                pages_lib.seq(ctypes.c_void_p(kv.data_ptr()), ctypes.c_void_p(cu.data_ptr()), 1, 17, 4, 4, 0, out)
                q0, q_len, first, keys = out
                if q_len:
                    assert first == max(-2 ** 31, length - (hi - q0)), (length, lo, hi)
                    assert first + q_len - 1 < max(length, 0) or first + q_len - 1 < 0, (length, lo, hi)
