"""CPU check of the inputs of tests/test_moe_exact_gpu.py: rows of 30 bits leave the outputs as they are, rows that lack
their lowest byte, or two of them, do not."""

import numpy as np
import pytest

pytest.importorskip("torch")
from tests.moe_exact import Exact, bits  # noqa: E402


@pytest.mark.parametrize("fmt,group", [("q4", 32), ("tq2", 128)])
@pytest.mark.parametrize("scale", [(1.0, 1.0), (2.0 ** -70, 2.0 ** -70), (1.0, 2.0 ** -133)])
def test_every_bit_counts(fmt, group, scale):
    c = Exact(1, 4, 2, 3, 256, fmt, group, scale)
    want = c.out()
    assert np.array_equal(want, want.astype(np.float32)) and np.count_nonzero(want) > 0.9 * want.size
    assert np.array_equal(c.x, c.x.astype(np.float32))
    assert np.array_equal(c.out(bits(30)), want)
    for n in (22, 14):
        wrong = c.out(bits(n)) != want
        assert wrong.any(1).all() and wrong.mean() > 0.5
