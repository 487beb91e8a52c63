"""GPU parity of tq2_q4_gemv at the ends of x's range, against the definition in float64.

Tolerance: 1e-5 * S as in test_q4_gpu.py (one rounding more, of scale times sum: 151 * 2^-24 = 9e-6), and where numbers
are not normal, half the least step of f32, 2^-150, for each group and join that is added up, and half the least step of
binary16 times the least power of two, 2^-25 * 2^-126, for each x.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests.test_q4_gpu import TOL, dev, expected, make, q4  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def weights(c):
    return np.abs(expected({**c, "x": np.ones((1, 2 * c["codes"].shape[1]), dtype=np.float32), "residual": None})[1])


@pytest.mark.parametrize("n", [40, 65540])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_tiny_rows(q4, n, group):  # noqa: F811
    """Rows of x from 1e-28 down to the subnormal numbers, weights of ordinary size."""
    c = make(n + group, 14, n, 512, group)
    c["scales"] = (c["scales"].astype(np.float32) * 0.05).astype(np.float16)
    c["x"] *= (10.0 ** np.linspace(-28, -41, 14)).astype(np.float32)[:, None]
    ref, s = expected(c)
    tol = TOL * s + 2.0 ** -150 * (512 // group + 10) + 2.0 ** -151 * weights(c)
    for rows in (slice(0, 14), slice(3, 9)):                       # two operands for high and low parts, one for both
        y = q4.gemv(dev(c["codes"]), dev(c["scales"]), dev(c["x"][rows])).cpu().numpy().astype(np.float64)
        err = np.abs(y - ref[rows])
        print("tiny n%d g%d worst err / tol" % (n, group), np.round((err / tol[rows]).max(1), 3), flush=True)
        assert np.all(err <= tol[rows])


@pytest.mark.parametrize("group", [32, 128])
def test_huge_rows(q4, group):  # noqa: F811
    """x near the end of f32 and scales near binary16's least: the results are ordinary numbers."""
    c = make(group, 3, 40, 512, group)
    c["scales"] = np.full_like(c["scales"], 2.0 ** -20)
    c["x"] = (np.clip(c["x"], -3, 3) * 1e38).astype(np.float32)
    ref, s = expected(c)
    y = q4.gemv(dev(c["codes"]), dev(c["scales"]), dev(c["x"])).cpu().numpy().astype(np.float64)
    assert np.all(np.abs(y - ref) <= TOL * s)
