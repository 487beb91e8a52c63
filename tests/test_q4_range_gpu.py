"""GPU parity of tq2_q4_gemv at the ends of x's range, against the definition in float64.

Tolerance: 1e-5 * S as in test_q4_gpu.py (one rounding more, of scale times sum: 151 * 2^-24 = 9e-6), and where numbers
are not normal, half the least step of f32, 2^-150, for each group and join that is added up, and half the least step of
binary16 times the least power of two, 2^-25 * 2^-126, for each x.  An x far below the largest of its 128 columns keeps
an error of 2^-25, half the least step of binary16, under a power of two that takes the largest to 2^13 at least: 2^-38 of it.
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


@pytest.mark.parametrize("m", [2, 16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_columns_far_above_the_others(q4, m, group):  # noqa: F811
    """A column of 1e8 that adds nothing, because its weights or its group's scale are zero, and one that does."""
    k, n = 512, 60
    c = make(m + group, m, n, k, group)
    c["x"][:, 5] = 1e8                                             # its codes are 8
    c["codes"][:, 2] = c["codes"][:, 2] & 15 | 8 << 4
    c["x"][:, 128 + 7] = -1e9                                      # its group's scale is zero
    c["scales"][:, 128 // group] = 0
    c["x"][1:, 300] = 1e6
    ref, s = expected(c)
    w = np.empty((n, k))
    w[:, 0::2], w[:, 1::2] = (c["codes"] & 15) - 8.0, (c["codes"] >> 4) - 8.0
    w = np.abs(w * np.repeat(c["scales"].astype(np.float64), group, axis=1))
    top = np.abs(c["x"].astype(np.float64)).reshape(m, -1, 128).max(2).repeat(128, 1)
    tol = TOL * s + 2.0 ** -38 * (top @ w.T)
    y = q4.gemv(dev(c["codes"]), dev(c["scales"]), dev(c["x"])).cpu().numpy().astype(np.float64)
    err = np.abs(y - ref)
    print("far m%d g%d worst err / tol %.3f, err / S %.3g" % (m, group, (err / tol).max(), (err / s).max()), flush=True)
    assert np.all(err <= tol)


@pytest.mark.parametrize("n", [1, 5, 65541])
@pytest.mark.parametrize("k", [128, 1152])
def test_what_follows_the_scales_takes_no_part(q4, n, k):  # noqa: F811
    """An odd number of scales: the last is loaded with the two bytes after it, here NaN."""
    c = make(n + k, 3, n, k, 128)
    count = n * (k // 128)
    held = torch.full((count + 64,), float("nan"), dtype=torch.float16, device="cuda")
    held[:count] = dev(c["scales"]).flatten()
    y = q4.gemv(dev(c["codes"]), held[:count].reshape(n, k // 128), dev(c["x"])).cpu().numpy().astype(np.float64)
    ref, s = expected(c)
    assert np.all(np.abs(y - ref) <= TOL * s)
