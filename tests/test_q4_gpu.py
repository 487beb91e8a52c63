"""GPU parity of tq2_q4_gemv against the definition in float64.

Tolerance 1e-5 * S with S = sum_k |x w| + |residual|: codes and scales are
exact, x = hi + lo is within 2^-22 |x| (two binary16 roundings of 2^-11), and a
sum passes at most about 150 f32 roundings of 2^-24 (128 terms of a group in
the matrix core, the groups of a wave's columns, eight waves): 9e-6.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOL = 1e-5


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    from gemv_tq2_g128_amd import q4 as mod
    return mod


def make(seed, m, n, k, group, residual=False, spread=False):
    rng = np.random.default_rng(seed)
    c = {"codes": rng.integers(0, 256, (n, k // 2), dtype=np.uint8),
         "scales": rng.uniform(-0.02, 0.02, (n, k // group)).astype(np.float16),
         "x": rng.standard_normal((m, k)).astype(np.float32),
         "residual": rng.standard_normal((m, n)).astype(np.float32) if residual else None}
    if spread:                  # columns over twelve binary orders, rows over sixty
        c["x"] *= np.exp2(rng.integers(-6, 7, k)).astype(np.float32)
        c["x"] *= np.exp2(np.linspace(-30, 30, m)).astype(np.float32)[:, None]
    return c


def expected(c):
    n, k = c["codes"].shape[0], 2 * c["codes"].shape[1]
    w = np.empty((n, k))
    w[:, 0::2] = (c["codes"] & 15).astype(np.float64) - 8
    w[:, 1::2] = (c["codes"] >> 4).astype(np.float64) - 8
    w *= np.repeat(c["scales"].astype(np.float64), k // c["scales"].shape[1], axis=1)
    x = c["x"].astype(np.float64)
    y, s = x @ w.T, np.abs(x) @ np.abs(w).T
    if c["residual"] is not None:
        y, s = y + c["residual"], s + np.abs(c["residual"])
    return y, s


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(q4, c, label):
    y = q4.gemv(dev(c["codes"]), dev(c["scales"]), dev(c["x"]), residual=dev(c["residual"]))
    torch.cuda.synchronize()
    ref, s = expected(c)
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    worst = float((err / np.maximum(s, 1e-300)).max())
    print(label, "worst err/S %.3g" % worst, flush=True)
    assert np.all(err <= TOL * s), label


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 16])
def test_rows_of_x(q4, m, group):
    check(q4, make(m, m, 100, 1152, group, residual=m % 2 == 0), "m%d g%d" % (m, group))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("k", [128, 384, 1024, 4096, 4224, 8192, 12416])
def test_columns(q4, k, group):
    """One 128-wide block, blocks that leave waves idle, one pass over K, and several with a short last one."""
    check(q4, make(k, 3, 50, k, group, residual=True), "k%d g%d" % (k, group))
    check(q4, make(k + 1, 11, 20, k, group), "m11 k%d g%d" % (k, group))


@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 33, 4097, 16384, 16401, 33000])
def test_weight_rows(q4, n):
    """Tiles that end early, one and two row tiles per step, and blocks that walk over several steps."""
    check(q4, make(n, 1, n, 256, 128, residual=True), "n%d" % n)
    check(q4, make(n + 1, 8, n, 384, 32), "m8 n%d" % n)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,k", [(1, 128), (5, 1152), (8, 4224), (9, 2304), (16, 1280)])
def test_many_weight_rows(q4, m, k, group):
    """Tiles walked by single waves: columns that end inside a round, one pass over K and several, a last tile that
    ends early.  (The reference is taken on the GPU, in float64.)"""
    n = 65543
    gen = torch.Generator(device="cuda").manual_seed(m + k)
    codes = torch.randint(0, 256, (n, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(n, k // group, generator=gen, device="cuda") * 0.04 - 0.02).half()
    x = torch.randn(m, k, generator=gen, device="cuda")
    res = torch.randn(m, n, generator=gen, device="cuda") if m != 5 else None
    y = q4.gemv(codes, scales, x, residual=res)
    w = (torch.stack((codes & 15, codes >> 4), -1).flatten(1).double() - 8) * \
        scales.double().repeat_interleave(group, 1)
    ref, s = torch.mm(x.double(), w.T.contiguous()), torch.mm(x.double().abs(), w.abs().T.contiguous())
    if res is not None:
        ref, s = ref + res, s + res.abs()
    err = (y.double() - ref).abs()
    print("tall m%d k%d g%d worst err/S %.3g" % (m, k, group, float((err / s).max())), flush=True)
    assert bool((err <= TOL * s).all())


def test_inputs_at_the_end_of_their_memory(q4):
    """Scales and codes whose last row ends with the allocation, an odd number of scales in a row."""
    for n in (5, 65541):
        c = make(n, 2, n, 1152, 128)
        codes, scales = dev(c["codes"]), dev(c["scales"])
        y = q4.gemv(codes, scales, dev(c["x"])).cpu().numpy()
        ref, s = expected(c)
        assert np.all(np.abs(y - ref) <= TOL * s), n


def test_refusals_name_the_argument(q4):
    codes = torch.zeros(8, 128, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(8, 2, dtype=torch.float16, device="cuda")
    x = torch.zeros(2, 256, device="cuda")
    for args, more, match in (((codes.int(), scales, x), {}, "codes must have dtype"),
                              ((codes, scales.float(), x), {}, "scales must have dtype"),
                              ((codes, scales, x.double()), {}, "x must have dtype"),
                              ((codes, scales, x[:, ::2]), {}, "x must be contiguous"),
                              ((codes, scales, x), dict(residual=x[:1]), "residual must be contiguous"),
                              ((codes, scales, x), dict(out=x), "out must be contiguous"),
                              ((codes.cpu(), scales, x), {}, "codes must be a device tensor")):
        with pytest.raises(ValueError, match=match):
            q4.gemv(*args, **more)
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        q4.gemv(codes, scales, None)
    with pytest.raises(RuntimeError, match="q4_gemv"):
        q4.gemv(codes, scales, torch.zeros(17, 256, device="cuda"))


@pytest.mark.parametrize("m", [1, 8, 16])
def test_magnitudes_of_x(q4, m):
    """Rows of x sixty binary orders apart keep their own accuracy."""
    check(q4, make(70 + m, m, 64, 1024, 64, spread=True), "spread m%d" % m)


def test_every_code_at_every_place(q4):
    """A unit vector reads one weight of each row back, exactly: (code - 8) * scale has no rounding in f32."""
    k, n = 256, 16
    codes = np.add.outer(np.arange(n), np.arange(k)) % 16
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    for group in (32, 64, 128):
        scales = (0.5 + np.arange(n * (k // group)).reshape(n, -1) / 64.0).astype(np.float16)
        w = (codes - 8) * np.repeat(scales.astype(np.float64), group, axis=1)
        for lo in range(0, k, 16):
            x = np.zeros((16, k), dtype=np.float32)
            x[np.arange(16), lo + np.arange(16)] = 1.0
            y = q4.gemv(dev(packed), dev(scales), dev(x)).cpu().numpy()
            assert np.array_equal(y, w[:, lo:lo + 16].T.astype(np.float32)), (group, lo)


def test_zero_and_tiny_x(q4):
    c = make(5, 4, 40, 512, 32)
    c["x"][0] = 0.0
    c["x"][1] = 1e-40            # subnormal
    c["x"][2, 128:] = 0.0        # whole blocks of zeros
    y = q4.gemv(dev(c["codes"]), dev(c["scales"]), dev(c["x"])).cpu().numpy()
    assert np.all(y[0] == 0.0) and np.all(np.isfinite(y))
    ref, s = expected(c)
    assert np.all(np.abs(y[2:] - ref[2:]) <= TOL * s[2:])


def test_a_non_finite_row_stays_alone(q4):
    c = make(6, 8, 40, 512, 128)
    c["x"][3, 100] = np.inf
    c["x"][5, 7] = np.nan
    y = q4.gemv(dev(c["codes"]), dev(c["scales"]), dev(c["x"])).cpu().numpy()
    rows = [0, 1, 2, 4, 6, 7]
    c["x"][3, 100] = c["x"][5, 7] = 0.0
    ref, s = expected(c)
    assert np.all(np.abs(y[rows] - ref[rows]) <= TOL * s[rows])
    assert not np.isfinite(y[5]).any()


def test_in_place_residual_vector_and_stream(q4):
    c = make(7, 1, 300, 4224, 128, residual=True)
    ref, s = expected(c)
    codes, scales, x = dev(c["codes"]), dev(c["scales"]), dev(c["x"])
    out = dev(c["residual"])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        q4.gemv(codes, scales, x, residual=out, out=out)
    stream.synchronize()
    assert np.all(np.abs(out.cpu().numpy() - ref) <= TOL * s)
    y = q4.gemv(codes, scales, x[0])
    assert y.shape == (300,)


def test_graph_replays_match_eager(q4):
    c = make(8, 5, 1000, 1152, 64, residual=True)
    codes, scales, x, res = (dev(c[n]) for n in ("codes", "scales", "x", "residual"))
    out = torch.empty(5, 1000, device="cuda")
    eager = q4.gemv(codes, scales, x, residual=res).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.gemv(codes, scales, x, residual=res, out=out)
    for replay in range(3):
        out.fill_(float("nan"))
        q4.gemv(codes, scales, x * (replay + 2.0))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), replay
