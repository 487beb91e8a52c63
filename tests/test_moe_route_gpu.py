"""GPU tests of tq2_moe_route against the definition in float64.

Ids have to be equal: products are exact in f64 and sums pass fewer than 2^14 roundings of 2^-53, 2e-12 of sum |x w| at
the very most, while random scores lie further apart.  Weights: one rounding to f32 (2^-24) beside the f64 steps, 2^-23.9; half
the step of the smallest f32 numbers, 2^-150, where they lie below 2^-126.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import moe_ref as M  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TOL = 2.0 ** -23.9


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    from gemv_tq2_g128_amd import moe as mod
    return mod


def make(seed, tokens, experts, hidden, act, kind, bias=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=g).to(TYPES[act])
    w = (torch.randn(experts, hidden, generator=g) * 2.0 / hidden ** 0.5).to(TYPES[kind])
    b = torch.randn(experts, generator=g) * 0.1 if bias else None
    return x, w, b


def check(moe, x, w, b, top_k, scoring="softmax", renormalize=True, scale=1.0):
    weights, ids = moe.route(x.cuda(), w.cuda(), top_k, bias=None if b is None else b.cuda(), scoring=scoring,
                             renormalize=renormalize, scale=scale)
    torch.cuda.synchronize()
    want, at = M.route(x.double().numpy(), w.double().numpy(), top_k, None if b is None else b.numpy(), scoring,
                       renormalize, scale)
    assert ids.dtype == torch.int32 and weights.dtype == torch.float32 and ids.shape == weights.shape == want.shape
    assert np.array_equal(ids.cpu().numpy(), at)
    err = np.abs(weights.cpu().numpy().astype(np.float64) - want)
    assert (err <= TOL * np.abs(want) + 2.0 ** -150).all(), (err / np.maximum(want, 1e-300)).max()


@pytest.mark.parametrize("act", list(TYPES))
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("tokens", [1, 3, 20])
def test_types(moe, act, kind, tokens):
    check(moe, *make(1, tokens, 60, 520, act, kind), 4)


@pytest.mark.parametrize("tokens,experts,hidden,top_k", [
    (1, 1, 8, 1), (1, 2, 24, 2), (2, 16, 2048, 16), (4, 5, 1000, 5), (5, 63, 264, 3), (8, 64, 4096, 6), (9, 65, 4096, 6),
    (16, 128, 2048, 8), (17, 129, 2056, 8), (33, 256, 7168, 8), (64, 300, 512, 10), (100, 513, 136, 12),
    (15, 1024, 16384, 16), (1, 1024, 16384, 16), (1000, 17, 2880, 4)])
def test_sizes(moe, tokens, experts, hidden, top_k):
    check(moe, *make(2, tokens, experts, hidden, "bf16", "f32"), top_k)


@pytest.mark.parametrize("tokens", [2, 40])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_scores(moe, tokens, scoring, renormalize, bias):
    check(moe, *make(3, tokens, 160, 640, "f32", "f32", bias), 6, scoring, renormalize, 2.5)


@pytest.mark.parametrize("tokens", [1, 18])
def test_equal_scores_take_the_lowest_index(moe, tokens):
    # Scores are small whole numbers, which every order of summation gives exactly.
    g = torch.Generator().manual_seed(5)
    x = torch.ones(tokens, 64)
    w = torch.zeros(200, 64)
    w[:, 0] = torch.randint(-2, 3, (200,), generator=g).float()
    w[7, 1], w[7, 0] = 0.0, -0.0
    check(moe, x, w, None, 16)
    check(moe, x, w, None, 16, "sigmoid")
    check(moe, x, torch.zeros(200, 64), None, 16)
    check(moe, x, torch.zeros(200, 64), torch.zeros(200), 16)


@pytest.mark.parametrize("tokens", [1, 12])
def test_scores_far_apart_and_huge(moe, tokens):
    x, w, _ = make(6, tokens, 96, 256, "f32", "f32")
    check(moe, x * 1e4, w, None, 4, renormalize=False)       # all but the first probability near or at zero
    weights, ids = moe.route((x * 1e30).cuda(), (w * 1e30).cuda(), 4)
    s = (x.double() * 1e60) @ w.double().T
    assert torch.equal(ids[:, 0].cpu().long(), s.argmax(1))
    assert bool((weights[:, 0] == 1).all()) and bool((weights[:, 1:] == 0).all())


@pytest.mark.parametrize("tokens", [2, 20])
def test_nan_comes_last_and_stays_in_its_token(moe, tokens):
    x, w, _ = make(7, tokens, 40, 512, "f32", "f32")
    w[3, 5] = float("nan")
    clean = w.clone()
    clean[3] = 0
    weights, ids = moe.route(x.cuda(), w.cuda(), 16, scoring="sigmoid")
    s = x.double() @ clean.double().T
    s[:, 3] = -float("inf")
    assert torch.equal(ids.cpu().long(), torch.sort(s, dim=1, descending=True, stable=True).indices[:, :16])
    x[1, 9] = float("nan")
    weights, ids = moe.route(x.cuda(), clean.cuda(), 8)
    ids = ids.cpu()
    assert sorted(set(ids[1].tolist())) == sorted(ids[1].tolist()) and 0 <= int(ids.min()) and int(ids.max()) < 40
    keep = [i for i in range(tokens) if i != 1]
    want, at = M.route(x[keep].double().numpy(), clean.double().numpy(), 8, None, "softmax", True, 1.0)
    assert np.array_equal(ids[keep].numpy(), at)
    assert np.abs(weights.cpu().numpy()[keep] / want - 1).max() <= TOL


def test_graph_and_outputs_of_the_caller(moe):
    x, w, b = (t.cuda() for t in make(8, 20, 128, 2048, "bf16", "bf16", True))
    weights, ids = torch.empty(20, 8, device="cuda"), torch.empty(20, 8, device="cuda", dtype=torch.int32)
    moe.route(x, w, 8, bias=b, weights=weights, ids=ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.route(x, w, 8, bias=b, weights=weights, ids=ids)
    for seed in range(3):
        x.copy_(make(20 + seed, 20, 128, 2048, "bf16", "bf16")[0])
        graph.replay()
        torch.cuda.synchronize()
        want = moe.route(x, w, 8, bias=b)
        assert torch.equal(want[0], weights) and torch.equal(want[1], ids)


def test_no_tokens(moe):
    x, w, _ = make(9, 0, 16, 64, "f32", "f32")
    weights, ids = moe.route(x.cuda(), w.cuda(), 4)
    assert weights.shape == ids.shape == (0, 4)


def test_many_tokens(moe):
    # More token tiles than an axis of 16 bits holds.
    tokens = 16 * 65536 - 3
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, 16, device="cuda", generator=g)
    w = torch.randn(8, 16, device="cuda", generator=g)
    weights, ids = moe.route(x, w, 2)
    at = torch.sort(torch.matmul(x.double(), w.double().t()), dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(ids.long(), at)
