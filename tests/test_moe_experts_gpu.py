"""GPU tests of tq2_moe_experts against the definition in float64 (tests/moe_ref.py, which carries the bound).

Each projection keeps 1e-5 * sum |x w|: sums over a scale's columns are whole numbers, joined and scaled in four f32
roundings of 2^-24, and a row meets fewer than 70 of them in a wave and 16 waves.  Beside that x is rounded to 31 bits.
A 16-bit output adds half a step of itself.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import moe_ref as M  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TOL = 1e-5


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    from gemv_tq2_g128_amd import moe as mod
    return mod


class Case:
    def __init__(self, seed, tokens, top_k, experts, hidden, inter, fmt="q4", group=128, act="f32", residual=False,
                 ids=None):
        from gemv_tq2_g128_amd import tq2
        rng = np.random.default_rng(seed)
        self.count, self.kind = experts, TYPES[act]
        if fmt == "q4":
            up, down = (M.q4_weight(rng, experts, n, k, group) for n, k in ((2 * inter, hidden), (hidden, inter)))
            self.up, self.down = M.q4_values(up), M.q4_values(down)
            self.weights_on = [tuple(torch.from_numpy(a).cuda() for a in w) for w in (up, down)]
            self.named = None
        else:
            up, down = (M.ternary_weight(rng, experts, n, k) for n, k in ((2 * inter, hidden), (hidden, inter)))
            self.up = M.ternary_values(up, experts, 2 * inter, hidden)
            self.down = M.ternary_values(down, experts, hidden, inter)
            self.weights_on = [tq2.reformat_aos_to_soa(torch.from_numpy(w).cuda(), experts * n, k)
                               for w, n, k in ((up, 2 * inter, hidden), (down, hidden, inter))]
            self.named = experts
        self.x = torch.from_numpy(rng.standard_normal((tokens, hidden)).astype(np.float32)).to(self.kind)
        self.residual = torch.from_numpy(rng.standard_normal((tokens, hidden)).astype(np.float32)).to(self.kind) \
            if residual else None
        if ids is None:
            ids = np.stack([rng.permutation(experts)[:top_k] for _ in range(tokens)])
        self.ids = torch.from_numpy(np.asarray(ids, dtype=np.int32).reshape(tokens, top_k))
        w = rng.uniform(0.05, 1.0, (tokens, top_k)).astype(np.float32)
        self.share = torch.from_numpy(w)

    def run(self, moe, **over):
        here = dict(x=self.x, ids=self.ids, weights=self.share, residual=self.residual)
        args = {n: over[n] if n in over else None if t is None else t.cuda() for n, t in here.items()}
        return moe.experts(args["x"], *self.weights_on, args["ids"], args["weights"], experts=self.named,
                           residual=args["residual"], out=over.get("out"))

    def check(self, y):
        torch.cuda.synchronize()
        want, bound = M.experts(self.x.float().numpy(), self.up, self.down, self.ids.numpy(), self.share.numpy(),
                                None if self.residual is None else self.residual.float().numpy(), TOL)
        assert y.dtype == self.kind and y.shape == self.x.shape
        if self.kind != torch.float32:
            bound = bound + (np.abs(want) + bound) * torch.finfo(self.kind).eps / 2 + 2.0 ** -25
        err = np.abs(y.double().cpu().numpy() - want)
        worst = float((err / np.maximum(bound, 1e-30)).max())
        print("worst error of its bound %.3f" % worst, flush=True)
        assert worst <= 1.0


FORMATS = [("q4", 32), ("q4", 64), ("q4", 128), ("tq2", 128)]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("act", list(TYPES))
@pytest.mark.parametrize("residual", [False, True])
def test_types(moe, fmt, group, act, residual):
    c = Case(1, 5, 3, 8, 384, 256, fmt, group, act, residual)
    c.check(c.run(moe))


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("tokens,top_k,experts,hidden,inter", [
    (1, 1, 1, 128, 128), (1, 2, 2, 128, 256), (1, 8, 64, 512, 128), (2, 4, 4, 640, 384), (3, 1, 16, 1152, 640),
    (4, 2, 6, 2176, 128), (7, 6, 12, 256, 1408), (8, 2, 3, 128, 2176), (9, 16, 20, 384, 384), (33, 2, 5, 256, 640),
    (64, 4, 16, 640, 256), (128, 2, 4, 128, 128)])
def test_sizes(moe, fmt, group, tokens, top_k, experts, hidden, inter):
    c = Case(2, tokens, top_k, experts, hidden, inter, fmt, group)
    c.check(c.run(moe))


@pytest.mark.parametrize("fmt,group", [("q4", 64), ("tq2", 128)])
@pytest.mark.parametrize("tokens,hidden,inter", [(9, 7168, 128), (3, 16384, 128), (9, 128, 7168), (2, 128, 16384),
                                                 (5, 4224, 4224)])
def test_long_rows(moe, fmt, group, tokens, hidden, inter):
    # Rows of x that do not all fit LDS at once.
    c = Case(3, tokens, 2, 2, hidden, inter, fmt, group)
    c.check(c.run(moe))


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_all_tokens_on_one_expert(moe, fmt, group):
    c = Case(4, 37, 1, 40, 256, 256, fmt, group, ids=np.full((37, 1), 39))
    c.check(c.run(moe))


@pytest.mark.parametrize("fmt,group", [("q4", 128), ("tq2", 128)])
def test_the_same_expert_twice_and_no_expert(moe, fmt, group):
    ids = [[2, 2, 0], [-1, 1, -1], [-1, -1, -1], [4, 5, 100000], [3, 3, 3], [-2 ** 31, 2 ** 31 - 1, 0]]
    for experts in (4, 40):                          # block rows by expert and by pair
        for residual in (False, True):
            c = Case(5, 6, 3, experts, 256, 384, fmt, group, residual=residual, ids=ids)
            y = c.run(moe)
            c.check(y)
            still = c.residual[2] if residual else torch.zeros(256)
            assert torch.equal(y[2].cpu(), still)


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("residual", [False, True])
def test_many_pairs_with_none_twice_and_beyond(moe, fmt, group, residual):
    # More than 64 pairs, which are sorted by their expert.
    rng = np.random.default_rng(16)
    ids = rng.integers(-2, 13, (50, 4))                  # 11 experts; -2, -1, 11 and 12 are none
    ids[3] = [5, 5, 5, 5]
    ids[7] = [-1, 11, -2 ** 31, 2 ** 31 - 1]
    ids[20:45, 0] = 2
    c = Case(17, 50, 4, 11, 384, 256, fmt, group, residual=residual, ids=ids)
    y = c.run(moe)
    c.check(y)
    assert torch.equal(y[7].cpu(), c.residual[7] if residual else torch.zeros(384))
    none = c.run(moe, ids=torch.full((50, 4), -1, dtype=torch.int32, device="cuda"))
    assert torch.equal(none.cpu(), c.residual if residual else torch.zeros(50, 384))


def test_two_calls_at_once(moe):
    for tokens in (3, 40):
        cases = [Case(18 + i, tokens, 4, 16, 512, 384, "tq2", act="bf16") for i in range(2)]
        on = [dict(x=c.x.cuda(), ids=c.ids.cuda(), weights=c.share.cuda()) for c in cases]
        want = [c.run(moe, **t) for c, t in zip(cases, on)]
        torch.cuda.synchronize()
        streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
        for _ in range(8):
            for i, stream in enumerate(streams):
                with torch.cuda.stream(stream):
                    got[i].append(cases[i].run(moe, **on[i]))
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(g, want[i]) for g in got[i])


def test_most_tokens_and_places(moe):
    c = Case(6, 128, 16, 48, 128, 128)
    c.check(c.run(moe))


def test_one_token_among_many_experts(moe):
    c = Case(7, 1, 16, 1024, 128, 128, "tq2")
    c.check(c.run(moe))


@pytest.mark.parametrize("alias", ["x", "residual"])
def test_in_place(moe, alias):
    c = Case(8, 6, 2, 8, 256, 256, residual=True)
    t = {"x": c.x.cuda(), "residual": c.residual.cuda()}
    y = c.run(moe, out=t[alias], **t)
    assert y is t[alias]
    c.check(y)


@pytest.mark.parametrize("fmt", ["q4", "tq2"])
def test_rows_that_are_not_finite_stay_by_themselves(moe, fmt):
    c = Case(9, 6, 2, 3, 256, 256, fmt)
    y = c.run(moe)
    x = c.x.clone()
    x[1, 7], x[4, 200] = float("nan"), float("inf")
    z = c.run(moe, x=x.cuda())
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], z[keep])
    assert bool(torch.isnan(z[1]).all()) and not bool(torch.isfinite(z[4]).any())


def test_scales_of_x_and_repetition(moe):
    for power in (-60, -20, 20):
        c = Case(10, 4, 2, 5, 512, 256)
        c.x = c.x * 2.0 ** power
        c.up = c.up                                 # silu is linear near zero and for large positive values
        y = c.run(moe)
        c.check(y)
        assert torch.equal(y, c.run(moe))


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_a_column_far_above_the_others(moe, fmt, group):
    # Columns of 1e6 among those of 1, one of them under weights of zero (codes 8 and 1 stand for zero).
    c = Case(14, 3, 2, 2, 384, 256, fmt, group)
    c.x[:, 70], c.x[1, 200] = 1e6, -1e6
    c.up[:, :, 70] = 0
    if fmt == "q4":
        c.weights_on[0][0][:, :, 35] = c.weights_on[0][0][:, :, 35] & 0xF0 | 8
    else:
        from gemv_tq2_g128_amd import tq2
        blocks = M.ternary_weight(np.random.default_rng(14), 2, 512, 384)     # the case's own, drawn first
        fields = blocks.reshape(2, 512, 3, 34)
        fields[:, :, 0, 70 // 4] = fields[:, :, 0, 70 // 4] & (0xFF - (3 << 2 * (70 % 4))) | 1 << 2 * (70 % 4)
        c.weights_on[0] = tq2.reformat_aos_to_soa(torch.from_numpy(blocks).cuda(), 2 * 512, 384)
    c.check(c.run(moe))


@pytest.mark.parametrize("fmt", ["q4", "tq2"])
def test_rows_of_zeros_and_tiny_values(moe, fmt):
    c = Case(15, 4, 2, 3, 256, 256, fmt)
    c.x[0], c.x[1, 128:], c.x[2] = 0, 0, c.x[2] * 1e-38
    y = c.run(moe)
    c.check(y)
    assert bool((y[0] == 0).all())


def test_graph_another_stream_and_caller_memory(moe):
    c = Case(11, 9, 4, 16, 512, 384, "tq2", act="bf16", residual=True)
    x, ids, share, res = c.x.cuda(), c.ids.cuda(), c.share.cuda(), c.residual.cuda()
    out = torch.empty_like(x)
    run = lambda: c.run(moe, x=x, ids=ids, weights=share, residual=res, out=out)  # noqa: E731
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    stream.synchronize()
    c.check(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    rng = np.random.default_rng(3)
    for _ in range(3):
        x.copy_(torch.from_numpy(rng.standard_normal(x.shape).astype(np.float32)))
        ids.copy_(torch.from_numpy(rng.integers(-1, 16, ids.shape).astype(np.int32)))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.run(moe, x=x, ids=ids, weights=share, residual=res))


def test_no_tokens(moe):
    c = Case(12, 0, 2, 4, 128, 128, ids=np.zeros((0, 2)))
    assert c.run(moe).shape == (0, 128)


def test_routed_experts(moe):
    """Both operators in turn, as a layer uses them."""
    c = Case(13, 11, 4, 24, 512, 256, act="bf16", residual=True)
    g = torch.Generator().manual_seed(3)
    w = torch.randn(24, 512, generator=g) * 0.08
    share, ids = moe.route(c.x.cuda(), w.cuda(), 4, scale=1.5)
    y = c.run(moe, ids=ids, weights=share)
    want, at = M.route(c.x.double().numpy(), w.numpy(), 4, None, "softmax", True, 1.5)
    assert np.array_equal(ids.cpu().numpy(), at)
    c.ids, c.share = ids.cpu(), share.cpu()
    c.check(y)
