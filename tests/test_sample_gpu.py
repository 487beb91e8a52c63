"""GPU tests of tq2_sample against the definition in float64 (tests/sample_ref.py).

Tokens have to be equal.  e is held in units of 2^-43 of the largest (half a unit each, n tokens), so that a running sum
is off by n 2^-44 and the share of the whole that it is compared with by as much: n 2^-43 together, in units of the
largest e.  The exponentials' own 2^-47 and the sums' roundings of 2^-53 add less than 2^-44 of the whole sum, which is
below n.  Inputs are checked, on the host, to lie further than 1.5 n 2^-43 from every border; their seeds were chosen for
nothing else.  min_p is compared with one e: 2^-47 of it.
Log probabilities: one rounding to f32 of a number below 64 (2^-19 at most), beside n 2^-43 of the sum.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import sample_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sampling():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    from gemv_tq2_g128_amd import sampling as mod
    return mod


def column(v, rows):
    return [float(x) for x in v] if isinstance(v, torch.Tensor) else [v] * rows


def check(sampling, logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """logits on the host, in their type; settings numbers or host tensors."""
    rows, vocab = logits.shape
    def on(v):
        return v.cuda() if isinstance(v, torch.Tensor) else v
    logprob = torch.full((rows,), 7.0, device="cuda")
    ids = sampling.sample(logits.cuda(), u.cuda(), on(temperature), on(top_k), on(top_p), on(min_p), logprob=logprob)
    torch.cuda.synchronize()
    assert ids.dtype == torch.int32 and ids.shape == (rows,)
    settings = [column(v, rows) for v in (temperature, top_k, top_p, min_p)]
    for r in range(rows):
        row = np.nan_to_num(logits[r].double().numpy(), nan=-np.inf, posinf=np.inf, neginf=-np.inf)
        token, lp, margin = R.sample(row, float(u[r]), *(s[r] for s in settings))
        assert margin > 1.5 * vocab * 2.0 ** -43, "row %d: the input lies on a border" % r
        assert int(ids[r]) == token, (r, [s[r] for s in settings], float(u[r]))
        got = float(logprob[r])
        assert got == lp or abs(got - lp) <= 2.0 ** -19 + vocab * 2.0 ** -43, (r, got, lp)
    return ids


def logits_of(seed, rows, vocab, kind="f32", spread=2.0, sure=8.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * spread
    for r in range(rows):
        x[r, torch.randint(0, vocab, (12,), generator=g)] = sure + torch.randn(12, generator=g)
    return x.to(TYPES[kind]), torch.rand(rows, generator=g)


SETTINGS = [dict(), dict(temperature=0.0), dict(temperature=0.5), dict(top_k=1), dict(top_k=7), dict(top_k=50, top_p=0.9),
            dict(top_p=0.3), dict(top_p=0.95, temperature=1.7), dict(min_p=0.1), dict(min_p=0.02, top_p=0.8, top_k=400),
            dict(top_p=0.0), dict(min_p=1.0), dict(top_k=3000), dict(temperature=100.0), dict(temperature=0.01)]


@pytest.mark.parametrize("settings", SETTINGS, ids=str)
@pytest.mark.parametrize("kind", list(TYPES))
def test_settings(sampling, settings, kind):
    check(sampling, *logits_of(1, 6, 5003, kind), **settings)


@pytest.mark.parametrize("vocab", [1, 2, 3, 5, 7, 8, 9, 63, 64, 65, 511, 513, 1000, 2047, 2049, 4099, 32000, 100003])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_vocabularies(sampling, vocab, kind):
    logits, u = logits_of(2, 5, vocab, kind)
    check(sampling, logits, u, top_k=40, top_p=0.9)
    check(sampling, logits, u)
    check(sampling, logits, u, top_p=0.97)


@pytest.mark.parametrize("rows", [1, 2, 31, 300])
def test_rows_of_their_own_settings(sampling, rows):
    logits, u = logits_of(3, rows, 3001, "f16")
    g = torch.Generator().manual_seed(rows)
    def pick(values, dtype=torch.float32):
        return torch.tensor(values, dtype=dtype)[torch.randint(0, len(values), (rows,), generator=g)]
    check(sampling, logits, u, pick([0.0, 0.4, 1.0, 2.0, -1.0]), pick([-3, 0, 1, 5, 100, 10 ** 6], torch.int32),
          pick([0.5, 0.9, 1.0, 2.0, -0.5]), pick([0.0, 0.0, 0.05, -1.0, 3.0]))


def test_nan_settings_are_none(sampling):
    logits, u = logits_of(4, 3, 700)
    nan = torch.full((3,), float("nan"))
    plain = check(sampling, logits, u)
    got = sampling.sample(logits.cuda(), u.cuda(), 1.0, 0, nan.cuda(), nan.cuda())
    assert torch.equal(plain, got)
    greedy = sampling.sample(logits.cuda(), u.cuda(), nan.cuda())
    assert torch.equal(greedy.cpu().long(), logits.argmax(1))
    low = sampling.sample(logits.cuda(), nan.cuda())
    assert torch.equal(low.cpu().long(), logits.argmax(1))


def test_random_numbers_at_their_ends(sampling):
    logits, _ = logits_of(5, 1, 900)
    logits = logits.repeat(5, 1)
    u = torch.tensor([0.0, 1.0, 5.0, -3.0, float("inf")])
    order = torch.sort(logits[0], descending=True, stable=True).indices
    ids = sampling.sample(logits.cuda(), u.cuda(), top_k=20).cpu().tolist()
    assert ids == [int(order[0]), int(order[19]), int(order[19]), int(order[0]), int(order[19])]


@pytest.mark.parametrize("vocab", [70, 5000, 90001])
def test_equal_logits_go_by_index(sampling, vocab):
    # Whole numbers of equal weight: u * n is the index, up to the 24 bits of u.
    u = (torch.arange(9) * 2 + 1).float() / 18
    logits = torch.full((9, vocab), 3.25)
    ids = check(sampling, logits, u)
    assert ids.tolist() == [int(x * vocab) for x in u.tolist()]
    check(sampling, logits, u, top_k=vocab // 3)
    check(sampling, logits, u, top_p=0.51)
    two = logits.clone()
    two[:, ::2] = 2.5
    two[:, 3] = -0.0
    check(sampling, two, u, top_k=vocab // 2 + vocab // 7)


def test_one_far_above_a_crowd(sampling):
    # The bins are spread to the one above; the crowd shares few of them, more than the list holds.
    g = torch.Generator().manual_seed(6)
    logits = 1e-3 * torch.randn(8, 60000, generator=g)
    logits[:, 77] = 9.0
    u = torch.rand(8, generator=g)
    check(sampling, logits, u)
    check(sampling, logits, u, top_k=30000)
    check(sampling, logits, u, top_p=0.9)
    check(sampling, logits.half(), u, top_k=20000, top_p=0.7)


def test_masked_and_special_values(sampling):
    inf, nan = float("inf"), float("nan")
    logits, u = logits_of(7, 8, 1200)
    logits[0] = -inf
    logits[1] = nan
    logits[2, 1:] = -inf
    logits[3, ::2] = -inf
    logits[4, 5::3] = nan
    logits[5, 100], logits[5, 900], logits[5, 901] = inf, inf, nan
    logits[6] = torch.finfo(torch.float32).min
    logits[7, 600:] = torch.finfo(torch.float32).min
    ids = check(sampling, logits, u)
    assert ids[:3].tolist() == [-1, -1, 0] and int(ids[5]) in (100, 900)
    check(sampling, logits, u, top_k=30, top_p=0.9, min_p=0.01)
    check(sampling, logits, u, temperature=0.0)
    lowest = torch.full((2, 50), torch.finfo(torch.float32).min)
    lowest[1, 7] = torch.finfo(torch.float32).max
    check(sampling, lowest, u[:2])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
def test_strided_rows_at_any_place(sampling, kind, offset):
    logits, u = logits_of(8, 4, 4097, kind)
    wide = torch.full((4 * 4100 + 64,), float("inf"), dtype=TYPES[kind], device="cuda")
    view = wide.as_strided((4, 4097), (4099, 1), offset)
    view.copy_(logits)
    want = check(sampling, logits, u, top_p=0.9)
    assert torch.equal(sampling.sample(view, u.cuda(), top_p=0.9), want)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("temperature", [1e-38, 1e-30, 1e-3, 1.0, 1e30, float("inf")])
def test_rows_of_the_lowest_values_at_any_temperature(sampling, kind, temperature):
    # Logits times the grid of bins pass the largest f32, or all fall into one bin; around the rows lies +infinity.
    low, rows, vocab = torch.finfo(TYPES[kind]).min, 6, 1003
    logits = torch.full((rows, vocab), low, dtype=TYPES[kind])
    logits[1, ::3] = -float("inf")
    logits[2, 500] = low / 2
    logits[3, 700:] = low / 2
    logits[4] = -torch.arange(vocab).to(TYPES[kind]) - 30
    logits[5, 77] = float("inf")
    u = (torch.arange(rows) * 2 + 1).float() / 13
    around = torch.full((rows, 3 * vocab), float("inf"), dtype=TYPES[kind], device="cuda")
    around[:, vocab:2 * vocab] = logits.cuda()
    heat = torch.full((rows,), temperature)
    for settings in (dict(), dict(top_k=40), dict(top_k=600), dict(top_p=0.7), dict(min_p=0.2)):
        want = check(sampling, logits, u, heat, **settings)
        assert torch.equal(sampling.sample(around[:, vocab:2 * vocab], u.cuda(), heat.cuda(), **settings), want)


def test_subnormal_logits(sampling):
    tiny = torch.arange(900).float().repeat(3, 1) * 2.0 ** -149
    u = torch.tensor([0.11, 0.52, 0.93])
    check(sampling, tiny, u)
    check(sampling, tiny, u, top_k=300)
    check(sampling, tiny, u, temperature=1e-36, min_p=0.5)


def test_one_row_for_many_draws(sampling):
    # Rows of stride 0, and of windows that overlap.
    logits, _ = logits_of(11, 1, 5000)
    u = (torch.arange(64) + 0.37).float() / 64
    want = check(sampling, logits.repeat(64, 1), u, top_p=0.9)
    assert torch.equal(sampling.sample(logits.cuda().expand(64, 5000), u.cuda(), top_p=0.9), want)
    windows = logits[0].as_strided((64, 4000), (13, 1))
    want = check(sampling, windows, u)
    assert torch.equal(sampling.sample(logits[0].cuda().as_strided((64, 4000), (13, 1)), u.cuda()), want)


@pytest.mark.parametrize("rows,vocab", [
    (3, 4096), (3, 8191), (3, 8193), (2, 16384), (2, 16390), (2, 32769), (2, 65541), (2, 131075), (300, 32775),
    (140, 65536), (140, 131079)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1, 5, 7])
def test_borders_of_chunks(sampling, rows, vocab, kind, offset):
    # A few distinct rows, at places from which chunks and vectors start differently; some are drawn among the last tokens.
    few = 3
    logits, u = logits_of(12, few, vocab, kind, spread=1.0, sure=3.0)
    logits[1, -3:] = 6.0
    logits[2, :2] = 6.0
    wide = torch.full((rows * (vocab + 3) + 8,), float("inf"), dtype=TYPES[kind], device="cuda")
    view = wide.as_strided((rows, vocab), (vocab + 3, 1), offset)
    view.copy_(logits.cuda()[torch.arange(rows, device="cuda") % few])
    us = u.repeat(rows // few + 1)[:rows].cuda()
    for settings in (dict(), dict(top_k=300), dict(top_p=0.8, top_k=vocab // 2)):
        want = check(sampling, logits, u, **settings)
        got = sampling.sample(view, us, **settings)
        assert torch.equal(got, want.repeat(rows // few + 1)[:rows])


def test_two_calls_at_once(sampling):
    logits, u = (t.cuda() for t in logits_of(13, 32, 50000, "f16"))
    want = [sampling.sample(logits, u, top_p=p) for p in (0.5, 0.95)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(sampling.sample(logits, u, top_p=(0.5, 0.95)[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_graph_another_stream_and_caller_memory(sampling):
    logits, u = (t.cuda() for t in logits_of(9, 16, 32000, "bf16"))
    out, lp = torch.empty(16, dtype=torch.int32, device="cuda"), torch.empty(16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        assert sampling.sample(logits, u, 0.8, 50, 0.95, 0.01, out=out, logprob=lp) is out
    stream.synchronize()
    want = sampling.sample(logits, u, 0.8, 50, 0.95, 0.01)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sampling.sample(logits, u, 0.8, 50, 0.95, 0.01, out=out, logprob=lp)
    for seed in range(3):
        fresh = logits_of(20 + seed, 16, 32000, "bf16")
        logits.copy_(fresh[0])
        u.copy_(fresh[1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sampling.sample(logits, u, 0.8, 50, 0.95, 0.01))


def test_largest_sizes(sampling):
    g = torch.Generator().manual_seed(10)
    logits = torch.randn(2, 1 << 20, generator=g) * 3
    check(sampling, logits, torch.rand(2, generator=g), top_p=0.9)
    check(sampling, logits, torch.rand(2, generator=g), temperature=50.0)
    many = torch.randn(4096, 33, generator=g)
    check(sampling, many, torch.rand(4096, generator=g), top_k=9)
    assert sampling.sample(torch.empty(0, 10, device="cuda"), torch.empty(0, device="cuda")).shape == (0,)


def test_frequencies_follow_the_probabilities(sampling):
    # 4096 rows of one distribution, u evenly spread: each token's count is its share within one.
    p = torch.tensor([0.4, 0.05, 0.3, 0.15, 0.1])
    u = (torch.arange(4096) + 0.5) / 4096
    ids = sampling.sample(p.log().repeat(4096, 1).cuda(), u.cuda())
    counts = torch.bincount(ids.cpu().long(), minlength=5).float()
    assert bool(((counts - p * 4096).abs() <= 1).all()), counts
